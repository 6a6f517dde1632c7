"""Workloads of the 8-bit KV cache operators (dflash_kvq_*).

Four operators over one cache format.  The cache is a pool of pages
[page][kv head][128 slots][128] of e4m3 codes for K and for V, with one int8
exponent per 16 slots and head (value = code * 2^exponent), and a page table
[sequence][page index]:

  append   writes bf16 K/V rows behind a sequence's committed slots; a block
           of 16 slots takes the smallest exponent e in [-40, 40] with
           max |x| <= 448 * 2^e over its rows, committed rows included
           (the pass reads the touched blocks back as bf16)
  attend   softmax(q k / sqrt(128)) v over the cache, and its log-sum-exp;
           every row sees the whole cache, or causally, or the ancestors of a
           draft tree inside the last rows
  score    decay * score + the attention weights each slot received, summed
           over the rows and the query heads of its KV head
  evict    keeps the last `window` slots and the best-scored of the others, in
           slot order, in the pages of another sequence (read back as bf16)

`own` selects between the library's calls and the plain torch form.
"""
import math
import random

import numpy as np
import torch

own = False

HD, PAGE, SUB = 128, 128, 16
E_MIN, E_MAX, CODE_MAX = -40, 40, 448.0
SCALE = 1.0 / math.sqrt(HD)
MASKS = {"none": 0, "causal": 1, "tree": 2}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _case(name, op, batch, hkv, g, **kw):
    c = {"name": name, "op": op, "batch": batch, "hkv": hkv, "g": g, "block": 16, "mask": "none",
         "ctx_lo": 0, "ctx_hi": 0, "ragged_q": False, "budget": 0, "window": 0, "lens": 1}
    c.update(kw)
    return c


def listed():
    return [
        # one step of 32 sequences: the 16 rows of a drafted block each
        _case("append_block16_b32", "append", 32, 8, 4, ctx_lo=512, ctx_hi=4096),
        # a prompt chunk entering the cache behind an odd number of slots
        _case("append_prompt_b3", "append", 3, 8, 4, block=5000, ctx_lo=1, ctx_hi=301),
        # one sequence, block of 16: the latency of a step's attention
        _case("attend_block16_b1_2k", "attend", 1, 8, 4, ctx_lo=2032, ctx_hi=2032),
        # the same at a long context and a small batch
        _case("attend_block16_b8_16k", "attend", 8, 8, 4, ctx_lo=16384, ctx_hi=16384),
        # the verify pass of 32 ragged sequences
        _case("attend_causal16_b32_ragged", "attend", 32, 8, 4, ctx_lo=512, ctx_hi=4096,
              mask="causal"),
        # plain decoding, one token a sequence, long contexts: the largest cache
        _case("attend_token_b32_32k", "attend", 32, 8, 4, block=1, ctx_lo=24000, ctx_hi=32768),
        # a prompt chunk over the slots before it
        _case("attend_chunk1000_b2", "attend", 2, 8, 4, block=1000, ctx_lo=1500, ctx_hi=4097,
              mask="causal"),
        # tree verify: 64 drafted nodes and the root, ragged trees
        _case("attend_tree65_b4", "attend", 4, 8, 4, block=65, ctx_lo=2000, ctx_hi=2300,
              mask="tree", ragged_q=True),
        # weights of a committed block over a long cache
        _case("score_causal16_b8_16k", "score", 8, 8, 4, ctx_lo=16384, ctx_hi=16384,
              mask="causal"),
        # weights of the last token only, seven query heads a KV head, short ragged contexts
        _case("score_token_b5_g7", "score", 5, 4, 7, block=1, ctx_lo=100, ctx_hi=3001),
        # one long sequence cut to an eighth
        _case("evict_b1_32k", "evict", 1, 8, 4, ctx_lo=32768, ctx_hi=32768, budget=4096,
              window=256),
        # a batch cut to half or less
        _case("evict_b32_8k", "evict", 32, 8, 4, ctx_lo=4000, ctx_hi=8192, budget=2000, window=128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "score", "evict"])
    hkv = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 3, 4, 4, 5, 7, 8, 16])
    batch = _log(rng, 1, 32)
    ctx_hi = _log(rng, 20, 32768)
    ctx_lo = rng.randint(max(1, ctx_hi // 4), ctx_hi)
    kw = {"ctx_lo": ctx_lo, "ctx_hi": ctx_hi, "lens": rng.randint(1, 1 << 20)}
    if op == "append":
        kw["block"] = _log(rng, 1, 4096)
        if batch * kw["block"] > 15000:
            batch = max(1, 15000 // kw["block"])
    elif op in ("attend", "score"):
        mask = rng.choice(["none", "causal", "causal", "tree"])
        kw["mask"] = mask
        kw["block"] = rng.randint(2, 100) if mask == "tree" else _log(rng, 1, 800)
        kw["ragged_q"] = rng.random() < 0.5
        # no more query-key pairs and keys than in the largest listed cases
        pairs = 240000000 // (g * hkv * (ctx_hi + kw["block"]))
        kw["block"] = max(1, min(kw["block"], pairs))
        batch = max(1, min(batch, pairs // kw["block"], 7000000 // (hkv * ctx_hi)))
    else:
        ctx_hi = max(ctx_hi, 200)
        ctx_lo = min(ctx_lo, ctx_hi)
        batch = max(1, min(batch, 1600000 // (hkv * ctx_hi)))
        budget = rng.randint(16, max(17, ctx_hi // 2))
        kw.update(ctx_lo=ctx_lo, ctx_hi=ctx_hi, budget=budget,
                  window=rng.randint(0, min(budget, 300)))
    c = _case("", op, batch, hkv, g, **kw)
    del c["name"]
    return c


def _lens(case):
    """(committed slots, rows of the call) of every sequence."""
    r = random.Random(case["lens"] * 7919 + 17)
    ctx = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["batch"])]
    ctx[r.randrange(case["batch"])] = case["ctx_hi"]
    rows = [case["block"]] * case["batch"]
    if case["ragged_q"]:
        rows = [r.randint((x + 1) // 2, x) for x in rows]
    return ctx, rows


def _visible(case, n, ql):
    """Query-key pairs of one sequence and query head (n slots, ql rows)."""
    if case["mask"] == "none":
        return n * ql
    if case["mask"] == "causal":
        return ql * (n - ql) + ql * (ql + 1) // 2
    return ql * (n - ql) + sum(1 + _depth(i) for i in range(ql))


def _depth(i):
    d = 0
    while i > 0:
        i, d = _parent(i), d + 1
    return d


def _parent(i):
    return (i - 1) // 3 if i % 5 else i - 1


def work(case):
    ctx, rows = _lens(case)
    hkv, g, b = case["hkv"], case["g"], case["batch"]
    H = hkv * g
    slot = HD + 1.0 / SUB  # bytes of one slot of K or V of one head
    if case["op"] == "append":
        by = fl = 0
        for c, r in zip(ctx, rows):
            old = c % SUB
            by += hkv * 2 * (r * HD * 2 + (r + old) * (slot + HD * 2) + old * slot)
            fl += hkv * 2 * (r + old) * HD * 3
        return {"bytes": int(by), "flops": int(fl)}
    if case["op"] == "evict":
        by = 0
        for c in ctx:
            keep = min(c, case["budget"])
            by += hkv * (4 * c + keep * (2 * 2 * slot + 2 * HD * 2 + 4 + 4))
        return {"bytes": int(by), "flops": int(sum(ctx) * hkv + b * hkv * case["budget"] * HD * 4)}
    by = fl = 0
    for c, r in zip(ctx, rows):
        n = c + r
        vis = _visible(case, n, r)
        if case["op"] == "attend":
            by += hkv * n * 2 * slot + r * H * (HD * 4 + 4)
            fl += 4 * HD * H * vis
        else:
            by += hkv * n * (slot + 8) + r * H * (HD * 2 + 4)
            fl += 2 * HD * H * vis
    return {"bytes": int(by), "flops": int(fl)}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _rows(gen, n, hkv, kind):
    """n rows of K or V as a model makes them: K with a few strong channels, V
    with token magnitudes that differ."""
    x = torch.randn(n, hkv, HD, device="cuda", generator=gen)
    if kind == "k":
        ch = torch.randn(1, hkv, HD, device="cuda", generator=gen).mul_(0.5).exp_()
        x = x * ch
    else:
        x = x * torch.randn(n, hkv, 1, device="cuda", generator=gen).mul_(0.7).exp_()
    return x.to(torch.bfloat16)


def _pow2(e):
    """2^e as fp32, exactly (torch.ldexp goes through a rounded power)."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _encode(x):
    """x [blocks][16][hkv][128] -> (e4m3 codes, exponents [blocks][hkv])."""
    a = x.float().abs().amax(dim=(1, 3))
    m, e = torch.frexp(a / CODE_MAX)  # a / 448 = m * 2^e, m in [0.5, 1)
    e = torch.where(m == 0.5, e - 1, e)
    e = torch.where(a == 0, torch.full_like(e, E_MIN), e).clamp(E_MIN, E_MAX)
    y = x.float() * _pow2(-e)[:, None, :, None]
    return y.clamp(-CODE_MAX, CODE_MAX).to(torch.float8_e4m3fn), e.to(torch.int8)


def _fill(pool, exps, pages, rows):
    """Writes rows [n][hkv][128] into the pages (a list of page ids) of a pool."""
    n, hkv = rows.shape[0], rows.shape[1]
    npg = (n + PAGE - 1) // PAGE
    for p0 in range(0, npg, 64):
        p1 = min(npg, p0 + 64)
        part = torch.zeros((p1 - p0) * PAGE, hkv, HD, device="cuda", dtype=torch.bfloat16)
        src = rows[p0 * PAGE:min(n, p1 * PAGE)]
        part[:src.shape[0]] = src
        c, e = _encode(part.view(-1, SUB, hkv, HD))
        idx = pages[p0:p1].long()
        pool[idx] = (c.view(torch.uint8).view(p1 - p0, PAGE, hkv, HD).permute(0, 2, 1, 3)
                     .contiguous())
        exps[idx] = e.view(p1 - p0, PAGE // SUB, hkv).permute(0, 2, 1).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    ctx, rows = _lens(case)
    B, hkv, g, op = case["batch"], case["hkv"], case["g"], case["op"]
    H, blk = hkv * g, case["block"]
    in_cache = [c + (r if op in ("attend", "score") else 0) for c, r in zip(ctx, rows)]
    top = [c + (r if op != "evict" else 0) for c, r in zip(ctx, rows)]
    pps = (max(top) + PAGE - 1) // PAGE
    if op == "evict":
        pps = max(pps, (case["budget"] + PAGE - 1) // PAGE)
    n_seqs = 2 * B if op == "evict" else B
    need = [(t + PAGE - 1) // PAGE for t in top]
    if op == "evict":
        need += [(case["budget"] + PAGE - 1) // PAGE] * B
    n_pages = sum(need) + 3
    order = torch.randperm(n_pages, device="cuda", generator=gen).to(torch.int32)
    table = torch.full((n_seqs, pps), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, k in enumerate(need):
        table[i, :k] = order[at:at + k]
        at += k
    s = {"case": case, "B": B, "hkv": hkv, "H": H, "blk": blk, "op": op, "pps": pps,
         "table": table, "ctx": ctx, "rows": rows, "max_keys": max(top),
         "kv_lens": torch.tensor(in_cache, dtype=torch.int32, device="cuda"),
         "q_lens": torch.tensor(rows, dtype=torch.int32, device="cuda"),
         "start": torch.tensor(ctx, dtype=torch.int32, device="cuda"),
         "status": torch.zeros(1, dtype=torch.int32, device="cuda")}
    for kind in "kv":
        pool = torch.zeros(n_pages, hkv, PAGE, HD, dtype=torch.uint8, device="cuda")
        exps = torch.zeros(n_pages, hkv, PAGE // SUB, dtype=torch.int8, device="cuda")
        for i, n in enumerate(in_cache):
            if n:
                _fill(pool, exps, table[i], _rows(gen, n, hkv, kind))
        s[kind + "8"], s[kind + "_exp"] = pool, exps
    if op == "append":
        # one row buffer per token holds Q, K and V side by side, as a fused
        # projection leaves them
        s["qkv"] = torch.cat([torch.zeros(B * blk, H, HD, dtype=torch.bfloat16, device="cuda"),
                              _rows(gen, B * blk, hkv, "k"), _rows(gen, B * blk, hkv, "v")],
                             dim=1).view(B, blk, H + 2 * hkv, HD)
        s["read_start"] = s["start"] // SUB * SUB
        s["read_count"] = s["start"] + s["q_lens"] - s["read_start"]
        s["read_rows"] = blk + SUB - 1
    elif op == "evict":
        cap = pps * PAGE
        # accumulated weights: heavy-tailed, with exact ties among the untouched
        sc = torch.randn(n_seqs, hkv, cap, device="cuda", generator=gen).mul_(2.0).exp_()
        drop = torch.rand(n_seqs, hkv, cap, device="cuda", generator=gen) < 0.05
        s["score"] = torch.where(drop, torch.zeros_like(sc), sc)
        s["src"] = torch.randperm(B, device="cuda", generator=gen).to(torch.int32)
        s["kv_lens"] = s["kv_lens"][s["src"].long()].contiguous()
        s["dst"] = torch.arange(B, 2 * B, dtype=torch.int32, device="cuda")
        s["budget"], s["window"] = case["budget"], case["window"]
    else:
        q = torch.randn(B, blk, H, HD, device="cuda", generator=gen)
        s["q"] = (q * 1.5).to(torch.bfloat16)
        s["anc"] = None
        if case["mask"] == "tree":
            s["anc"] = _ancestors(blk)[None].expand(B, -1, -1).contiguous().cuda()
        if op == "score":
            s["lse"] = _attend_plain(s)[1]
            s["score_in"] = torch.rand(B, hkv, pps * PAGE, device="cuda", generator=gen) * 4
            s["decay"] = 0.96875
    return s


def _ancestors(n):
    """Ancestor bit sets [n][words] (int64) of the draft tree."""
    words = (n + 63) // 64
    sets = [1]
    for i in range(1, n):
        sets.append(sets[_parent(i)] | (1 << i))
    out = torch.zeros(n, words, dtype=torch.int64)
    for i, v in enumerate(sets):
        for w in range(words):
            x = (v >> (64 * w)) & ((1 << 64) - 1)
            out[i, w] = x - (1 << 64) if x >= (1 << 63) else x
    return out


# ---------------------------------------------------------------------------
# the plain form
# ---------------------------------------------------------------------------
def _gather(s, kind, seqs, slots):
    """fp32 values [len(seqs)][len(slots[i])][hkv][128] of cache slots."""
    tab = s["table"][seqs]
    pg = torch.gather(tab, 1, (slots // PAGE).clamp(max=s["pps"] - 1)).long().clamp(min=0)
    r = slots % PAGE
    codes = s[kind + "8"].view(torch.float8_e4m3fn)[pg, :, r]
    e = s[kind + "_exp"][pg, :, r // SUB]
    return codes.float() * _pow2(e)[..., None]


def _seen(s):
    """[B][block][n] visibility of slots 0 .. max_keys - 1."""
    n = s["max_keys"]
    k = torch.arange(n, device="cuda")[None, None, :]
    kl = s["kv_lens"].long()[:, None, None]
    ql = s["q_lens"].long()[:, None, None]
    j = torch.arange(s["blk"], device="cuda")[None, :, None]
    seen = (k < kl) & (j < ql)
    i = k - (kl - ql)
    if s["case"]["mask"] == "causal":
        seen = seen & (i <= j)
    elif s["case"]["mask"] == "tree":
        anc = s["anc"]
        ic = i.clamp(0, anc.shape[2] * 64 - 1).expand(-1, s["blk"], -1)
        bit = (torch.gather(anc, 2, ic // 64) >> (ic % 64)) & 1
        seen = seen & ((i < 0) | (bit == 1))
    return seen


def _weights(s, b, seen):
    """Scaled scores of sequence b [hkv][block * g][n], -inf where not seen."""
    slots = torch.arange(s["max_keys"], device="cuda")[None]
    k = _gather(s, "k", torch.tensor([b], device="cuda"), slots)[0]
    g = s["H"] // s["hkv"]
    q = s["q"][b].float().view(s["blk"], s["hkv"], g, HD).permute(1, 0, 2, 3)
    sc = torch.matmul(q.reshape(s["hkv"], -1, HD), k.permute(1, 2, 0)) * SCALE
    m = seen[b][None, :, None, :].expand(-1, -1, g, -1).reshape(1, s["blk"] * g, -1)
    return torch.where(m, sc, torch.full_like(sc, -math.inf))


def _attend_plain(s):
    B, blk, H, hkv = s["B"], s["blk"], s["H"], s["hkv"]
    out = torch.zeros(B, blk, H, HD, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, blk, H), -math.inf, device="cuda")
    seen = _seen(s)
    slots = torch.arange(s["max_keys"], device="cuda")[None]
    for b in range(B):
        sc = _weights(s, b, seen)
        m = sc.amax(dim=-1, keepdim=True)
        m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
        p = torch.exp(sc - m)
        l = p.sum(dim=-1, keepdim=True)
        v = _gather(s, "v", torch.tensor([b], device="cuda"), slots)[0].permute(1, 0, 2)
        v = torch.where((slots[0] < s["kv_lens"][b])[None, :, None], v, torch.zeros_like(v))
        o = torch.matmul(p, v) / torch.where(l > 0, l, torch.ones_like(l))
        out[b] = o.view(hkv, blk, H // hkv, HD).permute(1, 0, 2, 3).reshape(blk, H, HD)
        lse[b] = (m + torch.log(l)).view(hkv, blk, H // hkv).permute(1, 0, 2).reshape(blk, H)
    return out, lse


def _score_plain(s):
    out = s["score_in"].clone()
    seen = _seen(s)
    hkv, blk, g = s["hkv"], s["blk"], s["H"] // s["hkv"]
    for b in range(s["B"]):
        sc = _weights(s, b, seen)
        l = s["lse"][b].view(blk, hkv, g).permute(1, 0, 2).reshape(hkv, blk * g, 1)
        p = torch.where(torch.isinf(sc), torch.zeros_like(sc), torch.exp(sc - l))
        w = p.sum(dim=1)
        n = torch.arange(s["max_keys"], device="cuda") < s["kv_lens"][b]
        new = s["decay"] * s["score_in"][b, :, :s["max_keys"]] + w
        out[b, :, :s["max_keys"]] = torch.where(n[None], new, out[b, :, :s["max_keys"]])
    return out


def _append_plain(s):
    B, blk, hkv = s["B"], s["blk"], s["hkv"]
    nb = (blk + SUB - 1 + SUB - 1) // SUB + 1
    slots = s["read_start"].long()[:, None] + torch.arange(nb * SUB, device="cuda")[None]
    j = slots - s["start"].long()[:, None]
    new = (j >= 0) & (j < s["q_lens"].long()[:, None])
    live = slots < (s["start"] + s["q_lens"]).long()[:, None]
    seqs = torch.arange(B, device="cuda")
    res = []
    for x, kind in ((s["qkv"][:, :, s["H"]:s["H"] + hkv], "k"),
                    (s["qkv"][:, :, s["H"] + hkv:], "v")):
        old = _gather(s, kind, seqs, slots)
        jj = j.clamp(0, blk - 1)
        xin = x[seqs[:, None], jj].float()
        val = torch.where(new[..., None, None], xin,
                          torch.where(live[..., None, None], old, torch.zeros_like(old)))
        c, e = _encode(val.view(B * nb, SUB, hkv, HD))
        c = c.view(torch.uint8).view(B, nb * SUB, hkv, HD)
        bi, si = torch.nonzero(live, as_tuple=True)
        sl = slots[bi, si]
        pg = s["table"][bi, sl // PAGE].long()
        s[kind + "8"][pg, :, sl % PAGE] = c[bi, si]
        s[kind + "_exp"][pg, :, sl % PAGE // SUB] = e.view(B, nb, hkv)[bi, si // SUB]
        back = torch.where(live[..., None, None], _gather(s, kind, seqs, slots),
                           torch.zeros_like(old))
        res.append(back[:, :s["read_rows"]].to(torch.bfloat16))
    return res[0], res[1], s["k_exp"], s["v_exp"]


def _evict_plain(s):
    B, hkv, budget, window = s["B"], s["hkv"], s["budget"], s["window"]
    cap = s["pps"] * PAGE
    src, dst = s["src"].long(), s["dst"].long()
    n = s["kv_lens"].long()
    keep_n = n.clamp(max=budget)
    slot = torch.arange(cap, device="cuda")
    sc = s["score"][src]
    inf = torch.full_like(sc, math.inf)
    key = torch.where((slot[None] >= (n - window)[:, None])[:, None], inf, sc)
    key = torch.where((slot[None] < n[:, None])[:, None], key, -inf)
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(-1, order, slot.expand_as(order).contiguous())
    kept_mask = (rank < keep_n[:, None, None]) & (slot[None] < n[:, None])[:, None]
    pos = kept_mask.long().cumsum(-1) - 1
    kept = torch.full((B, hkv, budget), -1, dtype=torch.int32, device="cuda")
    b, h, i = torch.nonzero(kept_mask, as_tuple=True)
    kept[b, h, pos[b, h, i]] = i.to(torch.int32)
    # scores move along; the destination's other slots start at zero
    s["score"][dst] = 0.0
    at = torch.nonzero(kept >= 0, as_tuple=True)
    s["score"][dst[at[0]], at[1], at[2]] = s["score"][src[at[0]], at[1], kept[at].long()]
    nb = (budget + SUB - 1) // SUB
    idx = torch.zeros(B, hkv, nb * SUB, dtype=torch.long, device="cuda")
    idx[..., :budget] = kept.long()
    live = torch.zeros_like(idx, dtype=torch.bool)
    live[..., :budget] = kept >= 0
    idx = idx.clamp(min=0)
    heads = torch.arange(hkv, device="cuda")[None, :, None]
    res = []
    dslot = torch.arange(nb * SUB, device="cuda")
    for kind in "kv":
        pg = s["table"][src[:, None, None], idx // PAGE].long()
        codes = s[kind + "8"].view(torch.float8_e4m3fn)[pg, heads, idx % PAGE].float()
        e = s[kind + "_exp"][pg, heads, idx % PAGE // SUB]
        val = codes * _pow2(e)[..., None]
        val = torch.where(live[..., None], val, torch.zeros_like(val))
        c, e = _encode(val.view(B * hkv * nb, SUB, 1, HD))
        c = c.view(torch.uint8).view(B, hkv, nb * SUB, HD)
        e = e.view(B, hkv, nb)
        bi, hi, si = torch.nonzero(live, as_tuple=True)
        pg = s["table"][dst[bi], si // PAGE].long()
        s[kind + "8"][pg, hi, si % PAGE] = c[bi, hi, si]
        s[kind + "_exp"][pg, hi, si % PAGE // SUB] = e[bi, hi, si // SUB]
        back = _gather(s, kind, dst, dslot[None].expand(B, -1))
        back = torch.where(live[:, 0, :, None, None], back, torch.zeros_like(back))
        res.append(back[:, :budget].to(torch.bfloat16))
    return kept, keep_n.to(torch.int32), s["score"][dst], res[0], res[1]


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _own_state(s):
    """The handle, outputs and workspace that a program makes once."""
    from block_diffusion_speculative_injection_gb300 import capi
    B, H, hkv, blk = s["B"], s["H"], s["hkv"], s["blk"]
    o = {"capi": capi, "cache": capi.KvqCache(s["k8"], s["v8"], s["k_exp"], s["v_exp"], s["table"],
                                              s["status"])}

    def values(rows):
        return torch.zeros(B, rows, hkv, HD, dtype=torch.bfloat16, device="cuda")
    if s["op"] == "append":
        o["k"], o["v"] = s["qkv"][:, :, H:H + hkv], s["qkv"][:, :, H + hkv:]
        o["kb"], o["vb"] = values(s["read_rows"]), values(s["read_rows"])
    elif s["op"] == "attend":
        o["out"] = torch.zeros(B, blk, H, HD, dtype=torch.bfloat16, device="cuda")
        o["lse"] = torch.full((B, blk, H), -math.inf, device="cuda")
        n = capi.dflash_kvq_attention_workspace(B, H, hkv, blk, s["max_keys"])
        o["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
    elif s["op"] == "score":
        o["out"] = s["score_in"].clone()
    else:
        o["kept"] = torch.empty(B, hkv, s["budget"], dtype=torch.int32, device="cuda")
        o["lens"] = torch.empty(B, dtype=torch.int32, device="cuda")
        o["kb"], o["vb"] = values(s["budget"]), values(s["budget"])
    s["own"] = o
    return o


def _run_own(s):
    o = s.get("own") or _own_state(s)
    capi, cache = o["capi"], o["cache"]
    B, H, blk = s["B"], s["H"], s["blk"]
    if s["op"] == "append":
        capi.dflash_kvq_append(cache, B, blk, None, s["start"], s["q_lens"], o["k"], o["v"])
        capi.dflash_kvq_read(cache, B, s["read_rows"], None, s["read_start"], s["read_count"],
                             o["kb"], o["vb"])
        return o["kb"], o["vb"], s["k_exp"], s["v_exp"]
    if s["op"] == "attend":
        capi.dflash_kvq_attention(cache, B, H, blk, MASKS[s["case"]["mask"]], None, s["kv_lens"],
                                  s["q_lens"], s["anc"], s["max_keys"], s["q"], o["out"],
                                  o["lse"], o["ws"])
        return o["out"], o["lse"]
    if s["op"] == "score":
        capi.dflash_kvq_score(cache, B, H, blk, MASKS[s["case"]["mask"]], None, s["kv_lens"],
                              s["q_lens"], s["anc"], s["max_keys"], s["q"], s["lse"], s["decay"],
                              s["score_in"], o["out"])
        return o["out"]
    capi.dflash_kvq_evict(cache, B, s["src"], s["dst"], s["kv_lens"], s["max_keys"], s["budget"],
                          s["window"], s["score"], o["kept"], o["lens"])
    capi.dflash_kvq_read(cache, B, s["budget"], s["dst"], None, o["lens"], o["kb"], o["vb"])
    return o["kept"], o["lens"], s["score"][B:], o["kb"], o["vb"]


def run(state):
    if own:
        return _run_own(state)
    return {"append": _append_plain, "attend": _attend_plain, "score": _score_plain,
            "evict": _evict_plain}[state["op"]](state)


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def _exp_table():
    """2^e for e = -128 .. 127, indexed by e + 128."""
    return torch.tensor([math.ldexp(1.0, e) for e in range(-128, 128)], dtype=torch.float64).cuda()


def _e4m3_table():
    t = torch.zeros(256, dtype=torch.float64)
    for c in range(256):
        ex, ma = (c >> 3) & 15, c & 7
        v = math.ldexp(ma, -9) if ex == 0 else math.ldexp(8 + ma, ex - 10)
        t[c] = math.nan if (c & 127) == 127 else (-v if c & 128 else v)
    return t.cuda()


def _cache64(s, kind, seq, n, h):
    """Values [n][128] of a sequence's slots 0 .. n - 1 of one head."""
    pages = s["table"][seq, :(n + PAGE - 1) // PAGE].long()
    v = _e4m3_table()[s[kind + "8"][pages, h].int()]
    v = v * _exp_table()[s[kind + "_exp"][pages, h].int() + 128].repeat_interleave(SUB, 1)[..., None]
    return v.reshape(-1, HD)[:n]


def _quant64(x):
    """x [rows][heads][128] of whole blocks: the nearest coded values."""
    b = x.view(-1, SUB, x.shape[1], HD)
    a = b.abs().amax(dim=(1, 3), keepdim=True)
    e = torch.full_like(a, E_MIN)
    for t in range(E_MIN + 1, E_MAX + 1):
        e = torch.where(a > CODE_MAX * 2.0 ** (t - 1), torch.full_like(a, float(t)), e)
    two_e = _exp_table()[e.int() + 128]
    y = b / two_e
    ulp = torch.full_like(y, 2.0 ** -9)
    for t in range(-5, 9):
        ulp = torch.where(y.abs() >= 2.0 ** t, torch.full_like(y, 2.0 ** (t - 3)), ulp)
    y = (torch.round(y / ulp) * ulp).clamp(-CODE_MAX, CODE_MAX)
    return (y * two_e).view_as(x), e[:, 0, :, 0]


def _scores64(s, b, h):
    """Scores [block][g][n] of one sequence and KV head, -inf where not seen."""
    n, ql = int(s["kv_lens"][b]), int(s["q_lens"][b])
    k = _cache64(s, "k", b, n, h)
    g = s["H"] // s["hkv"]
    q = s["q"][b, :ql, h * g:(h + 1) * g].double()
    sc = torch.einsum("jgd,nd->jgn", q, k) / math.sqrt(HD)
    if s["case"]["mask"] != "none":
        ok = torch.ones(ql, n, dtype=torch.bool)
        if s["case"]["mask"] == "causal":
            ok[:, n - ql:] = torch.tril(torch.ones(ql, ql)).bool()
        else:
            ok[:, n - ql:] = False
            for j in range(ql):
                i = j
                while i > 0:
                    ok[j, n - ql + i] = True
                    i = _parent(i)
                ok[j, n - ql] = True
        sc = sc.masked_fill(~ok.cuda()[:, None, :], -math.inf)
    return sc, n, ql


def exact(case, seed):
    s = prepare(case, seed)
    B, hkv, H = s["B"], s["hkv"], s["H"]
    g = H // hkv
    if s["op"] == "attend":
        out = torch.zeros(B, s["blk"], H, HD, dtype=torch.float64, device="cuda")
        lse = torch.full((B, s["blk"], H), -math.inf, dtype=torch.float64, device="cuda")
        for b in range(B):
            for h in range(hkv):
                sc, n, ql = _scores64(s, b, h)
                lz = torch.logsumexp(sc, dim=-1)
                v = _cache64(s, "v", b, n, h)
                p = torch.exp(sc - lz[..., None])
                out[b, :ql, h * g:(h + 1) * g] = torch.einsum("jgn,nd->jgd", p, v)
                lse[b, :ql, h * g:(h + 1) * g] = lz
        return out, lse
    if s["op"] == "score":
        out = s["score_in"].double()
        for b in range(B):
            for h in range(hkv):
                sc, n, ql = _scores64(s, b, h)
                lz = s["lse"][b, :ql, h * g:(h + 1) * g].double()
                w = torch.exp(sc - lz[..., None]).sum(dim=(0, 1))
                out[b, h, :n] = s["decay"] * out[b, h, :n] + w
        return out
    if s["op"] == "append":
        res = []
        for kind, h0 in (("k", H), ("v", H + hkv)):
            back = torch.zeros(B, s["read_rows"], hkv, HD, dtype=torch.float64, device="cuda")
            exps = s[kind + "_exp"].clone()
            for b in range(B):
                c, r = s["ctx"][b], s["rows"][b]
                c0 = c // SUB * SUB
                n = c + r - c0
                x = torch.zeros((n + SUB - 1) // SUB * SUB, hkv, HD, dtype=torch.float64,
                                device="cuda")
                if c > c0:
                    for h in range(hkv):
                        x[:c - c0, h] = _cache64(s, kind, b, c, h)[c0:]
                x[c - c0:n] = s["qkv"][b, :r, h0:h0 + hkv].double()
                y, e = _quant64(x)
                back[b, :n] = y[:n]
                for i in range(e.shape[0]):
                    at = c0 + i * SUB
                    pg = int(s["table"][b, at // PAGE])
                    exps[pg, :, at % PAGE // SUB] = e[i].to(torch.int8)
            res.append((back, exps))
        return res[0][0], res[1][0], res[0][1], res[1][1]
    budget, window = s["budget"], s["window"]
    kept = torch.full((B, hkv, budget), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    score = torch.zeros(B, hkv, s["pps"] * PAGE, dtype=torch.float64, device="cuda")
    vals = [torch.zeros(B, budget, hkv, HD, dtype=torch.float64, device="cuda") for _ in "kv"]
    for b in range(B):
        n, src = int(s["kv_lens"][b]), int(s["src"][b])
        m = min(n, budget)
        lens[b] = m
        for h in range(hkv):
            w0 = max(0, n - window)
            row = s["score"][src, h, :w0].double().cpu().numpy()
            pool = np.lexsort((np.arange(w0), -row))[:m - (n - w0)]
            pick = np.sort(np.concatenate([pool, np.arange(w0, n)]))
            at = torch.from_numpy(pick).cuda()
            kept[b, h, :m] = at.to(torch.int32)
            score[b, h, :m] = s["score"][src, h, at].double()
            for i in range(2):
                x = torch.zeros((m + SUB - 1) // SUB * SUB, 1, HD, dtype=torch.float64,
                                device="cuda")
                x[:m, 0] = _cache64(s, "kv"[i], src, n, h)[at]
                vals[i][b, :m, h] = _quant64(x)[0][:m, 0]
    return kept, lens, score, vals[0], vals[1]
