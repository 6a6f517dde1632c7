"""Workloads of the packed-prompt operators.

A server takes a batch of prompts of different lengths as one packed run of
rows: sequence b's rows are offsets[b] .. offsets[b + 1] - 1.  Four operators
carry such a batch:

  attend   causal (or bidirectional) attention of every prompt over itself,
           grouped heads, head_dim 128, bf16, with the log-sum-exp
  append   the packed K/V rows into a paged cache held in 8 bits (e4m3 codes,
           one power-of-two exponent per 16 slots and head), behind the slots
           that a sequence has already
  pages    pages given back and mapped on the GPU from the requests' lengths:
           page table, free list, and the sequence, position and cache slot
           of every packed row
  logp     log probabilities of given tokens, the entropy of their
           distributions and the best alternatives, from the logits

`own` selects between the library's calls and the plain torch form.
"""
import math
import random

import torch

own = False

HD, PAGE, SUB = 128, 128, 16
E_MIN, E_MAX, CODE_MAX = -40, 40, 448.0


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _attend(name, batch, lo, hi, hkv, g, causal=True, pad=0, lens=1):
    return {"name": name, "op": "attend", "batch": batch, "lo": lo, "hi": hi, "hkv": hkv, "g": g,
            "causal": causal, "pad": pad, "lens": lens}


def _append(name, batch, lo, hi, hkv, ctx, pad=0, lens=1):
    return {"name": name, "op": "append", "batch": batch, "lo": lo, "hi": hi, "hkv": hkv,
            "ctx": ctx, "pad": pad, "lens": lens}


def _pages(name, batch, lo, hi, ctx, spare=64, lens=1):
    return {"name": name, "op": "pages", "batch": batch, "lo": lo, "hi": hi, "ctx": ctx,
            "spare": spare, "lens": lens}


def _logp(name, rows, vocab, dtype, top, unused=0.0, masked=0.0):
    return {"name": name, "op": "logp", "rows": rows, "vocab": vocab, "dtype": dtype, "top": top,
            "unused": unused, "masked": masked}


def listed():
    return [
        # three short prompts of a small model: the latency of a call
        _attend("attend_b3_short", 3, 40, 160, 2, 4),
        # one prompt of 2048 tokens, the usual single-request prefill
        _attend("attend_b1_2048", 1, 2048, 2048, 8, 4),
        # 32 ragged prompts of a busy server, with padding rows behind them
        _attend("attend_b32_ragged", 32, 512, 4096, 8, 4, pad=37),
        # one long prompt: the most work
        _attend("attend_b1_16k", 1, 16384, 16384, 8, 4),
        # bidirectional passages of odd lengths, seven query heads a KV head
        _attend("attend_none_b9_g7", 9, 1, 1999, 4, 7, causal=False),
        # short prompts entering the 8-bit cache behind an odd number of slots
        _append("append_b3_short", 3, 40, 160, 2, 301, pad=5),
        # the K and V of 32 ragged prompts
        _append("append_b32_ragged", 32, 512, 4096, 8, 0),
        # 256 sequences, the pages of a rejected block given back, those of the next one mapped
        _pages("pages_block16_b256", 256, 16, 16, 8192),
        # 32 ragged prompts arriving
        _pages("pages_prompts_b32", 32, 512, 4096, 0),
        # the 16 rows of one verified block, five alternatives each
        _logp("logp_block16_b1", 16, 151936, "f32", 5),
        # the verified blocks of 32 sequences, rows behind the accepted ones unused
        _logp("logp_block16_b32", 512, 151936, "f32", 20, unused=0.25),
        # scoring a prompt of 2048 tokens from 16-bit logits
        _logp("logp_prompt_2048", 2048, 128256, "bf16", 0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "append", "pages", "logp", "logp"])
    lens = rng.randint(1, 1 << 20)
    if op == "logp":
        vocab = _log(rng, 1000, 160000) | rng.choice([0, 0, 1])
        dtype = rng.choice(["f32", "bf16"])
        size = 4 if dtype == "f32" else 2
        rows = max(1, min(_log(rng, 1, 2048), 300000000 // (vocab * size)))
        c = _logp("", rows, vocab, dtype, rng.choice([0, 1, 3, 5, 8, 20, 32]),
                  unused=rng.choice([0.0, 0.25]), masked=rng.choice([0.0, 0.0, 0.9]))
    elif op == "pages":
        batch, hi = _log(rng, 1, 1024), _log(rng, 1, 4096)
        batch = max(1, min(batch, 100000 // hi))
        c = _pages("", batch, rng.randint((hi + 3) // 4, hi), hi, rng.choice([0, 1000, 16000]),
                   spare=rng.choice([64, 1, -8]), lens=lens)
    else:
        hkv = rng.choice([1, 2, 4, 8])
        batch, hi = _log(rng, 1, 64), _log(rng, 1, 16384)
        lo = rng.randint(1, hi)
        pad = rng.choice([0, 0, 1, 130])
        if op == "append":
            batch = max(1, min(batch, 500000 // (hkv * hi)))
            c = _append("", batch, lo, hi, hkv, rng.choice([0, 0, 5, 16, 500]), pad, lens)
        else:
            g = rng.choice([1, 2, 3, 4, 4, 5, 7, 8, 16])
            hi = min(hi, math.isqrt((1 << 33) // (hkv * g)))
            lo = min(lo, hi)
            batch = max(1, min(batch, (1 << 33) // (hkv * g * hi * hi), 600000 // (hkv * g * hi)))
            causal = rng.random() < 0.75
            c = _attend("", batch, lo, hi if causal else (hi * 2 + 2) // 3, hkv, g, causal, pad,
                        lens)
            c["lo"] = min(c["lo"], c["hi"])
    del c["name"]
    return c


def _lens(case):
    """Rows of every sequence; one of them has the most."""
    r = random.Random(case["lens"] * 7919 + 17)
    n = [r.randint(case["lo"], case["hi"]) for _ in range(case["batch"])]
    n[r.randrange(case["batch"])] = case["hi"]
    return n


def _ctx(case):
    """Slots that every sequence has already."""
    r = random.Random(case["lens"] * 104729 + 3)
    return [r.randint((case["ctx"] + 1) // 2, case["ctx"]) for _ in range(case["batch"])]


def work(case):
    op = case["op"]
    if op == "logp":
        size = 4 if case["dtype"] == "f32" else 2
        used = round(case["rows"] * (1 - case["unused"]))
        by = case["rows"] * 4 + used * (case["vocab"] * size + 8 + 8 * case["top"])
        return {"bytes": int(by), "flops": int(used * case["vocab"] * 5)}
    n = _lens(case)
    if op == "attend":
        H, hkv = case["hkv"] * case["g"], case["hkv"]
        pairs = sum(x * (x + 1) // 2 if case["causal"] else x * x for x in n)
        return {"bytes": sum(n) * (H * (2 * HD * 2 + 4) + hkv * 2 * HD * 2),
                "flops": 4 * HD * H * pairs}
    ctx = _ctx(case)
    if op == "append":  # rows in, codes and exponents out, and the touched blocks read back
        slot = HD + 1.0 / SUB
        by = sum(x * (2 * HD + slot) + (x + c % SUB) * (slot + 2 * HD) + 2 * (c % SUB) * slot
                 for x, c in zip(n, ctx)) * 2 * case["hkv"]
        return {"bytes": int(by), "flops": int(sum(n) * 2 * case["hkv"] * HD * 3)}
    new = sum((c + x + PAGE - 1) // PAGE - (c + PAGE - 1) // PAGE for x, c in zip(n, ctx))
    # a row's three numbers, a request's ids, lengths, offsets and counts; a page's entry moved
    # to the free list and back
    return {"bytes": 12 * sum(n) + 40 * case["batch"] + 16 * new,
            "flops": 8 * sum(n) + 16 * case["batch"]}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _offsets(n):
    o = [0]
    for x in n:
        o.append(o[-1] + x)
    return o


def _rows(gen, n, heads, kind):
    """n rows of Q, K or V as a model makes them: K with a few strong channels, V with token
    magnitudes that differ."""
    x = torch.randn(n, heads, HD, device="cuda", generator=gen)
    if kind == "q":
        x = x * 1.5
    elif kind == "k":
        x = x * torch.randn(1, heads, HD, device="cuda", generator=gen).mul_(0.5).exp_()
    else:
        x = x * torch.randn(n, heads, 1, device="cuda", generator=gen).mul_(0.7).exp_()
    return x.to(torch.bfloat16)


def _pow2(e):
    """2^e as fp32, exactly."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _encode(x):
    """x [blocks][16][hkv][128] -> (e4m3 codes, exponents [blocks][hkv])."""
    a = x.float().abs().amax(dim=(1, 3))
    m, e = torch.frexp(a / CODE_MAX)  # a / 448 = m * 2^e, m in [0.5, 1)
    e = torch.where(m == 0.5, e - 1, e)
    e = torch.where(a == 0, torch.full_like(e, E_MIN), e).clamp(E_MIN, E_MAX)
    y = x.float() * _pow2(-e)[:, None, :, None]
    return y.clamp(-CODE_MAX, CODE_MAX).to(torch.float8_e4m3fn), e.to(torch.int8)


def _prepare_attend(s, case, gen):
    n = _lens(case)
    hkv, H = case["hkv"], case["hkv"] * case["g"]
    T = sum(n) + case["pad"]
    # one row buffer per token holds Q, K and V side by side, as a fused projection leaves them
    qkv = torch.cat([_rows(gen, T, H, "q"), _rows(gen, T, hkv, "k"), _rows(gen, T, hkv, "v")], 1)
    s.update(T=T, H=H, hkv=hkv, n=n, off=_offsets(n), offsets=_i32(_offsets(n)), q=qkv[:, :H],
             k=qkv[:, H:H + hkv], v=qkv[:, H + hkv:])


def _prepare_append(s, case, gen):
    n, ctx, hkv, B = _lens(case), _ctx(case), case["hkv"], case["batch"]
    T = sum(n) + case["pad"]
    need = [(c + x + PAGE - 1) // PAGE for c, x in zip(ctx, n)]
    pps, n_pages = max(need), sum(need) + 3
    order = torch.randperm(n_pages, device="cuda", generator=gen).to(torch.int32)
    table = torch.full((B, pps), -1, dtype=torch.int32, device="cuda")
    for i, k in enumerate(need):
        table[i, :k] = order[sum(need[:i]):sum(need[:i + 1])]
    s.update(T=T, hkv=hkv, n=n, ctx=ctx, pps=pps, table=table, off=_offsets(n),
             offsets=_i32(_offsets(n)), start=_i32(ctx),
             status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    for kind in "kv":
        pool = torch.zeros(n_pages, hkv, PAGE, HD, dtype=torch.uint8, device="cuda")
        exps = torch.zeros(n_pages, hkv, PAGE // SUB, dtype=torch.int8, device="cuda")
        for b, c in enumerate(ctx):  # the slots that are there already
            if c:
                k = (c + PAGE - 1) // PAGE
                part = torch.zeros(k * PAGE, hkv, HD, dtype=torch.bfloat16, device="cuda")
                part[:c] = _rows(gen, c, hkv, kind)
                codes, e = _encode(part.view(-1, SUB, hkv, HD))
                at = table[b, :k].long()
                pool[at] = (codes.view(torch.uint8).view(k, PAGE, hkv, HD).permute(0, 2, 1, 3)
                            .contiguous())
                exps[at] = e.view(k, PAGE // SUB, hkv).permute(0, 2, 1).contiguous()
        s[kind + "8"], s[kind + "_exp"] = pool, exps
    kv = torch.cat([_rows(gen, T, hkv, "k"), _rows(gen, T, hkv, "v")], 1)
    s["k"], s["v"] = kv[:, :hkv], kv[:, hkv:]
    # what is read back: the blocks of 16 slots that the new rows touch
    s["read_start"] = s["start"] // SUB * SUB
    s["read_count"] = s["start"] + _i32(n) - s["read_start"]
    s["read_rows"] = max(c % SUB + x for c, x in zip(ctx, n))


def _prepare_pages(s, case, gen):
    n, ctx, B = _lens(case), _ctx(case), case["batch"]
    have = [(c + PAGE - 1) // PAGE for c in ctx]
    need = [(c + x + PAGE - 1) // PAGE for c, x in zip(ctx, n)]
    pps, n_seqs = max(need) + 1, B + 3
    n_free = max(0, sum(need) - sum(have) + case["spare"])
    n_pages = max(1, sum(have) + n_free)
    order = torch.randperm(n_pages, device="cuda", generator=gen).to(torch.int32)
    seq = torch.randperm(n_seqs, device="cuda", generator=gen)[:B].to(torch.int32)
    table = torch.full((n_seqs, pps), -1, dtype=torch.int32, device="cuda")
    mapped = torch.zeros(n_seqs, dtype=torch.int32, device="cuda")
    mapped[seq.long()] = _i32(have)
    owner = seq.long().repeat_interleave(_i32(have).long())
    if owner.numel():
        at = torch.cat([torch.arange(k, device="cuda") for k in have])
        table[owner, at] = order[:owner.numel()]
    free = torch.full((n_pages,), -1, dtype=torch.int32, device="cuda")
    free[:n_free] = order[sum(have):]
    s.update(T=sum(n), n=n, ctx=ctx, pps=pps, n_seqs=n_seqs, n_pages=n_pages, seq=seq, table=table,
             mapped=mapped, free=free, n_free=_i32([n_free]), start=_i32(ctx), counts=_i32(n),
             status=torch.zeros(1, dtype=torch.int32, device="cuda"))


def _prepare_logp(s, case, gen):
    R, V = case["rows"], case["vocab"]
    x = torch.empty(R, V, device="cuda", dtype=torch.float32 if case["dtype"] == "f32"
                    else torch.bfloat16)
    tok = torch.empty(R, dtype=torch.int64, device="cuda")
    for r0 in range(0, R, 256):
        r1 = min(R, r0 + 256)
        y = torch.randn(r1 - r0, V, device="cuda", generator=gen).mul_(2.2)
        if case["masked"]:  # a grammar that leaves some of the vocabulary
            drop = torch.rand(r1 - r0, V, device="cuda", generator=gen) < case["masked"]
            drop[:, :64] = False
            y.masked_fill_(drop, -math.inf)
        # some rows are sure of a token, some hesitate
        sure = torch.randint(0, min(V, 64), (r1 - r0, 1), device="cuda", generator=gen)
        y.scatter_add_(1, sure, 12 * torch.rand(r1 - r0, 1, device="cuda", generator=gen))
        x[r0:r1] = y
        u = torch.rand(r1 - r0, V, device="cuda", generator=gen).clamp_(1e-9, 1 - 1e-7)
        tok[r0:r1] = (y - torch.log(-torch.log(u))).argmax(dim=1)  # drawn from the softmax
    if case["unused"]:  # rows behind those that a block keeps
        tok[round(R * (1 - case["unused"])):] = -1
        tok = tok[torch.randperm(R, device="cuda", generator=gen)]
    s.update(R=R, V=V, top=case["top"], logits=x, tokens=tok.to(torch.int32))


def prepare(case, seed):
    s = {"case": case, "op": case["op"]}
    {"attend": _prepare_attend, "append": _prepare_append, "pages": _prepare_pages,
     "logp": _prepare_logp}[case["op"]](s, case, _gen(seed))
    return s


# ---------------------------------------------------------------------------
# the plain form
# ---------------------------------------------------------------------------
def _attend_plain(s):
    H, hkv, causal = s["H"], s["hkv"], s["case"]["causal"]
    g = H // hkv
    out = torch.zeros(s["T"], H, HD, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((s["T"], H), -math.inf, device="cuda")
    for b, n in enumerate(s["n"]):
        o = s["off"][b]
        k = s["k"][o:o + n].float().permute(1, 2, 0)  # [hkv][128][n]
        v = s["v"][o:o + n].float().permute(1, 0, 2)
        step = max(1, min(n, 400000000 // (H * n)))
        for i0 in range(0, n, step):
            i1 = min(n, i0 + step)
            top = i1 if causal else n  # no row of these sees a later key
            q = s["q"][o + i0:o + i1].float().view(i1 - i0, hkv, g, HD).permute(1, 0, 2, 3)
            x = torch.matmul(q.reshape(hkv, -1, HD), k[:, :, :top]).mul_(1 / math.sqrt(HD))
            if causal:
                i = torch.arange(i0, i1, device="cuda").repeat_interleave(g)
                x.masked_fill_(torch.arange(top, device="cuda")[None] > i[:, None], -math.inf)
            m = x.amax(dim=-1, keepdim=True)
            p = x.sub_(m).exp_()
            l = p.sum(dim=-1, keepdim=True)
            y = torch.matmul(p, v[:, :top]) / l
            out[o + i0:o + i1] = (y.view(hkv, i1 - i0, g, HD).permute(1, 0, 2, 3)
                                  .reshape(i1 - i0, H, HD))
            lse[o + i0:o + i1] = ((m + torch.log(l)).view(hkv, i1 - i0, g).permute(1, 0, 2)
                                  .reshape(i1 - i0, H))
    return out, lse


def _values(s, kind, b, slots):
    """fp32 values [slots][hkv][128] of cache slots of sequence b."""
    pg = s["table"][b, slots // PAGE].long()
    codes = s[kind + "8"].view(torch.float8_e4m3fn)[pg, :, slots % PAGE]
    return codes.float() * _pow2(s[kind + "_exp"][pg, :, slots % PAGE // SUB])[..., None]


def _append_plain(s):
    hkv, res = s["hkv"], []
    for kind in "kv":
        back = torch.zeros(len(s["n"]), s["read_rows"], hkv, HD, dtype=torch.bfloat16,
                           device="cuda")
        for b, (n, c) in enumerate(zip(s["n"], s["ctx"])):
            c0 = c // SUB * SUB
            slots = torch.arange(c0, c + n, device="cuda")
            x = torch.zeros((c + n - c0 + SUB - 1) // SUB * SUB, hkv, HD, device="cuda")
            x[:c - c0] = _values(s, kind, b, slots[:c - c0])
            x[c - c0:c + n - c0] = s[kind][s["off"][b]:s["off"][b] + n].float()
            codes, e = _encode(x.view(-1, SUB, hkv, HD))
            pg = s["table"][b, slots // PAGE].long()
            s[kind + "8"][pg, :, slots % PAGE] = codes.view(torch.uint8).view_as(x)[:c + n - c0]
            first = slots[::SUB]
            pg = s["table"][b, first // PAGE].long()
            s[kind + "_exp"][pg, :, first % PAGE // SUB] = e
            back[b, :c + n - c0] = _values(s, kind, b, slots).to(torch.bfloat16)
        res.append(back)
    return res[0], res[1], s["k_exp"], s["v_exp"]


def _spread(first, size):
    """(entry, index within it) of every element when entry i has size[i] of them."""
    e = torch.repeat_interleave(torch.arange(size.numel(), device=size.device), size)
    return e, torch.arange(e.numel(), device=size.device) - first[e]


def _pages_plain(s):
    seq, start, counts = s["seq"].long(), s["start"].long(), s["counts"].long()
    table, mapped, free, n_free = s["table"], s["mapped"], s["free"], s["n_free"]
    # pages behind the committed slots go back, so that the next ones mapped are these
    keep = (start + PAGE - 1) // PAGE
    give = (mapped[seq].long() - keep).clamp(min=0)
    end = give.cumsum(0)
    e, i = _spread(end - give, give)
    total = end[-1] + n_free[0]
    free[total - 1 - (end - give)[e] - i] = table[seq[e], keep[e] + i]
    table[seq[e], keep[e] + i] = -1
    mapped[seq] = torch.minimum(mapped[seq].long(), keep).to(torch.int32)
    n_free[0] = total
    # pages for the new rows
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    need = ((start + counts + PAGE - 1) // PAGE - mapped[seq]).clamp(min=0)
    end = need.cumsum(0)
    ok = (need == 0) | (end <= n_free[0])
    take = torch.where(ok, need, torch.zeros_like(need))
    e, i = _spread(take.cumsum(0) - take, take)
    taken = n_free[0] - 1 - (end - need)[e] - i
    table[seq[e], mapped[seq[e]].long() + i] = free[taken]
    free[taken] = -1
    mapped[seq] += take.to(torch.int32)
    n_free -= take.sum().to(torch.int32)
    # the packed rows
    row, j = _spread(offsets[:-1], counts)
    pos = start[row] + j
    pg = table[seq[row], (pos // PAGE)].long()
    live = ok[row]

    def pick(x):
        return torch.where(live, x, torch.full_like(x, -1)).to(torch.int32)
    return (offsets.to(torch.int32), torch.where(ok, start + counts, start).to(torch.int32),
            pick(seq[row]), pick(pos), pick(pg * PAGE + pos % PAGE), table, mapped, free, n_free)


def _logp_plain(s):
    R, n, x = s["R"], s["top"], s["logits"]
    tok = s["tokens"].long()
    used = tok >= 0
    logp, entropy = torch.zeros(R, device="cuda"), torch.zeros(R, device="cuda")
    ids = torch.zeros(R, n, dtype=torch.int32, device="cuda")
    best = torch.zeros(R, n, device="cuda")
    for r0 in range(0, R, 256):
        r1 = min(R, r0 + 256)
        y = x[r0:r1].float()
        m = y.amax(dim=1, keepdim=True)
        d = y - m
        p = torch.exp(d)
        total = p.sum(dim=1, keepdim=True)
        lse = torch.log(total)
        t = torch.where(p > 0, p * d, torch.zeros_like(p)).sum(dim=1, keepdim=True)
        u = used[r0:r1]
        logp[r0:r1] = torch.where(u, (d.gather(1, tok[r0:r1, None].clamp(min=0)) - lse)[:, 0], 0.0)
        entropy[r0:r1] = torch.where(u, (lse - t / total)[:, 0], 0.0)
        if n:
            v, i = torch.sort(y, dim=1, descending=True, stable=True)
            ids[r0:r1] = torch.where(u[:, None], i[:, :n], 0).to(torch.int32)
            best[r0:r1] = torch.where(u[:, None], v[:, :n] - m - lse, 0.0)
    return logp, entropy, ids, best


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _own_state(s):
    """The handle and the outputs that a program makes once."""
    from block_diffusion_speculative_injection_gb300 import capi
    o = {"capi": capi}
    if s["op"] == "attend":
        o["out"] = torch.zeros(s["T"], s["H"], HD, dtype=torch.bfloat16, device="cuda")
        o["lse"] = torch.full((s["T"], s["H"]), -math.inf, device="cuda")
        o["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    elif s["op"] == "append":
        o["cache"] = capi.KvqCache(s["k8"], s["v8"], s["k_exp"], s["v_exp"], s["table"],
                                   s["status"])
        for kind in "kv":
            o[kind] = torch.zeros(len(s["n"]), s["read_rows"], s["hkv"], HD, dtype=torch.bfloat16,
                                  device="cuda")
    elif s["op"] == "pages":
        o["pages"] = capi.Pages(s["table"], s["mapped"], s["free"], s["n_free"], s["status"])
        o["offsets"] = torch.empty(len(s["n"]) + 1, dtype=torch.int32, device="cuda")
        o["kv_lens"] = torch.empty(len(s["n"]), dtype=torch.int32, device="cuda")
        for k in ("row_seq", "row_pos", "row_slot"):
            o[k] = torch.empty(s["T"], dtype=torch.int32, device="cuda")
    else:
        o["logp"], o["entropy"] = (torch.zeros(s["R"], device="cuda") for _ in range(2))
        o["ids"] = torch.zeros(s["R"], s["top"], dtype=torch.int32, device="cuda")
        o["best"] = torch.zeros(s["R"], s["top"], device="cuda")
    s["own"] = o
    return o


def _run_own(s):
    o = s.get("own") or _own_state(s)
    capi, op = o["capi"], s["op"]
    if op == "attend":
        capi.dflash_prompt_attention(len(s["n"]), s["case"]["causal"], s["offsets"], s["q"], s["k"],
                                     s["v"], o["out"], o["lse"], o["status"])
        return o["out"], o["lse"]
    if op == "append":
        capi.dflash_kvq_append_packed(o["cache"], len(s["n"]), None, s["start"], s["offsets"],
                                      s["k"], s["v"])
        capi.dflash_kvq_read(o["cache"], len(s["n"]), s["read_rows"], None, s["read_start"],
                             s["read_count"], o["k"], o["v"])
        return o["k"], o["v"], s["k_exp"], s["v_exp"]
    if op == "pages":
        capi.dflash_pages_release(o["pages"], len(s["n"]), s["seq"], s["start"])
        capi.dflash_pages_map(o["pages"], len(s["n"]), s["T"], s["seq"], s["start"], s["counts"],
                              o["offsets"], o["kv_lens"], o["row_seq"], o["row_pos"],
                              o["row_slot"])
        return (o["offsets"], o["kv_lens"], o["row_seq"], o["row_pos"], o["row_slot"], s["table"],
                s["mapped"], s["free"], s["n_free"])
    capi.dflash_token_logprobs(s["logits"], s["tokens"], s["top"], o["logp"], o["entropy"],
                               o["ids"] if s["top"] else None, o["best"] if s["top"] else None)
    return o["logp"], o["entropy"], o["ids"], o["best"]


def run(state):
    if own:
        return _run_own(state)
    return {"attend": _attend_plain, "append": _append_plain, "pages": _pages_plain,
            "logp": _logp_plain}[state["op"]](state)


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def _exact_attend(s):
    H, hkv, causal = s["H"], s["hkv"], s["case"]["causal"]
    g = H // hkv
    out = torch.zeros(s["T"], H, HD, dtype=torch.float64, device="cuda")
    lse = torch.full((s["T"], H), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["n"]):
        o = s["off"][b]
        rows = max(1, 100000000 // n)
        for h in range(H):
            k = s["k"][o:o + n, h // g].double()
            v = s["v"][o:o + n, h // g].double()
            at = 0
            while at < n:
                i = torch.arange(at, min(n, at + min(rows, 1024)), device="cuda")
                end = int(i[-1]) + 1 if causal else n
                x = (s["q"][o + i, h].double() @ k[:end].T) / math.sqrt(HD)
                if causal:
                    seen = torch.arange(end, device="cuda")[None, :] <= i[:, None]
                    x = torch.where(seen, x, torch.full_like(x, -math.inf))
                z = torch.logsumexp(x, dim=1)
                lse[o + i, h] = z
                out[o + i, h] = torch.exp(x - z[:, None]) @ v[:end]
                at = int(i[-1]) + 1
    return out, lse


def _nearest_code(y):
    """y rounded to the values of e4m3: 3 significand bits, smallest exponent -6, ties to even."""
    step = torch.full_like(y, 2.0 ** -9)
    for t in range(-5, 9):
        step = torch.where(y.abs() >= 2.0 ** t, torch.full_like(y, 2.0 ** (t - 3)), step)
    return (torch.round(y / step) * step).clamp(-448, 448)


def _exact_append(s):
    two = torch.tensor([math.ldexp(1.0, e) for e in range(-128, 128)], dtype=torch.float64).cuda()
    value = torch.zeros(256, dtype=torch.float64)
    for c in range(256):
        ex, ma = (c >> 3) & 15, c & 7
        a = math.ldexp(ma, -9) if ex == 0 else math.ldexp(8 + ma, ex - 10)
        value[c] = math.nan if c & 127 == 127 else (-a if c & 128 else a)
    value = value.cuda()
    hkv, res = s["hkv"], []
    for kind in "kv":
        back = torch.zeros(len(s["n"]), s["read_rows"], hkv, HD, dtype=torch.float64, device="cuda")
        exps = s[kind + "_exp"].clone()
        for b, (n, c) in enumerate(zip(s["n"], s["ctx"])):
            old, o = c % SUB, s["off"][b]
            blocks = (old + n + SUB - 1) // SUB
            x = torch.zeros(blocks * SUB, hkv, HD, dtype=torch.float64, device="cuda")
            if old:  # committed rows of the first block
                pg, r = int(s["table"][b, (c - old) // PAGE]), (c - old) % PAGE
                v = value[s[kind + "8"][pg, :, r:r + old].int()]
                v = v * two[s[kind + "_exp"][pg, :, r // SUB].int() + 128][:, None, None]
                x[:old] = v.permute(1, 0, 2)
            x[old:old + n] = s[kind][o:o + n].double()
            x = x.view(blocks, SUB, hkv, HD)
            a = x.abs().amax(dim=(1, 3))
            e = torch.full_like(a, E_MIN)
            for t in range(E_MIN + 1, E_MAX + 1):
                e = torch.where(a > CODE_MAX * 2.0 ** (t - 1), torch.full_like(a, float(t)), e)
            scale = two[e.int() + 128][:, None, :, None]
            back[b, :old + n] = (_nearest_code(x / scale) * scale).view(-1, hkv, HD)[:old + n]
            at = c - old + SUB * torch.arange(blocks, device="cuda")
            exps[s["table"][b, at // PAGE].long(), :, at % PAGE // SUB] = e.to(torch.int8)
        res.append((back, exps))
    return res[0][0], res[1][0], res[0][1], res[1][1]


def _exact_pages(s):
    seq, mapped = s["seq"].tolist(), s["mapped"].tolist()
    table, n_free = s["table"].tolist(), int(s["n_free"])
    free = s["free"].tolist()[:n_free]
    given = []
    for q, c in zip(seq, s["ctx"]):
        keep = -(-c // PAGE)
        for i in range(keep, mapped[q]):
            given.append(table[q][i])
            table[q][i] = -1
        mapped[q] = min(mapped[q], keep)
    free += given[::-1]
    offsets, lens, rows, full = [0], [], [], False
    for q, c, n in zip(seq, s["ctx"], s["n"]):
        need = max(0, -(-(c + n) // PAGE) - mapped[q])
        full = full or need > len(free)
        ok = not (full and need)
        if ok:
            for _ in range(need):
                table[q][mapped[q]] = free.pop()
                mapped[q] += 1
        offsets.append(offsets[-1] + n)
        lens.append(c + n if ok else c)
        for p in range(c, c + n):
            rows.append((q, p, table[q][p // PAGE] * PAGE + p % PAGE) if ok else (-1, -1, -1))
    row = torch.tensor(rows, dtype=torch.int32, device="cuda").view(-1, 3)
    n_free = len(free)
    free += [-1] * (s["n_pages"] - n_free)
    return (_i32(offsets), _i32(lens), row[:, 0].contiguous(), row[:, 1].contiguous(),
            row[:, 2].contiguous(), _i32(table), _i32(mapped), _i32(free), _i32([n_free]))


def _exact_logp(s):
    R, n = s["R"], s["top"]
    logp = torch.zeros(R, dtype=torch.float64, device="cuda")
    entropy = torch.zeros(R, dtype=torch.float64, device="cuda")
    ids = torch.zeros(R, n, dtype=torch.int32, device="cuda")
    best = torch.zeros(R, n, dtype=torch.float64, device="cuda")
    used = torch.nonzero(s["tokens"] >= 0)[:, 0]
    for part in used.split(64):
        x = s["logits"][part].double()
        z = torch.logsumexp(x, dim=1, keepdim=True)
        lp = x - z
        logp[part] = lp.gather(1, s["tokens"][part].long()[:, None])[:, 0]
        entropy[part] = -torch.where(torch.isinf(lp), torch.zeros_like(lp), lp * lp.exp()).sum(1)
        index = torch.arange(s["V"], device="cuda")[None]
        for i in range(n):
            v = x.amax(dim=1, keepdim=True)
            at = torch.where(x == v, index, s["V"]).amin(dim=1)
            ids[part, i] = at.to(torch.int32)
            best[part, i] = (v - z)[:, 0]
            x.scatter_(1, at[:, None], -math.inf)
    return logp, entropy, ids, best


def exact(case, seed):
    s = prepare(case, seed)
    return {"attend": _exact_attend, "append": _exact_append, "pages": _exact_pages,
            "logp": _exact_logp}[s["op"]](s)
