"""Packed rows into the 8-bit KV cache (dflash_kvq_append_packed): the same codes, exponents and
values as dflash_kvq_append gives the sequences one by one; and a packed batch of prompts from its
lengths to its log probabilities."""
import numpy as np
import pytest
import torch

from kvq_util import HD, PAGE, Cache
from oracle import packed as op

pytestmark = pytest.mark.gpu


def capi():
    from block_diffusion_speculative_injection_gb300 import capi as c
    return c


def i32(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")


def filled(heads, n_seqs, pages, old, seed, mapped=None):
    rng = np.random.default_rng(seed)
    c = Cache(heads, n_seqs, pages, seed=seed, mapped=mapped)
    top = max(max(old), 1)
    scale = np.exp(rng.normal(size=(n_seqs, top, 1, 1)) * 2)
    c.append([0] * n_seqs, rng.normal(size=(n_seqs, top, heads, HD)) * scale,
             rng.normal(size=(n_seqs, top, heads, HD)) * scale, old, oracle=False)
    return c


def pool(c):
    return [c.t[k] for k in ("k8", "v8", "ke", "ve")]


@pytest.mark.parametrize("heads,lens,old,lead,pad,seqs", [
    (1, [1], [0], 0, 0, None), (2, [1, 1, 1], [15, 16, 17], 0, 2, None), (3, [0, 5, 0, 40], [3, 9, 0, 127], 1, 0, None),
    (8, [300, 1, 128], [0, 111, 128], 0, 7, [2, 0, 1]), (1, [16, 17, 31, 32, 33], [0, 1, 15, 8, 31], 3, 3, None),
    (2, [0, 0], [4, 4], 0, 1, None),
])
def test_equals_the_batched_call(heads, lens, old, lead, pad, seqs):
    B = len(lens)
    rng = np.random.default_rng(sum(lens) + heads)
    T = lead + sum(lens) + pad
    x = torch.from_numpy(rng.normal(size=(T, 3 * heads + 1, HD)) * np.exp(rng.normal(size=(T, 1, 1)) * 2))
    x = x.to(torch.bfloat16).cuda()
    k, v = x[:, heads:2 * heads], x[:, 2 * heads:3 * heads]
    off = np.cumsum([lead] + lens).tolist()
    ids = seqs or list(range(B))
    a, b = (filled(heads, B, 4, old, 7) for _ in range(2))
    start = [old[q] for q in ids]
    capi().dflash_kvq_append_packed(a.h, B, i32(seqs), i32(start), i32(off), k, v)
    capi().dflash_kvq_check(a.h)
    for q, s, n, o in zip(ids, start, lens, off):
        if n:
            capi().dflash_kvq_append(b.h, 1, n, i32([q]), i32([s]), None, k[None, o:o + n], v[None, o:o + n])
    capi().dflash_kvq_check(b.h)
    assert all(torch.equal(s, t) for s, t in zip(pool(a), pool(b)))


def test_elements_past_32_bits():
    x = torch.empty(1100, 2 ** 14, HD, dtype=torch.bfloat16, device="cuda")
    assert x.numel() > 2 ** 31
    x[1000:].normal_(generator=torch.Generator(device="cuda").manual_seed(0))
    a, b = (filled(2, 2, 2, [3, 70], 1) for _ in range(2))
    off = i32([1023, 1030, 1100])
    capi().dflash_kvq_append_packed(a.h, 2, None, i32([3, 70]), off, x[:, 5:7], x[:, -2:])
    k, v = x[1023:, 5:7].contiguous(), x[1023:, -2:].contiguous()
    capi().dflash_kvq_append_packed(b.h, 2, None, i32([3, 70]), off - 1023, k, v)
    capi().dflash_kvq_check(a.h)
    assert all(torch.equal(s, t) for s, t in zip(pool(a), pool(b)))


def test_many_ragged_sequences():
    rng = np.random.default_rng(11)
    B = 70
    lens = [int(n) for n in rng.integers(0, 60, B)]
    old = [int(n) for n in rng.integers(0, 60, B)]
    x = torch.from_numpy(rng.normal(size=(sum(lens), 4, HD))).to(torch.bfloat16).cuda()
    off = np.cumsum([0] + lens).tolist()
    a, b = (filled(2, B, 1, old, 3) for _ in range(2))
    capi().dflash_kvq_append_packed(a.h, B, None, i32(old), i32(off), x[:, :2], x[:, 2:])
    wide = torch.zeros(B, 60, 4, HD, dtype=torch.bfloat16, device="cuda")
    for i, n in enumerate(lens):
        wide[i, :n] = x[off[i]:off[i] + n]
    capi().dflash_kvq_append(b.h, B, 60, None, i32(old), i32(lens), wide[:, :, :2], wide[:, :, 2:])
    torch.cuda.synchronize()
    assert all(torch.equal(s, t) for s, t in zip(pool(a), pool(b)))


@pytest.mark.parametrize("kw,status", [
    ({"off": [0, 30, 20, 40]}, 5), ({"off": [0, 10, 20, 41]}, 5), ({"off": [-1, 10, 20, 40]}, 5),
    ({"seqs": [0, 3, 1]}, 5), ({"seqs": [0, -1, 1]}, 5), ({"start": [0, -5, 0]}, 5),
    ({"start": [0, 250, 0]}, 2), ({"start": [0, 2 ** 31 - 1, 0]}, 2), ({"mapped": [2, 0, 2]}, 2),
])
def test_bad_entries_set_the_status(kw, status):
    c = filled(2, 3, 2, [1, 1, 1], 5, mapped=kw.get("mapped"))
    capi().dflash_status_check(c.status) if "mapped" not in kw else c.status.zero_()
    x = torch.ones(40, 4, HD, dtype=torch.bfloat16, device="cuda")
    capi().dflash_kvq_append_packed(c.h, 3, i32(kw.get("seqs")), i32(kw.get("start", [0, 0, 0])),
                                    i32(kw.get("off", [0, 10, 20, 40])), x[:, :2], x[:, 2:])
    with pytest.raises(capi().DFlashError) as e:
        capi().dflash_kvq_check(c.h)
    assert e.value.status == status


def test_many_bad_offsets_write_nothing_elsewhere():
    """Sequence 3 is nobody's: its pages stay as they are."""
    rng = np.random.default_rng(0)
    c = filled(2, 4, 2, [1, 1, 1, 100], 5)
    before = [t.clone() for t in pool(c)]
    x = torch.ones(40, 4, HD, dtype=torch.bfloat16, device="cuda")
    for _ in range(30):
        off = rng.integers(-30, 70, 4)
        off[1] = off[2] + 1  # never in order
        capi().dflash_kvq_append_packed(c.h, 3, None, i32([0, 200, 17]), i32(off), x[:, :2], x[:, 2:])
        with pytest.raises(capi().DFlashError):
            capi().dflash_kvq_check(c.h)
    mine = torch.from_numpy(c.table[3]).long().cuda()
    spare = sorted(set(range(before[0].shape[0])) - set(c.table.reshape(-1).tolist()))
    keep = torch.cat([mine, torch.tensor(spare, device="cuda")])
    assert all(torch.equal(a[keep], b[keep]) for a, b in zip(before, pool(c)))


def test_packed_prompts_from_lengths_to_log_probabilities():
    """As a server would, captured once and replayed with other lengths: pages from the lengths,
    K and V into the 8-bit cache, attention of the prompts, log probabilities of their tokens; then
    one token more over the cache."""
    hkv, g, V, B, T, n_pages, pps = 2, 4, 1000, 3, 400, 12, 4
    H = hkv * g
    gen = torch.Generator(device="cuda").manual_seed(0)
    qkv = torch.randn(T, H + 2 * hkv, HD, device="cuda", generator=gen).to(torch.bfloat16)
    head = torch.randn(H * HD, V, device="cuda", generator=gen).mul_(0.05).to(torch.bfloat16)
    tokens = torch.randint(0, V, (T,), device="cuda", generator=gen).to(torch.int32)
    status = i32([0])
    pages = capi().Pages.empty(n_pages, 5, pps, status=status)
    codes = [torch.zeros(n_pages, hkv, PAGE, HD, dtype=torch.uint8, device="cuda") for _ in "kv"]
    exps = [torch.zeros(n_pages, hkv, PAGE // 16, dtype=torch.int8, device="cuda") for _ in "kv"]
    cache = capi().KvqCache(*codes, *exps, pages.tensors[0], status)
    seqs, counts = i32([4, 0, 2]), i32([1, 1, 1])
    off, lens = i32([0] * (B + 1)), i32([0] * B)
    row_seq, row_pos, row_slot = (torch.zeros(T, dtype=torch.int32, device="cuda") for _ in range(3))
    out = torch.zeros(T, H, HD, dtype=torch.bfloat16, device="cuda")
    lse, lp, en = torch.zeros(T, H, device="cuda"), torch.zeros(T, device="cuda"), torch.zeros(T, device="cuda")
    ids, best = torch.zeros(T, 3, dtype=torch.int32, device="cuda"), torch.zeros(T, 3, device="cuda")
    q, k, v = qkv[:, :H], qkv[:, H:H + hkv], qkv[:, H + hkv:]

    def step():
        c = capi()
        c.dflash_pages_release(pages, B, seqs)
        c.dflash_pages_map(pages, B, T, seqs, None, counts, off, lens, row_seq, row_pos, row_slot)
        c.dflash_kvq_append_packed(cache, B, seqs, i32_zero, off, k, v)
        c.dflash_prompt_attention(B, True, off, q, k, v, out, lse, status)
        logits = out.view(T, H * HD) @ head
        c.dflash_token_logprobs(logits, tokens, 3, lp, en, ids, best)
        return logits

    i32_zero = i32([0, 0, 0])
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        logits = step()
    for n in ([130, 1, 200], [5, 260, 129], [0, 399, 1]):
        counts.copy_(i32(n))
        out.zero_()
        graph.replay()
        capi().dflash_status_check(status)
        o = np.cumsum([0] + n)
        assert off.tolist() == o.tolist() and lens.tolist() == n
        used = int(o[-1])
        assert row_seq.tolist() == [q for q, c in zip([4, 0, 2], n) for _ in range(c)] + [-1] * (T - used)
        slot = row_slot[:used].long()
        assert slot.unique().numel() == used
        for x, src in ((0, k), (1, v)):  # the rows lie where the map says, to an e4m3 step
            got = codes[x].view(torch.float8_e4m3fn)[slot // PAGE, :, slot % PAGE].float()
            e = exps[x][slot // PAGE, :, slot % PAGE // 16].float()
            val, want = got * torch.exp2(e)[..., None], src[:used].float()
            assert ((val - want).abs() <= 2.0 ** -4 * want.abs() + torch.exp2(e - 10)[..., None]).all()
        host = [t.double().cpu().numpy() for t in (q, k, v)]
        for b in range(B):
            r = slice(o[b], o[b + 1])
            if n[b]:
                ref, _, mag = op.attend(host[0][r], host[1][r], host[2][r], True)
                err = np.abs(out[r].double().cpu().numpy() - ref)
                assert (err <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -10) * mag).all()
        for r in (0, used - 1):
            w = op.logprobs(logits[r].double().cpu().numpy(), int(tokens[r]), 3)
            assert ids[r].tolist() == w[2] and abs(float(lp[r]) - w[0]) < 1e-4 and abs(float(en[r]) - w[1]) < 1e-3
    # one more token of the second prompt over its cache: near the attention of a prompt with it
    n_new = 399
    nq = torch.randn(1, 1, H, HD, device="cuda", generator=gen).to(torch.bfloat16)
    nkv = torch.randn(1, 2 * hkv, HD, device="cuda", generator=gen).to(torch.bfloat16)
    one, zero, length = i32([1]), i32([0]), i32([n_new])
    capi().dflash_pages_map(pages, 1, 1, zero, length, one, i32([0, 0]), lens[:1].contiguous(), None, None, None)
    capi().dflash_kvq_append_packed(cache, 1, zero, length, i32([0, 1]), nkv[:, :hkv], nkv[:, hkv:])
    dec = torch.zeros(1, 1, H, HD, dtype=torch.bfloat16, device="cuda")
    capi().dflash_kvq_attention(cache, 1, H, 1, capi().MASK_CAUSAL, zero, i32([n_new + 1]), None, None, 512,
                                nq, dec)
    capi().dflash_kvq_check(cache)
    a = int(off[1])
    ref, _, mag = op.attend(*[np.concatenate([h[a:a + n_new], t[0].double().cpu().numpy()[None] if t.dim() == 4
                                              else t.double().cpu().numpy()])
                              for h, t in zip(host, (nq[0], nkv[:, :hkv], nkv[:, hkv:]))], True)
    got = dec[0, 0].double().cpu().numpy()
    # K and V in e4m3 (2^-4 of an element): scores move by about 2^-4 of a standard deviation
    assert np.abs(got - ref[-1]).max() <= 0.25 * mag[-1].max()


def test_host_memory_is_refused():
    """By each call, for each of its arrays, before anything is launched."""
    c, B, T, V = capi(), 2, 20, 50
    cuda = dict(device="cuda")
    ints = lambda *n: torch.zeros(*n, dtype=torch.int32, **cuda)
    rows = lambda h: torch.zeros(T, h, HD, dtype=torch.bfloat16, **cuda)
    status = ints(1)
    pages = c.Pages.empty(4, B, 2, status=status)
    codes = [torch.zeros(4, 2, PAGE, HD, dtype=torch.uint8, **cuda) for _ in "kv"]
    exps = [torch.zeros(4, 2, PAGE // 16, dtype=torch.int8, **cuda) for _ in "kv"]
    cache = c.KvqCache(*codes, *exps, pages.tensors[0], status)
    calls = [
        (lambda *a: c.dflash_pages_map(pages, B, T, *a), [ints(B), ints(B), ints(B), ints(B + 1), ints(B)]
         + [ints(T) for _ in range(3)]),
        (lambda *a: c.dflash_pages_release(pages, B, *a), [ints(B), ints(B)]),
        (lambda *a: c.dflash_kvq_append_packed(cache, B, *a), [ints(B), ints(B), ints(B + 1), rows(2), rows(2)]),
        (lambda *a: c.dflash_prompt_attention(B, True, *a),
         [ints(B + 1), rows(4), rows(2), rows(2), rows(4), torch.zeros(T, 4, **cuda), ints(1)]),
        (lambda x, t, *a: c.dflash_token_logprobs(x, t, 2, *a),
         [torch.zeros(T, V, **cuda), ints(T), torch.zeros(T, **cuda), torch.zeros(T, **cuda), ints(T, 2),
          torch.zeros(T, 2, **cuda)]),
        (c.dflash_status_check, [ints(1)]),
    ]
    for call, args in calls:
        for i in range(len(args)):
            with pytest.raises(c.DFlashError) as e:
                call(*[a.cpu() if j == i else a for j, a in enumerate(args)])
            assert e.value.status == 1, (args[i].shape, i)
    with pytest.raises(c.DFlashError):
        c.dflash_pages_release(c.Pages.empty(4, B, 2, device="cpu"), B)
    torch.cuda.synchronize()
    assert int(status) == 0
