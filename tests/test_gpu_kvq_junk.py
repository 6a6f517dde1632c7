"""Uninitialised memory in the places of the 8-bit cache that no result depends on."""
import numpy as np
import pytest
import torch

from kvq_util import HD, PAGE, Cache, ancestors, bf16
from test_gpu_kvq import check_rows, i32, run_attention
from oracle import kvq as ok

pytestmark = pytest.mark.gpu


def capi():
    from block_diffusion_speculative_injection_gb300 import capi as c
    return c


def fill_exponents(c, junk, seed=0):
    """Every exponent of the pool, before anything is written: one byte, or all 256."""
    rng = np.random.default_rng(seed)
    for x in "kv":
        t = c.t[x + "e"]
        e = rng.integers(-128, 128, tuple(t.shape), dtype=np.int8) if junk is None else \
            np.full(tuple(t.shape), junk, dtype=np.int8)
        t.copy_(torch.from_numpy(e))


@pytest.mark.parametrize("junk", [None, -128, -127, -70, 127])
@pytest.mark.parametrize("lens,block,mask", [
    ([1, 16, 17, 129], 1, "none"), ([300, 5, 128, 64], 16, "causal"), ([1600, 33, 240, 700], 3, "none"),
])
def test_attention_with_junk_exponents_behind_the_last_slot(junk, lens, block, mask):
    c = Cache(2, len(lens), 13, seed=3)
    fill_exponents(c, junk)
    rng = np.random.default_rng(block)
    c.append([0] * len(lens), rng.normal(size=(len(lens), max(lens), 2, HD)),
             rng.normal(size=(len(lens), max(lens), 2, HD)), lens)
    q = rng.normal(size=(len(lens), block, 8, HD))
    q[:, block - 1, 3] = 0  # a row of zeros has the smallest scale
    for ws in (True, False):
        got, lse, qe = run_attention(c, q, mask, lens, ws=ws)
        for b, n in enumerate(lens):
            check_rows(c, qe, got, lse, mask, n, block, b, b)
    capi().dflash_kvq_check(c.h)


@pytest.mark.parametrize("junk", [None, -128, -127, -70, 127])
def test_attention_with_junk_exponents_of_page_zero(junk):
    """An unmapped page counts as unseen, whatever page 0 of the pool holds."""
    c = Cache(1, 1, 3, seed=4, spare=2)
    tab = np.array([[1, 2, 3]], dtype=np.int32)  # page 0 belongs to nobody
    c.h.tensors[4].copy_(torch.from_numpy(tab))
    c.table[:] = tab
    fill_exponents(c, junk)
    rng = np.random.default_rng(8)
    c.append([0], rng.normal(size=(1, 384, 1, HD)), rng.normal(size=(1, 384, 1, HD)))
    c.h.tensors[4][0, 1] = -1
    q = rng.normal(size=(1, 3, 4, HD))
    q[0, 1, 2] = 0
    vis = np.ones((3, 384), dtype=bool)
    vis[:, 128:256] = False
    for ws in (True, False):
        got, lse, qe = run_attention(c, q, "none", [384], ws=ws)
        check_rows(c, qe, got, lse, "none", 384, 3, 0, 0, ok_mask=vis)
        with pytest.raises(capi().DFlashError):
            capi().dflash_kvq_check(c.h)


@pytest.mark.parametrize("mask", ["none", "causal", "tree"])
@pytest.mark.parametrize("g,block,q_lens", [(4, 16, [5, 16, 0]), (8, 40, [33, 1, 20]), (5, 7, [6, 2, 7])])
def test_score_with_junk_rows_past_q_lens(mask, g, block, q_lens):
    """Whatever bits the rows behind a sequence's last one hold, the scores are the same."""
    lens, heads = [300, 140, 90], 2
    c = Cache(heads, 3, 3, seed=6)
    rng = np.random.default_rng(g)
    c.append([0] * 3, rng.normal(size=(3, 300, heads, HD)), rng.normal(size=(3, 300, heads, HD)), lens)
    H = heads * g
    t, _ = bf16(rng.normal(size=(3, block, H, HD)))
    lse = torch.full((3, block, H), 8.0, device="cuda")
    anc = torch.full((3, block, 1), -1, dtype=torch.int64, device="cuda") if mask == "tree" else None
    code = {"none": 0, "causal": 1, "tree": 2}[mask]

    def call():
        out = torch.zeros(3, heads, c.pages * PAGE, device="cuda")
        capi().dflash_kvq_score(c.h, 3, H, block, code, None, i32(lens), i32(q_lens), anc, 300, t, lse,
                                1.0, None, out)
        capi().dflash_kvq_check(c.h)
        return out
    for b, r in enumerate(q_lens):
        t[b, r:] = 0
    want = call()
    assert torch.isfinite(want).all() and (want[0, :, :300] > 0).all()
    junk = torch.from_numpy(rng.integers(-2 ** 15, 2 ** 15, (block, H, HD)).astype(np.int16)).cuda()
    junk = junk.view(torch.bfloat16)
    big = torch.full_like(junk, 1.875 * 2.0 ** 126)
    lone = torch.zeros_like(big)
    lone[..., 77] = 1.875 * 2.0 ** 126
    for rows in (junk, big, lone, torch.full_like(big, float("nan")), torch.full_like(big, float("inf"))):
        for b, r in enumerate(q_lens):
            t[b, r:] = rows[r:]
            lse[b, r:] = float("nan")
        assert torch.equal(call(), want)


def test_evict_with_junk_in_the_list_of_kept_slots():
    """The call whose choice is open (a destination that is another entry's source) may leave
    entries of `kept` unwritten: negative ones must not be read as slots.  The rows that come out
    are open too, but come from the pool's (ones), whose blocks move under their readers, or are
    zero; exponents are the format's."""
    n, budget, window = 20000, 3000, 100
    pages = (n + PAGE - 1) // PAGE
    guard = 8  # exponents of another page lie before the pool's
    c = Cache(1, 3, pages, spare=0)
    room = torch.full((c.t["ke"].shape[0] + guard, 1, 8), 127, dtype=torch.int8, device="cuda")
    room[guard:] = -8
    one = torch.full_like(c.t["k8"], 0x78)  # 256 * 2^-8
    tab = np.arange(3 * pages, dtype=np.int32).reshape(3, pages)
    h = capi().KvqCache(one, one.clone(), room[guard:], room[guard:].clone(), torch.from_numpy(tab).cuda(),
                        c.status)
    g = torch.Generator(device="cuda").manual_seed(5)
    nl = torch.zeros(2, dtype=torch.int32, device="cuda")
    for junk in (-1, -127, -128, -2 ** 31):
        for mk in (n, 1):
            score = torch.rand(3, 1, pages * PAGE, device="cuda", generator=g)
            kept = torch.full((2, 1, budget), junk, dtype=torch.int32, device="cuda")
            capi().dflash_kvq_evict(h, 2, i32([0, 1]), i32([1, 2]), i32([n, n]), mk, budget, window,
                                    score, kept, nl)
            assert nl.tolist() == [budget, budget]
            assert ((kept == junk) | ((kept >= 0) & (kept < n))).all()
            out = torch.empty(2, budget, 1, HD, dtype=torch.bfloat16, device="cuda")
            capi().dflash_kvq_read(h, 2, budget, i32([1, 2]), None, None, out, None)
            assert ((out >= 0) & (out <= 1)).all()
    assert (room[:guard] == 127).all() and (room[guard:] >= -40).all() and (room[guard:] <= 40).all()
    capi().dflash_kvq_check(c.h)


@pytest.mark.parametrize("heads,lens,budget,window", [(3, [9000, 700, 40, 0], 256, 16), (1, [40000], 300, 7)])
def test_evict_updates_lengths_in_place(heads, lens, budget, window):
    """new_lens may be kv_lens: the same slots, rows and scores as with an array of its own."""
    B = len(lens)
    pages = (max(lens) + PAGE - 1) // PAGE
    rng = np.random.default_rng(budget)
    scores = rng.random((2 * B, heads, pages * PAGE)).astype(np.float32)
    runs = []
    for in_place in (False, True, True, True):
        c = Cache(heads, 2 * B, pages, seed=11, spare=0)
        for x in "kv":
            c.t[x + "e"].zero_()
        torch.manual_seed(0)
        c.t["k8"].copy_(torch.randint(0, 0x78, tuple(c.t["k8"].shape), dtype=torch.uint8, device="cuda"))
        c.t["v8"].copy_(torch.randint(0, 0x78, tuple(c.t["v8"].shape), dtype=torch.uint8, device="cuda"))
        score, n = torch.from_numpy(scores).cuda(), i32(lens)
        new = n if in_place else torch.zeros_like(n)
        kept = torch.zeros(B, heads, budget, dtype=torch.int32, device="cuda")
        capi().dflash_kvq_evict(c.h, B, i32(list(range(B))), i32(list(range(B, 2 * B))), n, max(lens),
                                budget, window, score, kept, new)
        capi().dflash_kvq_check(c.h)
        assert new.tolist() == [min(x, budget) for x in lens]
        runs.append((kept, score, c.t["k8"], c.t["v8"], c.t["ke"], c.t["ve"]))
    for b, x in enumerate(lens):
        for h in range(heads):
            pick = ok.evict_pick(scores[b, h], x, budget, window)
            assert runs[0][0][b, h, :len(pick)].tolist() == pick
    for run in runs[1:]:
        for a, z in zip(run, runs[0]):
            assert torch.equal(a, z)


@pytest.mark.parametrize("mask,n,block,g", [("causal", 700, 300, 1), ("causal", 520, 140, 3), ("tree", 640, 130, 2),
                                            ("tree", 300, 200, 1)])
def test_attention_nan_of_v_over_several_partly_seen_pages(mask, n, block, g):
    """Rows see the NaN of V of the slots they see, dim by dim, and no other's."""
    rng = np.random.default_rng(n)
    c = Cache(1, 1, (n + PAGE - 1) // PAGE, seed=n)
    k, v = rng.normal(size=(1, n, 1, HD)), rng.normal(size=(1, n, 1, HD))
    slots = np.sort(rng.choice(np.arange(n - block, n), 12, replace=False))
    dims = rng.choice(HD, 12)
    v[0, slots, 0, dims] = np.nan
    v[0, 5, 0, 77] = np.nan  # seen by every row
    v[0, slots[3], 0, :] = np.nan
    c.append([0], k, v)
    anc = sets = None
    if mask == "tree":
        parents = [-1] + [int(rng.integers(max(0, i - 9), i)) for i in range(1, block)]
        sets, bits = ancestors(parents, (block + 63) // 64)
        anc = bits[None].copy()
    q = rng.normal(size=(1, block, g, HD))
    vis = ok.visible(mask, n, block, sets)
    held = c.val["v"][0, :n]
    nan = (vis.astype(float) @ np.isnan(held[:, 0])) > 0  # [block][128]
    c.val["v"][0, :n] = np.nan_to_num(held)
    for ws in (True, False):
        got, lse, qe = run_attention(c, q, mask, [n], anc=anc, ws=ws)
        assert (np.isnan(got[0]) == nan[:, None]).all()
        ref, ref_lse, mag = ok.attend(qe[0], c.val["k"][0, :n], c.val["v"][0, :n], vis)
        tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -10) * mag + 1e-30
        ok_at = np.broadcast_to(~nan[:, None], ref.shape)
        assert (np.abs(got[0] - ref) <= tol)[ok_at].all()
        assert np.isfinite(lse).all()
