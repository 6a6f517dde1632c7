"""The 8-bit KV cache operators (dflash_kvq_*) against the fp64 oracle.

Codes, exponents, kept slots and read-back values are exact.  Tolerances:

attention  The kernel may hold a weight p with an error of at most 2^-8 p (two
           e4m3 parts: the first is off by at most 2^-4 of the weight's binade,
           the second carries that residual to within one step of it, 2^-8;
           its fp16 form adds 2^-12) and bf16 rounds the result by at most 2^-8 of
           it; scores in fp32 add less than 2^-11.  So
             |out - ref| <= 2^-8 |ref| + (2^-8 + 2^-10) sum_k p_k |v_k|.
lse        fp32 scores: dot products of 128 terms and an exponent, off by at most
           2^-17 of sum |q_d k_d| / sqrt(128) (two e4m3 parts of q leave at most
           2^-18 of max |q| an element), and a sum off by 2^-18.
score      a weight is off by its score's and its lse's error, relatively.
"""
import numpy as np
import pytest
import torch

from kvq_util import HD, PAGE, SUB, Cache, ancestors, bf16
from oracle import kvq as ok

pytestmark = pytest.mark.gpu


def capi():
    from block_diffusion_speculative_injection_gb300 import capi as c
    return c


def i32(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------------------
# append and read
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("heads,starts,rows,counts,pad", [
    (1, [0], 1, None, 0), (2, [0, 15], 16, None, 3), (3, [127, 128, 5], 17, [17, 0, 3], 0),
    (8, [37], 300, None, 32), (1, [111, 3], 2, [1, 2], 1),
])
def test_append_is_exact(heads, starts, rows, counts, pad):
    rng = np.random.default_rng(rows)
    B = len(starts)
    c = Cache(heads, B + 1, 4, seed=rows)
    seqs = [B - b for b in range(B)]
    old = max(starts)
    if old:
        scale = np.exp(rng.normal(size=(B, old, 1, 1)) * 3)
        c.append([0] * B, rng.normal(size=(B, old, heads, HD)) * scale,
                 rng.normal(size=(B, old, heads, HD)) * scale, starts, seqs)
    before = {x: c.codes(x) for x in "kv"}
    scale = np.exp(rng.normal(size=(B, rows, 1, 1)) * 3)
    c.append(starts, rng.normal(size=(B, rows, heads, HD)) * scale,
             rng.normal(size=(B, rows, heads, HD)) / scale, counts, seqs, pad)
    for x in "kv":
        codes, exps = c.codes(x)
        got = c.values(x)
        for b in range(B):
            n = rows if counts is None else counts[b]
            q, end = seqs[b], starts[b] + n
            np.testing.assert_array_equal(got[q, :end], c.val[x][q, :end])
            nb = (end + SUB - 1) // SUB
            np.testing.assert_array_equal(exps[q, :nb], c.exp[x][q, :nb])
            # everything behind is as it was
            np.testing.assert_array_equal(codes[q, end:], before[x][0][q, end:])
            np.testing.assert_array_equal(exps[q, nb:], before[x][1][q, nb:])
        np.testing.assert_array_equal(codes[0], before[x][0][0])  # a sequence not named
    capi().dflash_kvq_check(c.h)
    # read back, with and without one of the outputs, rows past the count kept
    R = rows + 3
    ko = torch.full((B, R, heads, HD), 7.0, dtype=torch.bfloat16, device="cuda")
    vo = ko.clone()
    n = [rows if counts is None else k for k in (counts or [0] * B)]
    capi().dflash_kvq_read(c.h, B, R, i32(seqs), i32(starts), i32(n), ko, vo)
    only = ko.clone().fill_(7.0)
    capi().dflash_kvq_read(c.h, B, R, i32(seqs), i32(starts), i32(n), None, only)
    assert torch.equal(only, vo)
    for t, x in ((ko, "k"), (vo, "v")):
        for b in range(B):
            np.testing.assert_array_equal(t[b, :n[b]].double().cpu().numpy(),
                                          c.val[x][seqs[b], starts[b]:starts[b] + n[b]])
            assert (t[b, n[b]:] == 7.0).all()


def test_append_rolls_back_by_length():
    """A rejected block leaves nothing behind: writing over it from the same
    length gives what writing there at once gives."""
    rng = np.random.default_rng(3)
    base, new = (rng.uniform(1, 2, size=(1, n, 2, HD)) * rng.choice([-1, 1], size=(1, n, 2, HD))
                 for n in (21, 16))
    a, b = Cache(2, 1, 2, seed=1), Cache(2, 1, 2, seed=1)
    for c in (a, b):
        c.append([0], base, base)
    a.append([21], new * 4, new * 4, oracle=False)  # larger values, same binades kept exact
    a.append([21], new, new)
    b.append([21], new, new)
    for x in "kv":
        np.testing.assert_array_equal(a.values(x)[0, :37], b.values(x)[0, :37])
        np.testing.assert_array_equal(a.values(x)[0, :37], a.val[x][0, :37])


def test_append_edges():
    """Zeros, saturation, tiny values, non-finite values."""
    rows = np.zeros((1, 64, 1, HD))
    rows[0, 16, 0, :6] = [1e38, -1e38, 448 * 2.0 ** 40, 2.0 ** 40, 1.0, 0]
    rows[0, 32, 0, :4] = [2.0 ** -50, 2.0 ** -49, 2.0 ** -126, -2.0 ** -48]
    rows[0, 48, 0, :6] = [np.nan, np.inf, -np.inf, 1.0, 448.0, -450.0]
    c = Cache(1, 1, 1)
    c.append([0], rows, rows)
    got = c.values("k")[0, :64]
    np.testing.assert_array_equal(got, c.val["k"][0, :64])
    assert (got[:16] == 0).all() and got[16, 0, 0] == 448 * 2.0 ** 40
    assert np.isnan(got[48, 0, :3]).all() and got[48, 0, 4] == 448.0
    # a later append keeps the NaN and the values
    c.append([57], np.ones((1, 2, 1, HD)), np.ones((1, 2, 1, HD)))
    np.testing.assert_array_equal(c.values("v")[0, :59], c.val["v"][0, :59])


def test_bad_ids_counts_and_pages_are_reported():
    c = Cache(2, 3, 2, mapped=[2, 1, 2])
    before = c.t["k8"].clone()
    one = np.ones((1, 4, 2, HD))
    for kw, status in ((dict(starts=[0], seqs=[3]), 5), (dict(starts=[0], seqs=[-1]), 5),
                       (dict(starts=[-1], seqs=[0]), 5), (dict(starts=[0], counts=[5]), 5),
                       (dict(starts=[0], counts=[-1]), 5), (dict(starts=[256], seqs=[0]), 2),
                       (dict(starts=[128], seqs=[1]), 2), (dict(starts=[2 ** 31 - 2], seqs=[0]), 2)):
        c.append(kw["starts"], one, one, kw.get("counts"), kw.get("seqs"), oracle=False)
        with pytest.raises(capi().DFlashError) as e:
            capi().dflash_kvq_check(c.h)
        assert e.value.status == status, kw
        capi().dflash_kvq_check(c.h)  # cleared
    assert torch.equal(before, c.t["k8"])
    # rows with a page are written (behind whatever the slots before hold), those
    # without are dropped
    want, exps = c.values("k")[1].copy(), c.exp["k"][1]
    ok.append(want, exps, 126, one[0, :2])
    c.append([126], one, one, seqs=[1], oracle=False)
    with pytest.raises(capi().DFlashError):
        capi().dflash_kvq_check(c.h)
    np.testing.assert_array_equal(c.values("k")[1, 112:128], want[112:128])
    out = torch.full((1, 4, 2, HD), 7.0, dtype=torch.bfloat16, device="cuda")
    capi().dflash_kvq_read(c.h, 1, 4, i32([1]), i32([126]), None, out, None)
    np.testing.assert_array_equal(out[0, :2].double().cpu().numpy(), want[126:128])
    assert (out[0, 2:] == 0).all()
    with pytest.raises(capi().DFlashError):
        capi().dflash_kvq_check(c.h)


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
def filled(heads, lens, seed, v_scale=1.0, pages=None, k_scale=1.0):
    """A cache whose sequences hold lens[b] random rows."""
    rng = np.random.default_rng(seed)
    pages = pages or max(1, max((n + PAGE - 1) // PAGE for n in lens))
    c = Cache(heads, len(lens), pages, seed=seed)
    R = max(max(lens), 1)
    k = rng.normal(size=(len(lens), R, heads, HD)) * k_scale
    v = rng.normal(size=(len(lens), R, heads, HD)) * v_scale
    c.append([0] * len(lens), k, v, list(lens))
    return c, rng


def run_attention(c, q, mask, lens, q_lens=None, anc=None, ws=True, lse=True, seqs=None,
                  max_keys=None, pad=0, splits=None):
    """out, lse as fp64 arrays (rows not written keep 9)."""
    B, R, H = q.shape[:3]
    t, exact = bf16(np.concatenate([q, np.zeros((B, R, pad, HD))], axis=2))
    out = torch.full((B, R, H, HD), 9.0, dtype=torch.bfloat16, device="cuda")
    ls = torch.full((B, R, H), 9.0, device="cuda") if lse else None
    mk = max_keys or max(max(lens), 1)
    need = capi().dflash_kvq_attention_workspace(B, H, c.heads, R, mk)
    assert need >= 0
    w = torch.full((need,), 255, dtype=torch.uint8, device="cuda") if ws and need else None
    code = {"none": 0, "causal": 1, "tree": 2}[mask]
    a = None if anc is None else torch.from_numpy(anc).cuda()
    capi().dflash_kvq_attention(c.h, B, H, R, code, i32(seqs), i32(lens), i32(q_lens), a, mk,
                                t[:, :, :H], out, ls, w)
    torch.cuda.synchronize()
    return (out.double().cpu().numpy(), ls.double().cpu().numpy() if lse else None,
            exact[:, :, :H])


def check_rows(c, q, got, lse, mask, n, r, b, seq, sets=None, ok_mask=None):
    vis = ok.visible(mask, n, r, sets) if ok_mask is None else ok_mask
    k, v = c.val["k"][seq, :n], c.val["v"][seq, :n]
    ref, ref_lse, mag = ok.attend(q[b, :r], k, v, vis)
    tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -10) * mag + 1e-30
    assert (np.abs(got[b, :r] - ref) <= tol).all(), float((np.abs(got[b, :r] - ref) / tol).max())
    if lse is not None:
        check_lse(lse[b, :r], ref_lse, q[b, :r], k)
    return ref, ref_lse


def check_lse(got, ref, q, k):
    if got.size == 0:
        return
    seen = np.isfinite(ref)
    np.testing.assert_array_equal(np.isneginf(got), ~seen)
    if k.shape[0]:
        top = np.abs(q).max() * np.abs(k).sum(axis=-1).max() / np.sqrt(HD)
        assert (np.abs(got - ref)[seen] <= 2.0 ** -17 * top + 2.0 ** -18 * (1 + np.abs(ref[seen]))).all()


CASES = [
    # heads, group, lens, block, q_lens, mask
    (2, 4, [1, 40], 1, None, "none"), (1, 1, [128, 129, 127], 1, None, "causal"),
    (2, 4, [16, 300], 16, None, "none"), (1, 4, [17, 256, 640], 16, [16, 1, 7], "causal"),
    (1, 3, [200, 90], 30, [30, 11], "causal"), (1, 7, [130], 9, None, "none"),
    (1, 16, [77, 500], 5, None, "causal"), (1, 64, [260], 2, None, "causal"),
    (3, 5, [61, 0, 140], 13, [13, 0, 12], "none"),
    # rows that see nothing: fewer slots than rows, and no slot at all
    (1, 4, [3, 0, 1], 8, None, "causal"), (1, 2, [0, 5], 4, None, "none"),
    (1, 1, [150], 100, None, "causal"),
]


@pytest.mark.parametrize("heads,g,lens,block,q_lens,mask", CASES)
def test_attention(heads, g, lens, block, q_lens, mask):
    c, rng = filled(heads, lens, seed=block + g)
    q = rng.normal(size=(len(lens), block, heads * g, HD)) * 1.5
    got, lse, qe = run_attention(c, q, mask, lens, q_lens, pad=3)
    for b, n in enumerate(lens):
        r = block if q_lens is None else q_lens[b]
        check_rows(c, qe, got, lse, mask, n, r, b, b)
        assert (got[b, r:] == 9).all() and (lse[b, r:] == 9).all()  # rows behind: as they were
        if n == 0 or (mask == "causal" and r > n):
            assert (got[b, :max(0, r - n) or r] == 0).all()
    capi().dflash_kvq_check(c.h)
    again, _, _ = run_attention(c, q, mask, lens, q_lens, lse=False)
    np.testing.assert_array_equal(got, again)  # same bits, with or without lse
    plain, l2, _ = run_attention(c, q, mask, lens, q_lens, ws=False)
    for b, n in enumerate(lens):
        check_rows(c, qe, plain, l2, mask, n, block if q_lens is None else q_lens[b], b, b)


@pytest.mark.parametrize("block,words,lens,q_lens", [
    (9, 1, [40, 9, 5], None), (65, 2, [400, 65], [65, 40]), (70, 1, [200], None),
])
def test_attention_tree(block, words, lens, q_lens):
    rng = np.random.default_rng(block)
    parents = [-1] + [int(rng.integers(max(0, i - 6), i)) for i in range(1, block)]
    sets, bits = ancestors(parents, 2)
    bits = bits[:, :words].copy()  # ancestors past the words given are not seen
    sets = [{m for m in s if m < 64 * words} for s in sets]
    c, rng = filled(2, lens, seed=block)
    q = rng.normal(size=(len(lens), block, 8, HD))
    anc = np.broadcast_to(bits, (len(lens), block, words)).copy()
    got, lse, qe = run_attention(c, q, "tree", lens, q_lens, anc)
    for b, n in enumerate(lens):
        check_rows(c, qe, got, lse, "tree", n, block if q_lens is None else q_lens[b], b, b, sets)


def test_attention_long_context_splits():
    """Two KV heads over a long context: many splits; the bound on the keys may
    be too small or too large."""
    lens = [5000, 3, 2200]
    c, rng = filled(2, lens, seed=5)
    q = rng.normal(size=(3, 4, 4, HD)) * 1.5
    for mk in (5000, 1, 1 << 20):
        got, lse, qe = run_attention(c, q, "causal", lens, max_keys=mk)
        for b, n in enumerate(lens):
            check_rows(c, qe, got, lse, "causal", n, 4, b, b)


def test_attention_unseen_places_do_not_enter():
    """NaN in slots a row does not see (later rows' K and V, codes behind the
    last slot) leaves it finite; a row that sees NaN gets NaN where the formula
    does."""
    c, rng = filled(1, [64], seed=9, pages=1)
    new = rng.normal(size=(1, 8, 1, HD))
    kn, vn = new.copy(), new.copy()
    kn[0, 6, 0, 5] = np.nan
    vn[0, 4, 0, 17] = np.inf
    c.append([64], kn, vn)
    q = rng.normal(size=(1, 8, 2, HD))
    got, lse, qe = run_attention(c, q, "causal", [72])
    k, v = np.nan_to_num(c.val["k"][0, :72]), np.nan_to_num(c.val["v"][0, :72])
    ref, rl, mag = ok.attend(qe[0], k, v, ok.visible("causal", 72, 8))
    tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -10) * mag
    dims = np.arange(HD) != 17
    assert (np.abs(got[0, :4] - ref[:4]) <= tol[:4]).all()
    assert (np.abs(got[0, 4:6] - ref[4:6]) <= tol[4:6])[..., dims].all()
    assert np.isnan(got[0, 4:6, :, 17]).all()
    assert np.isnan(got[0, 6:]).all() and np.isnan(lse[0, 6:]).all()
    check_lse(lse[0, :6], rl[:6], qe[0], k)


def test_attention_nan_query_stays_in_its_row():
    c, rng = filled(1, [200], seed=10)
    q = rng.normal(size=(1, 6, 4, HD))
    q[0, 2, 1, 3] = np.nan
    q[0, 5, 0, 0] = np.inf
    got, lse, qe = run_attention(c, q, "none", [200])
    bad = np.zeros((6, 4), dtype=bool)
    bad[2, 1] = bad[5, 0] = True
    assert np.isnan(got[0][bad]).all() and np.isfinite(got[0][~bad]).all()
    ref, _, mag = ok.attend(np.nan_to_num(qe[0], posinf=0), c.val["k"][0], c.val["v"][0],
                            np.broadcast_to(np.arange(256) < 200, (6, 256)))
    assert (np.abs(got[0] - ref)[~bad] <= (2.0 ** -8 * np.abs(ref) + 2.0 ** -7 * mag)[~bad]).all()


def test_attention_value_scales_far_apart():
    """Blocks of V whose exponents differ by tens: a heavy weight on tiny
    values still counts in the normaliser, and the reverse."""
    rng = np.random.default_rng(12)
    n = 300
    k = rng.normal(size=(1, n, 1, HD))
    v = rng.normal(size=(1, n, 1, HD))
    q = rng.normal(size=(1, 1, 1, HD))
    k[0, 0, 0] = q[0, 0, 0] * 3          # the first slot draws most of the weight,
    v[0, :16] *= 2.0 ** -30              # with tiny values
    v[0, 128:144] *= 2.0 ** 30           # and one block is huge
    v[0, 200:216] = 0
    for scale in (1.0, 2.0 ** 5, 2.0 ** -20):
        c = Cache(1, 1, 3)
        c.append([0], k, v * scale)
        got, lse, qe = run_attention(c, q, "none", [n])
        check_rows(c, qe, got, lse, "none", n, 1, 0, 0)


def test_attention_small_weights_add_up():
    """One slot draws nearly half of the weight, 6000 others share the rest in
    weights of about 2^-13 of it: none of them may be rounded away."""
    n = 6000
    k = np.zeros((1, n, 1, HD))
    q = np.zeros((1, 1, 1, HD))
    q[0, 0, 0, 0] = 16.0
    k[0, 77, 0, 0] = 9.0 * np.log(2) * np.sqrt(HD) / 16.0 * 13 / 9
    v = np.ones((1, n, 1, HD))
    v[0, 77] = 0
    c = Cache(1, 1, 47)
    c.append([0], k, v)
    got, lse, qe = run_attention(c, q, "none", [n])
    check_rows(c, qe, got, lse, "none", n, 1, 0, 0)
    assert got[0, 0, 0, 0] > 0.3


def test_attention_unmapped_pages_count_as_unseen():
    c, rng = filled(1, [384], seed=13, pages=4)
    tab = c.h.tensors[4]
    tab[0, 1] = -1
    q = rng.normal(size=(1, 3, 4, HD))
    got, lse, qe = run_attention(c, q, "none", [384])
    vis = np.ones((3, 384), dtype=bool)
    vis[:, 128:256] = False
    check_rows(c, qe, got, lse, "none", 384, 3, 0, 0, ok_mask=vis)
    with pytest.raises(capi().DFlashError) as e:
        capi().dflash_kvq_check(c.h)
    assert e.value.status == 2
    tab[0, 1] = 10 ** 6  # an id past the pool
    again, _, _ = run_attention(c, q, "none", [384])
    np.testing.assert_array_equal(again, got)
    with pytest.raises(capi().DFlashError):
        capi().dflash_kvq_check(c.h)
    # a length past the table
    tab[0, 1] = int(c.table[0, 1])
    run_attention(c, q, "none", [5000])
    with pytest.raises(capi().DFlashError):
        capi().dflash_kvq_check(c.h)
    # bad ids and lengths skip their entry only
    for kw in (dict(seqs=[1]), dict(lens=[-1]), dict(q_lens=[4])):
        a = dict(lens=[100], seqs=None, q_lens=None)
        a.update(kw)
        got, _, _ = run_attention(c, q, "none", a["lens"], a["q_lens"], seqs=a["seqs"])
        assert (got == 9).all()
        with pytest.raises(capi().DFlashError) as e:
            capi().dflash_kvq_check(c.h)
        assert e.value.status == 5


# ---------------------------------------------------------------------------
# accumulated weights
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("heads,g,lens,block,q_lens,mask", CASES)
def test_score(heads, g, lens, block, q_lens, mask):
    c, rng = filled(heads, lens, seed=2 * block + g)
    B, H = len(lens), heads * g
    q = rng.normal(size=(B, block, H, HD)) * 1.5
    t, qe = bf16(np.concatenate([q, q[:, :, :1]], axis=2))
    qe = qe[:, :, :H]
    old = rng.random(size=(B, heads, c.pages * PAGE)).astype(np.float32)
    lse, want = np.full((B, block, H), np.nan), old.astype(np.float64)
    tol = np.zeros_like(want)
    for b, n in enumerate(lens):
        r = block if q_lens is None else q_lens[b]
        vis = ok.visible(mask, n, r)
        k = c.val["k"][b, :n]
        _, l64, _ = ok.attend(qe[b, :r], k, c.val["v"][b, :n], vis)
        lse[b, :r] = l64
        w = ok.score(qe[b, :r], k, vis, np.float32(l64).astype(np.float64))
        want[b, :, :n] = 0.75 * old[b, :, :n] + w
        top = np.abs(qe[b]).max() * (np.abs(k).sum(axis=-1).max() if n else 0) / np.sqrt(HD)
        tol[b, :, :n] = 2.0 ** -22 + 2.0 ** -20 * want[b, :, :n] + (2.0 ** -17 * top + 2.0 ** -20) * w
    lt = torch.from_numpy(lse).float().cuda()
    src = torch.from_numpy(old).cuda()
    out = src.clone()
    code = {"none": 0, "causal": 1}[mask]

    def call(a, z):
        capi().dflash_kvq_score(c.h, B, H, block, code, None, i32(lens), i32(q_lens), None,
                                max(max(lens), 1), t[:, :, :H], lt, 0.75, a, z)
    call(src, out)
    got = out.double().cpu().numpy()
    assert (np.abs(got - want) <= tol).all(), float((np.abs(got - want) - tol).max())
    inplace = src.clone()
    call(inplace, inplace)
    assert torch.equal(inplace, out)
    fresh = torch.zeros_like(src)
    call(None, fresh)
    zero = torch.zeros_like(src)
    call(zero, zero)
    assert torch.equal(fresh, zero)
    capi().dflash_kvq_check(c.h)


def test_score_tree_and_its_sum():
    """Each row's weights sum to one, so a call adds rows * group to a head."""
    block, lens = 33, [300, 150]
    parents = [-1] + [max(0, i - 1 - i % 3) for i in range(1, block)]
    sets, bits = ancestors(parents, 1)
    c, rng = filled(2, lens, seed=21)
    q = rng.normal(size=(2, block, 12, HD))
    anc = np.broadcast_to(bits, (2, block, 1)).copy()
    got, lse, qe = run_attention(c, q, "tree", lens, [33, 20], anc, pad=0)
    t, _ = bf16(q)
    ls = torch.from_numpy(lse).float().cuda()
    out = torch.zeros(2, 2, c.pages * PAGE, device="cuda")
    capi().dflash_kvq_score(c.h, 2, 12, block, 2, None, i32(lens), i32([33, 20]),
                            torch.from_numpy(anc).cuda(), 300, t, ls, 1.0, None, out)
    o = out.double().cpu().numpy()
    for b, (n, r) in enumerate(zip(lens, (33, 20))):
        vis = ok.visible("tree", n, r, sets)
        w = ok.score(qe[b, :r], c.val["k"][b, :n], vis, lse[b, :r])
        assert np.abs(o[b, :, :n] - w).max() <= 2.0 ** -12 * (1 + w.max())
        assert (o[b, :, n:] == 0).all()
        np.testing.assert_allclose(o[b].sum(axis=1), r * 6, rtol=1e-4)


# ---------------------------------------------------------------------------
# eviction
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("heads,lens,budget,window", [
    (2, [300, 100, 0, 129], 128, 16), (1, [1], 1, 0), (3, [700], 333, 0), (1, [513, 40], 40, 40),
    (1, [2000], 1, 1), (2, [1000, 999], 250, 100),
])
def test_evict(heads, lens, budget, window):
    B = len(lens)
    c, rng = filled(heads, lens + [0] * B, seed=budget, v_scale=3.0,
                    pages=max((max(lens + [budget]) + PAGE - 1) // PAGE, 1))
    sc = np.round(rng.random((2 * B, heads, c.pages * PAGE)) * 40).astype(np.float32)  # many ties
    sc[rng.random(sc.shape) < 0.02] = np.nan
    sc[rng.random(sc.shape) < 0.02] = -0.0
    sc[rng.random(sc.shape) < 0.02] = np.inf
    sc[rng.random(sc.shape) < 0.02] = -3.5
    score = torch.from_numpy(sc).cuda()
    src, dst = list(range(B))[::-1], [B + (b + 1) % B for b in range(B)]
    kept = torch.full((B, heads, budget), 99, dtype=torch.int32, device="cuda")
    nl = torch.full((B,), 99, dtype=torch.int32, device="cuda")
    n_of = [lens[s] for s in src]
    before = {x: c.codes(x)[0] for x in "kv"}
    capi().dflash_kvq_evict(c.h, B, i32(src), i32(dst), i32(n_of), max(max(lens), 1), budget, window,
                            score, kept, nl)
    capi().dflash_kvq_check(c.h)
    kept, new = kept.cpu().numpy(), score.cpu().numpy()
    assert nl.tolist() == [min(n, budget) for n in n_of]
    vals = {x: c.values(x) for x in "kv"}
    for b in range(B):
        n, m = n_of[b], min(n_of[b], budget)
        np.testing.assert_array_equal(new[src[b]], sc[src[b]])
        for h in range(heads):
            pick = ok.evict_pick(sc[src[b], h], n, budget, window)
            assert kept[b, h].tolist() == pick + [-1] * (budget - m)
            np.testing.assert_array_equal(new[dst[b], h, :m], sc[src[b], h, pick])
            assert (new[dst[b], h, m:] == 0).all()
            for x in "kv":
                rows = c.val[x][src[b]][pick, h]
                for s in range(0, m, SUB):
                    want, _ = ok.code_block(rows[s:s + SUB])
                    np.testing.assert_array_equal(vals[x][dst[b], s:min(m, s + SUB), h], want)
    for x in "kv":
        after = c.codes(x)[0]
        for b in range(B):
            np.testing.assert_array_equal(after[src[b]], before[x][src[b]])
            m = min(n_of[b], budget)
            np.testing.assert_array_equal(after[dst[b], m:], before[x][dst[b], m:])


def test_evict_reports_bad_entries():
    c, _ = filled(1, [300, 0, 0], seed=2)
    c.h.tensors[4][2, 0] = -1
    score = torch.rand(3, 1, c.pages * PAGE, device="cuda")
    kept = torch.zeros(1, 1, 150, dtype=torch.int32, device="cuda")
    nl = torch.zeros(1, dtype=torch.int32, device="cuda")
    for src, dst, n, status in ((0, 0, 300, 5), (0, 3, 300, 5), (-1, 1, 300, 5), (0, 1, -4, 5),
                                (0, 2, 300, 2), (0, 1, 4000, 2)):
        capi().dflash_kvq_evict(c.h, 1, i32([src]), i32([dst]), i32([n]), 300, 150, 8, score, kept,
                                nl)
        with pytest.raises(capi().DFlashError) as e:
            capi().dflash_kvq_check(c.h)
        assert e.value.status == status


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
def test_generation_with_eviction_captured():
    """Steps as a server runs them (append a block, attend, accumulate), then an
    eviction into fresh pages and attention there; the step is captured into
    two CUDA graphs with a workspace each, replayed on another stream, and gives
    the eager results bit for bit."""
    m = capi()
    heads, g, block, B = 2, 4, 16, 2
    H, n0 = heads * g, [400, 250]
    c, rng = filled(heads, n0 + [0, 0], seed=31, pages=5)
    rows, exact = bf16(rng.normal(size=(B, block, H + 2 * heads, HD)))
    q, k, v = rows[:, :, :H], rows[:, :, H:H + heads], rows[:, :, H + heads:]
    start, lens = i32(n0), i32([x + block for x in n0])
    need = m.dflash_kvq_attention_workspace(B, H, heads, block, 640)

    def buffers():
        return (torch.zeros(B, block, H, HD, dtype=torch.bfloat16, device="cuda"),
                torch.zeros(B, block, H, device="cuda"),
                torch.zeros(4, heads, c.pages * PAGE, device="cuda"),
                torch.empty(max(need, 16), dtype=torch.uint8, device="cuda"))

    def step(o):
        m.dflash_kvq_append(c.h, B, block, None, start, None, k, v)
        m.dflash_kvq_attention(c.h, B, H, block, 1, None, lens, None, None, 640, q, o[0], o[1], o[3])
        m.dflash_kvq_score(c.h, B, H, block, 1, None, lens, None, None, 640, q, o[1], 0.5, None, o[2])
    eager = buffers()
    step(eager)
    torch.cuda.synchronize()
    for b in range(B):
        for x, at in (("k", H), ("v", H + heads)):
            ok.append(c.val[x][b], c.exp[x][b], n0[b], exact[b, :, at:at + heads])
        check_rows(c, exact[:, :, :H], eager[0].double().cpu().numpy(),
                   eager[1].double().cpu().numpy(), "causal", n0[b] + block, block, b, b)
    graphs, outs = [], [buffers(), buffers()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for o in outs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step(o)
        graphs.append(graph)
    for _ in range(3):
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for o in outs:
        for a, z in zip(o[:3], eager[:3]):
            assert torch.equal(a, z)
    # evict both sequences to 128 slots, then attend with new rows there
    kept = torch.zeros(B, heads, 128, dtype=torch.int32, device="cuda")
    nl = torch.zeros(B, dtype=torch.int32, device="cuda")
    with torch.cuda.stream(side):
        m.dflash_kvq_evict(c.h, B, i32([0, 1]), i32([2, 3]), lens, 640, 128, 32, eager[2], kept, nl)
        m.dflash_kvq_append(c.h, B, block, i32([2, 3]), nl, None, k, v)
        m.dflash_kvq_attention(c.h, B, H, block, 1, i32([2, 3]), nl + block, None, None, 640, q,
                               eager[0], eager[1], eager[3])
    side.synchronize()
    m.dflash_kvq_check(c.h)
    assert nl.tolist() == [128, 128]
    vals = {x: c.values(x) for x in "kv"}
    for b in range(B):
        for x in "kv":
            c.val[x][2 + b, :144] = vals[x][2 + b, :144]
            pick = kept[b, 0].cpu().numpy()
            err = np.abs(vals[x][2 + b, :128, 0] - c.val[x][b, pick, 0]).max()
            assert err <= np.abs(c.val[x][b, pick, 0]).max() * 2.0 ** -17
        check_rows(c, exact[:, :, :H], eager[0].double().cpu().numpy(),
                   eager[1].double().cpu().numpy(), "causal", 144, block, b, 2 + b)


def test_offsets_past_32_bits():
    """A pool of more than 4 GiB of codes: pages at its end are addressed right."""
    m = capi()
    heads, n_pages = 8, 36000  # 36000 * 8 * 16 KB = 4.7 GB of K, as much of V
    k8 = torch.zeros(n_pages, heads, PAGE, HD, dtype=torch.uint8, device="cuda")
    v8 = torch.zeros_like(k8)
    ke = torch.zeros(n_pages, heads, PAGE // SUB, dtype=torch.int8, device="cuda")
    tab = i32([[35999, 3, 35000], [35998, 34999, 0]])
    h = m.KvqCache(k8, v8, ke, ke.clone(), tab, torch.zeros(1, dtype=torch.int32, device="cuda"))
    g = torch.Generator(device="cuda").manual_seed(1)
    rows = torch.randn(2, 300, 2 * heads, HD, device="cuda", generator=g).to(torch.bfloat16)
    m.dflash_kvq_append(h, 2, 300, None, i32([0, 0]), None, rows[:, :, :heads], rows[:, :, heads:])
    kb = torch.empty(2, 300, heads, HD, dtype=torch.bfloat16, device="cuda")
    vb = torch.empty_like(kb)
    m.dflash_kvq_read(h, 2, 300, None, None, None, kb, vb)
    for t, x in ((kb, rows[:, :, :heads]), (vb, rows[:, :, heads:])):
        # half a step is 2^-4 of a value, or 2^-10 * 2^e with 448 * 2^e < 16
        err = (t.float() - x.float()).abs()
        assert (err <= x.float().abs() * 2.0 ** -4 + 2.0 ** -14).all()
    q = torch.randn(2, 1, heads, HD, device="cuda", generator=g).to(torch.bfloat16)
    out = torch.empty_like(q)
    m.dflash_kvq_attention(h, 2, heads, 1, 0, None, i32([300, 300]), None, None, 300, q, out)
    s = torch.einsum("bihd,bnhd->bhn", q.double(), kb.double()) / HD ** 0.5
    ref = torch.einsum("bhn,bnhd->bhd", s.softmax(-1), vb.double())
    mag = torch.einsum("bhn,bnhd->bhd", s.softmax(-1), vb.double().abs())
    assert ((out[:, 0].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -7 * mag).all()
    m.dflash_kvq_check(h)


def test_score_many_q_tiles_and_pages():
    """Passes of many q tiles over several groups of pages, and rows that see
    only part of the pages."""
    for heads, g, lens, block, q_lens, mask in ((2, 8, [900, 700, 70], 40, [40, 33, 5], "causal"),
                                                (1, 5, [1300, 640], 300, None, "causal"),
                                                (1, 2, [1100], 130, None, "none")):
        c, rng = filled(heads, lens, seed=block)
        B, H = len(lens), heads * g
        t, qe = bf16(rng.normal(size=(B, block, H, HD)) * 1.5)
        q_lens = q_lens or [block] * B
        k = torch.from_numpy(np.stack([c.val["k"][b] for b in range(B)])).cuda()
        q = torch.from_numpy(qe).cuda().view(B, block, heads, g, HD)
        s = torch.einsum("bjhgd,bnhd->bjhgn", q, k) / HD ** 0.5
        n = torch.tensor(lens).cuda()[:, None, None]
        r = torch.tensor(q_lens).cuda()[:, None, None]
        slot = torch.arange(k.shape[1]).cuda()[None, None]
        row = torch.arange(block).cuda()[None, :, None]
        seen = (slot < n) & (row < r) & ((slot - (n - r) <= row) | (mask == "none"))
        s = s.masked_fill(~seen[:, :, None, None], float("-inf"))
        lse = torch.logsumexp(s, dim=-1)
        p = torch.where(seen[:, :, None, None], torch.exp(s - lse[..., None]), torch.zeros_like(s))
        want = p.sum(dim=(1, 3))
        out = torch.zeros(B, heads, k.shape[1], device="cuda")
        lf = lse.reshape(B, block, H).float()
        capi().dflash_kvq_score(c.h, B, H, block, {"none": 0, "causal": 1}[mask], None, i32(lens),
                                i32(q_lens), None, max(lens), t, lf, 1.0, None, out)
        # a weight is off by its score's error, see test_score; lse in fp32 by 2^-22
        top = np.abs(qe).max() * float(k.abs().sum(-1).max()) / HD ** 0.5
        tol = 2.0 ** -22 + (2.0 ** -17 * top + 2.0 ** -18) * want
        assert ((out.double() - want).abs() <= tol).all()
        capi().dflash_kvq_check(c.h)


def test_evict_recodes_rows_of_far_exponents_and_nan():
    """Kept rows whose source blocks differ by up to 60 binades land in one
    block; NaN codes stay NaN and do not count for the exponent."""
    n, budget = 256, 64
    c = Cache(1, 2, 2, seed=7)
    rng = np.random.default_rng(7)
    x = rng.normal(size=(1, n, 1, HD)) * 2.0 ** np.repeat(rng.integers(-30, 31, n // SUB), SUB)[:, None, None]
    near = rng.normal(size=(1, n, 1, HD)) * 2.0 ** np.repeat(rng.integers(-7, 8, n // SUB), SUB)[:, None, None]
    near[0, 40, 0, 3], near[0, 100, 0, 9] = np.nan, np.inf
    c.append([0], x, near, seqs=[0])
    score = torch.from_numpy(rng.random((2, 1, n)).astype(np.float32)).cuda()
    score[0, 0, [40, 100]] = 2.0
    kept = torch.zeros(1, 1, budget, dtype=torch.int32, device="cuda")
    nl = torch.zeros(1, dtype=torch.int32, device="cuda")
    capi().dflash_kvq_evict(c.h, 1, i32([0]), i32([1]), i32([n]), n, budget, 8, score, kept, nl)
    capi().dflash_kvq_check(c.h)
    pick = kept[0, 0].tolist()
    assert 40 in pick and 100 in pick
    for x in "kv":
        got = c.values(x)[1, :budget, 0]
        rows = c.val[x][0][pick, 0]
        for s in range(0, budget, SUB):
            np.testing.assert_array_equal(got[s:s + SUB], ok.code_block(rows[s:s + SUB])[0])


@pytest.mark.parametrize("n,kind", [(40000, "random"), (9000, "zeros"), (100000, "ties")])
def test_evict_long_lists(n, kind):
    """Lists longer than a cluster holds in shared memory, and all-equal scores."""
    budget, window, pages = 3000, 100, (n + PAGE - 1) // PAGE
    c = Cache(1, 2, pages, spare=0)
    g = torch.Generator(device="cuda").manual_seed(n)
    score = torch.rand(2, 1, pages * PAGE, device="cuda", generator=g)
    if kind == "zeros":
        score.zero_()
    elif kind == "ties":
        score = torch.round(score * 8) / 8
    kept = torch.zeros(1, 1, budget, dtype=torch.int32, device="cuda")
    nl = torch.zeros(1, dtype=torch.int32, device="cuda")
    src = score[0, 0].clone()
    for mk in (n, 1):  # a cluster of eight, and one CTA
        kept.zero_()
        capi().dflash_kvq_evict(c.h, 1, i32([0]), i32([1]), i32([n]), mk, budget, window, score, kept, nl)
        key = src[:n - window].double().cpu().numpy()
        best = np.lexsort((np.arange(n - window), -key))[:budget - window]
        want = np.sort(np.concatenate([best, np.arange(n - window, n)]))
        np.testing.assert_array_equal(kept[0, 0].cpu().numpy(), want)
        assert torch.equal(score[1, 0, :budget], src[torch.from_numpy(want).cuda()])
        assert (score[1, 0, budget:] == 0).all()


def test_evict_into_another_entry_s_source_stays_in_bounds():
    """Scores that change while they are searched leave the choice open, not where it
    is written: nothing beside the lists changes, and no slot is out of range."""
    n, budget, window = 20000, 3000, 100
    c = Cache(1, 3, (n + PAGE - 1) // PAGE, spare=0)
    g = torch.Generator(device="cuda").manual_seed(5)
    score = torch.rand(3, 1, c.pages * PAGE, device="cuda", generator=g)
    room = torch.full((4, 1, budget), -7, dtype=torch.int32, device="cuda")
    nl = torch.zeros(2, dtype=torch.int32, device="cuda")
    for mk in (n, 1):
        room[1:3] = 0
        capi().dflash_kvq_evict(c.h, 2, i32([0, 1]), i32([1, 2]), i32([n, n]), mk, budget, window,
                                score, room[1:3], nl)
        assert (room[0] == -7).all() and (room[3] == -7).all()
        assert (room[1:3] >= 0).all() and (room[1:3] < n).all()
        assert nl.tolist() == [budget, budget]
    capi().dflash_kvq_check(c.h)


@pytest.mark.parametrize("mask", ["none", "causal"])
def test_score_rows_with_lse_minus_infinity_add_nothing(mask):
    """Not where the row itself or K holds a NaN either: sequence 0 has one such row, of
    NaN; all of sequence 1's are, and its K holds a NaN in slot 3."""
    lens, block, heads, g = [300, 140], 6, 2, 3
    c, rng = filled(heads, lens, seed=9)
    k = c.val["k"][1:2, :4].copy()
    k[0, 3, :, 5] = np.nan
    c.append([0], k, c.val["v"][1:2, :4], seqs=[1], oracle=False)
    # (appending restarts the block of 16: its later slots are junk now, NaN among it)
    q = rng.normal(size=(2, block, heads * g, HD))
    t, qe = bf16(q)
    lse = np.full((2, block, heads * g), -np.inf)
    vis = ok.visible(mask, 300, block)
    lse[0] = ok.attend(qe[0], c.val["k"][0, :300], c.val["v"][0, :300], vis)[1]
    lse[0, 2] = -np.inf
    t[0, 2] = float("nan")
    old = torch.from_numpy(rng.random(size=(2, heads, c.pages * PAGE))).float().cuda()
    out = torch.zeros_like(old)
    capi().dflash_kvq_score(c.h, 2, heads * g, block, {"none": 0, "causal": 1}[mask], None, i32(lens),
                            None, None, 300, t, torch.from_numpy(lse).float().cuda(), 0.5, old, out)
    assert torch.equal(out[1, :, :140], 0.5 * old[1, :, :140])
    w = ok.score(qe[0], c.val["k"][0, :300], vis, np.float32(lse[0]).astype(np.float64))
    top = np.abs(qe[0]).max() * np.abs(c.val["k"][0, :300]).sum(axis=-1).max() / np.sqrt(HD)
    want = 0.5 * old[0, :, :300].double().cpu().numpy() + w
    tol = 2.0 ** -22 + 2.0 ** -20 * want + (2.0 ** -17 * top + 2.0 ** -20) * w
    assert (np.abs(out[0, :, :300].double().cpu().numpy() - want) <= tol).all()
    capi().dflash_kvq_check(c.h)
