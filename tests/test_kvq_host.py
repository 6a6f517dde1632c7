"""The 8-bit KV cache without a GPU: the oracle's block format against torch's
e4m3 casts, and the refusals of the dflash_kvq_* calls (made before any device
call, so made-up addresses do)."""
import ctypes

import numpy as np
import pytest
import torch

from block_diffusion_speculative_injection_gb300 import capi
from oracle import kvq as ok


def test_oracle_codes_match_torch():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(codes, ok.E4M3)
    rng = np.random.default_rng(0)
    y = np.concatenate([rng.normal(size=4000) * 2.0 ** rng.integers(-12, 8, 4000),
                        (np.arange(-900, 900) * 2.0 ** -11)]).astype(np.float32)
    y = np.clip(y, -448, 448)
    t = torch.from_numpy(y).to(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(t, ok.round_e4m3(y.astype(np.float64)))


@pytest.mark.parametrize("x,e", [(0.0, -40), (448.0, 0), (448.1, 1), (1.75, -8), (1.7501, -7),
                                 (1e38, 40), (2.0 ** -60, -40), (np.nan, -40), (np.inf, -40)])
def test_oracle_exponent(x, e):
    assert ok.exponent([0.0, x]) == e


def test_oracle_append_growth_is_lossless_in_the_normal_codes():
    v, e = np.zeros((16, 1, 128)), np.zeros((1, 1), dtype=int)
    rng = np.random.default_rng(1)
    ok.append(v, e, 0, rng.uniform(1, 2, size=(4, 1, 128)))
    held, e0 = v[:4].copy(), int(e[0, 0])
    ok.append(v, e, 4, rng.uniform(16, 31, size=(2, 1, 128)))
    assert int(e[0, 0]) == e0 + 4
    np.testing.assert_array_equal(v[:4], held)


def test_oracle_evict_pick():
    s = [5.0, 1.0, np.nan, 5.0, 0.0, -0.0, 9.0, 2.0]
    assert ok.evict_pick(s, 8, 4, 1) == [0, 3, 6, 7]
    assert ok.evict_pick(s, 8, 7, 1) == [0, 1, 3, 4, 5, 6, 7]  # NaN goes first
    assert ok.evict_pick(s, 6, 4, 0) == [0, 1, 3, 4]           # -0 ties with 0, lowest slot
    assert ok.evict_pick(s, 3, 4, 2) == [0, 1, 2]


# ---------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------
A = 1 << 20  # an aligned address that nothing reads


@pytest.fixture(scope="module")
def lib():
    try:
        return capi.load()
    except FileNotFoundError:
        pytest.skip("libdflash.so not built (run __graft_entry__.build())")


def cache(**kw):
    f = dict(k8=A, v8=A, k_exp=A, v_exp=A, page_table=A, status=A, n_pages=10, n_kv_heads=2,
             n_seqs=3, pages_per_seq=4)
    f.update(kw)
    return capi._KvqCacheStruct(*[f[n] for n, _ in capi._KvqCacheStruct._fields_])


def calls(lib, c, **kw):
    """(name, status) of every call with its arguments changed by kw where it
    has them."""
    r = ctypes.byref(c) if c is not None else None
    d = dict(batch=2, rows=3, H=8, block=4, mask=0, ids=None, lens=A, cnt=None, anc=None, words=0,
             mk=500, q=A, qs=8 * 128, out=A, lse=A, ws=None, wb=0, k=A, v=A, ks=256, vs=256,
             start=A, ko=A, vo=A, si=None, so=A, src=A, dst=A, budget=64, window=8, kept=A, nl=A)
    used = set(kw)
    d.update(kw)
    all_ = {
        "append": (("batch", "rows", "start", "k", "v", "ks", "vs"),
                   lambda: lib.dflash_kvq_append(r, d["batch"], d["rows"], d["ids"], d["start"],
                                                 d["cnt"], d["k"], d["v"], d["ks"], d["vs"], None)),
        "read": (("batch", "rows", "ko", "vo"),
                 lambda: lib.dflash_kvq_read(r, d["batch"], d["rows"], d["ids"], d["start"],
                                             d["cnt"], d["ko"], d["vo"], None)),
        "attention": (("batch", "H", "block", "mask", "lens", "anc", "words", "mk", "q", "qs", "out",
                       "lse", "ws", "wb"),
                      lambda: lib.dflash_kvq_attention(r, d["batch"], d["H"], d["block"], d["mask"],
                                                       d["ids"], d["lens"], d["cnt"], d["anc"],
                                                       d["words"], d["mk"], d["q"], d["qs"], d["out"],
                                                       d["lse"], d["ws"], d["wb"], None)),
        "score": (("batch", "H", "block", "mask", "lens", "anc", "words", "mk", "q", "qs", "lse", "si",
                   "so"),
                  lambda: lib.dflash_kvq_score(r, d["batch"], d["H"], d["block"], d["mask"], d["ids"],
                                               d["lens"], d["cnt"], d["anc"], d["words"], d["mk"],
                                               d["q"], d["qs"], d["lse"], 1.0, d["si"], d["so"],
                                               None)),
        "evict": (("batch", "src", "dst", "lens", "mk", "budget", "window", "so", "kept", "nl"),
                  lambda: lib.dflash_kvq_evict(r, d["batch"], d["src"], d["dst"], d["lens"], d["mk"],
                                               d["budget"], d["window"], d["so"], d["kept"], d["nl"],
                                               None)),
        "check": ((), lambda: lib.dflash_kvq_check(r, None)),
    }
    return [(n, f()) for n, (args, f) in all_.items() if not used or used & set(args)]


@pytest.mark.parametrize("field,value", [
    ("k8", None), ("v8", None), ("k_exp", None), ("v_exp", None), ("page_table", None),
    ("status", None), ("k8", A + 8), ("v8", A + 4), ("k_exp", A + 4), ("v_exp", A + 1),
    ("page_table", A + 2), ("status", A + 2), ("n_pages", 0), ("n_pages", 1 << 23),
    ("n_kv_heads", 0), ("n_seqs", 0), ("pages_per_seq", 0), ("pages_per_seq", (1 << 22) + 1),
])
def test_bad_caches_are_refused(lib, field, value):
    for name, st in calls(lib, cache(**{field: value})):
        assert st == 1, name


def test_null_cache_is_refused(lib):
    for name, st in calls(lib, None):
        assert st == 1, name


@pytest.mark.parametrize("kw", [
    {"batch": 0}, {"batch": -1}, {"rows": 0}, {"start": None, "k": None}, {"k": None}, {"v": None},
    {"k": A + 8}, {"v": A + 2}, {"ks": 255}, {"ks": 128}, {"vs": 260}, {"vs": 1 << 31},
    {"ko": None, "vo": None}, {"ko": A + 8}, {"vo": A + 4},
    {"H": 7}, {"H": 0}, {"H": 130}, {"block": 0}, {"mask": 3}, {"mask": -1}, {"mask": 2},
    {"mask": 2, "anc": A, "words": 0}, {"mask": 2, "anc": A + 4, "words": 1}, {"lens": None},
    {"mk": 0}, {"mk": (1 << 29) + 1}, {"q": None}, {"q": A + 8}, {"qs": 1023}, {"qs": 512},
    {"qs": 1028}, {"out": None}, {"out": A + 8}, {"ws": A + 8, "wb": 4096}, {"wb": -1},
    {"so": None}, {"src": None}, {"dst": None}, {"budget": 0}, {"budget": 513},
    {"window": -1}, {"window": 65}, {"kept": None}, {"nl": None},
    {"batch": 65536, "block": 65536, "rows": 1 << 29},
])
def test_bad_arguments_are_refused(lib, kw):
    hit = calls(lib, cache(), **kw)
    assert hit
    for name, st in hit:
        if name == "read" and set(kw) & {"start"}:
            continue
        assert st == 1, name


def test_workspace_of_bad_sizes(lib):
    for a in ((0, 8, 2, 4, 100), (1, 7, 2, 4, 100), (1, 130, 2, 4, 100), (1, 8, 2, 0, 100),
              (1, 8, 2, 4, 0), (1, 8, 0, 4, 100)):
        assert capi.dflash_kvq_attention_workspace(*a) == -1


def test_wrappers_check_tensors():
    k8 = torch.zeros(4, 2, 128, 128, dtype=torch.uint8)
    e = torch.zeros(4, 2, 8, dtype=torch.int8)
    tab, st = torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    c = capi.KvqCache(k8, k8.clone(), e, e.clone(), tab, st)
    assert c.slots == 512
    for bad in ((k8[:, :1], k8, e, e, tab, st), (k8, k8.float(), e, e, tab, st),
                (k8, k8, e[:3], e, tab, st), (k8, k8, e, e, tab.long(), st),
                (k8, k8, e, e, tab, st.float())):
        with pytest.raises(capi.DFlashError):
            capi.KvqCache(*bad)
    x = torch.zeros(2, 3, 6, 128, dtype=torch.bfloat16)
    assert capi._kvq_rows(x[:, :, 2:4], "k", 2, 3, 2) == 768
    assert capi._kvq_rows(x[:, :1, 2:4], "k", 2, 1, 2) == 3 * 768
    for bad in (x[:, :, 2:4].float(), x[:, :2, :2], x[:, :, ::3], x[..., :2, :64]):
        with pytest.raises(capi.DFlashError):
            capi._kvq_rows(bad, "k", 2, bad.shape[1], 2)


@pytest.mark.parametrize("name,kw", [
    ("append", {"start": A + 2}), ("append", {"k": A, "cnt": A + 1}), ("append", {"k": A, "ids": A + 2}),
    ("read", {"ko": A, "start": A + 2}), ("read", {"ko": A, "cnt": A + 3}), ("read", {"ko": A, "ids": A + 1}),
    ("attention", {"lens": A + 2}), ("attention", {"q": A, "cnt": A + 2}), ("attention", {"q": A, "ids": A + 2}),
    ("score", {"lens": A + 1}), ("score", {"q": A, "cnt": A + 1}), ("score", {"q": A, "ids": A + 1}),
    ("evict", {"src": A + 2}), ("evict", {"dst": A + 2}), ("evict", {"lens": A + 2}),
    ("evict", {"kept": A + 2}), ("evict", {"nl": A + 2}),
])
def test_misaligned_integer_arrays_are_refused(lib, name, kw):
    assert dict(calls(lib, cache(), **kw))[name] == 1


def test_workspace_of_the_longest_blocks(lib):
    """Far more CTAs than SMs: nothing is gained by splitting."""
    for block in (2 ** 31 - 1, 2 ** 31 - 64):
        assert capi.dflash_kvq_attention_workspace(1, 1, 1, block, 4096) == 0
