"""The calls over packed batches without a GPU: their refusals (made before any device call, so
made-up addresses do), the wrappers' checks of tensors, and the oracle's page lists."""
import ctypes

import pytest
import torch

from block_diffusion_speculative_injection_gb300 import capi
from oracle import packed as op
from test_kvq_host import cache

A = 1 << 20  # an aligned address that nothing reads
FAR = 1 << 40


@pytest.fixture(scope="module")
def lib():
    try:
        return capi.load()
    except FileNotFoundError:
        pytest.skip("libdflash.so not built (run __graft_entry__.build())")


def attention(lib, **kw):
    d = dict(batch=2, rows=100, H=8, hkv=2, causal=1, off=A, q=FAR, qs=1024, k=2 * FAR, ks=256, v=3 * FAR, vs=256,
             out=4 * FAR, lse=5 * FAR, status=A + 4096)
    assert set(kw) <= set(d)
    d.update(kw)
    return lib.dflash_prompt_attention(*d.values(), None)


@pytest.mark.parametrize("kw", [
    {"batch": 0}, {"batch": -1}, {"batch": 1 << 26}, {"rows": 0}, {"rows": 1 << 30}, {"H": 0}, {"H": 7},
    {"H": 65536, "hkv": 1024, "qs": 1 << 23, "ks": 1 << 17, "vs": 1 << 17}, {"H": 130, "qs": 130 * 128},
    {"hkv": 0}, {"causal": 2}, {"causal": -1}, {"off": None}, {"q": None}, {"k": None}, {"v": None},
    {"out": None}, {"status": None}, {"qs": 1016}, {"qs": 1028}, {"ks": 248}, {"vs": 255}, {"ks": 1 << 31},
    {"q": FAR + 8}, {"k": FAR + 2}, {"v": FAR + 4}, {"out": FAR + 8}, {"lse": FAR + 2}, {"off": A + 2},
    {"status": A + 1},
    # outputs over inputs, or over each other
    {"out": FAR}, {"out": FAR + 1024}, {"out": 2 * FAR - 16}, {"out": 3 * FAR + 512}, {"lse": FAR + 2048},
    {"lse": 4 * FAR + 1024}, {"out": A}, {"lse": A + 4096}, {"lse": A + 4},
    {"rows": (1 << 30) - 1, "H": 64, "hkv": 1, "qs": 64 * 128},
])
def test_attention_refuses(lib, kw):
    assert attention(lib, **kw) == 1


def pages_struct(**kw):
    f = dict(page_table=A, n_mapped=2 * A, free_pages=3 * A, n_free=4 * A, status=5 * A, n_pages=10, n_seqs=3,
             pages_per_seq=4)
    f.update(kw)
    return capi._PagesStruct(*[f[n] for n, _ in capi._PagesStruct._fields_])


def page_calls(lib, p, **kw):
    d = dict(batch=2, n_rows=50, ids=6 * A, start=7 * A, counts=8 * A, off=9 * A, lens=10 * A, rs=11 * A, rp=12 * A,
             rl=13 * A)
    rel = {"batch", "ids", "start"}
    assert set(kw) <= set(d)
    d.update(kw)
    r = ctypes.byref(p) if p is not None else None
    out = [lib.dflash_pages_map(r, *d.values(), None)]
    if not kw or set(kw) <= rel:
        out.append(lib.dflash_pages_release(r, d["batch"], d["ids"], d["start"], None))
    return out


@pytest.mark.parametrize("field,value", [
    ("page_table", None), ("n_mapped", None), ("free_pages", None), ("n_free", None), ("status", None),
    ("page_table", A + 2), ("n_mapped", A + 1), ("free_pages", A + 2), ("n_free", A + 3), ("status", A + 2),
    ("n_pages", 0), ("n_pages", 1 << 24), ("n_seqs", 0), ("pages_per_seq", 0), ("pages_per_seq", (1 << 22) + 1),
    ("n_mapped", A + 40), ("free_pages", 2 * A + 8), ("n_free", A), ("status", 4 * A),
])
def test_bad_pages_are_refused(lib, field, value):
    assert page_calls(lib, pages_struct(**{field: value})) == [1, 1]


@pytest.mark.parametrize("kw", [
    {"batch": 0}, {"batch": 4097}, {"ids": A + 2}, {"start": 7 * A + 1}, {"ids": A}, {"start": 2 * A + 4},
    {"n_rows": -1}, {"n_rows": 1 << 30}, {"counts": None}, {"off": None}, {"lens": None}, {"counts": A + 2},
    {"off": A + 2}, {"lens": A + 2}, {"rs": A + 1}, {"rp": A + 2}, {"rl": A + 3},
    {"lens": 7 * A}, {"lens": 8 * A}, {"off": 6 * A}, {"off": 10 * A - 8}, {"rs": 12 * A - 4}, {"rl": A + 16},
    {"rp": 3 * A}, {"lens": 5 * A}, {"counts": 4 * A},
])
def test_bad_mappings_are_refused(lib, kw):
    assert set(page_calls(lib, pages_struct(), **kw)) == {1}


def test_null_pages_are_refused(lib):
    assert page_calls(lib, None) == [1, 1]


@pytest.mark.parametrize("kw", [
    {"batch": 0}, {"rows": 0}, {"rows": 1 << 30}, {"batch": 1 << 26}, {"start": None}, {"off": None}, {"k": None},
    {"v": None}, {"k": A + 8}, {"v": A + 2}, {"ks": 255}, {"ks": 128}, {"vs": 260}, {"vs": 1 << 31}, {"ids": A + 2},
    {"start": A + 2}, {"off": A + 1}, {"rows": (1 << 30) - 1, "batch": (1 << 26) - 1},
])
def test_packed_append_refuses(lib, kw):
    d = dict(batch=2, rows=10, ids=None, start=A, off=A, k=A, v=A, ks=256, vs=256)
    d.update(kw)
    c = cache(n_kv_heads=2 if "batch" not in kw or "rows" not in kw else 16)
    if c.n_kv_heads == 16:
        d.update(ks=2048, vs=2048)
    assert lib.dflash_kvq_append_packed(ctypes.byref(c), *d.values(), None) == 1
    assert lib.dflash_kvq_append_packed(None, *d.values(), None) == 1


@pytest.mark.parametrize("kw", [
    {"rows": 0}, {"rows": 1 << 27}, {"vocab": 0}, {"vocab": 1 << 30, "stride": 1 << 30}, {"dtype": 2}, {"dtype": -1},
    {"x": None}, {"stride": 99}, {"stride": 1 << 40}, {"top": -1}, {"top": 33}, {"tokens": None},
    {"ids": None}, {"best": None}, {"lp": None, "en": None, "top": 0}, {"x": A + 2}, {"dtype": 1, "x": A + 1},
    {"lp": 3 * A + 2}, {"en": 4 * A + 1}, {"best": 6 * A + 2}, {"tokens": 2 * A + 2}, {"ids": 5 * A + 3},
    {"rows": 1 << 20, "stride": 1 << 39, "vocab": 100, "x": FAR},
    # outputs over inputs, or over each other
    {"lp": A}, {"lp": A + 1196}, {"en": A - 8}, {"ids": A + 400}, {"best": A - 44}, {"lp": 2 * A}, {"ids": 2 * A + 8},
    {"lp": 4 * A + 8}, {"ids": 6 * A}, {"best": 3 * A - 40},
])
def test_logprobs_refuse(lib, kw):
    d = dict(rows=3, vocab=100, dtype=0, x=A, stride=100, tokens=2 * A, top=4, lp=3 * A, en=4 * A, ids=5 * A,
             best=6 * A)
    d.update(kw)
    assert lib.dflash_token_logprobs(*d.values(), None) == 1


def test_status_check_refuses(lib):
    assert lib.dflash_status_check(None, None) == 1
    assert lib.dflash_status_check(A + 2, None) == 1


def test_wrappers_check_tensors():
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    p = capi.Pages.empty(6, 2, 3, device="cpu")
    assert p.tensors[2].tolist() == [5, 4, 3, 2, 1, 0] and int(p.tensors[3]) == 6
    for bad in ((i32(2, 3), i32(3), i32(6), i32(1), i32(1)), (i32(6), i32(2), i32(6), i32(1), i32(1)),
                (i32(2, 3).long(), i32(2), i32(6), i32(1), i32(1)), (i32(2, 3), i32(2), i32(6), i32(2), i32(1)),
                (i32(2, 6)[:, ::2], i32(2), i32(6), i32(1), i32(1))):
        with pytest.raises(capi.DFlashError):
            capi.Pages(*bad)
    x = torch.zeros(5, 6, 128, dtype=torch.bfloat16)
    assert capi._packed_rows(x[:, 2:4], "k", 5, 2) == 768
    for bad in (x[:, 2:4].float(), x[:4, :2], x[:, ::3], x[:, :2, :64], x[0]):
        with pytest.raises(capi.DFlashError):
            capi._packed_rows(bad, "k", 5, 2)
    logits = torch.zeros(3, 8)
    for bad in (logits.double(), logits.T, logits[0], logits[:, ::2]):
        with pytest.raises(capi.DFlashError):
            capi.dflash_token_logprobs(bad, i32(bad.shape[0]), 0, torch.zeros(bad.shape[0]))
    with pytest.raises(capi.DFlashError):
        capi.dflash_token_logprobs(logits, i32(3), 2, torch.zeros(3), None, i32(3, 1), torch.zeros(3, 2))


def test_oracle_pages():
    p = op.Pages(5, 3, 3)
    off, lens, rows, wrong = p.map([1, 0], [0, 0], [130, 1], 131)
    assert (off, lens, wrong) == ([0, 130, 131], [130, 1], set())
    assert p.table == [[2, -1, -1], [0, 1, -1], [-1, -1, -1]] and p.free == [4, 3]
    assert rows[0] == (1, 0, 0) and rows[129] == (1, 129, 129) and rows[130] == (0, 0, 256)
    assert p.release([1], [1]) == set() and p.free == [4, 3, 1]
    assert p.map([1], [1], [200], 200)[1] == [201] and p.table[1] == [0, 1, -1]
    assert p.map([2, 0, 1], [0, 1, 201], [380, 1, 1], 382)[1] == [0, 2, 202]  # three pages of two
    assert p.map([2, 2], [0, 0], [1, 1], 2)[3] == {"check"}
