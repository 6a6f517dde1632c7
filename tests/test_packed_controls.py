"""Controls of the refusals in test_packed_host: the arguments those tests change one of pass all
checks unchanged.  Without a GPU the next thing a call asks for is the device (DFLASH_E_CUDA), so there
a refusal (DFLASH_E_INVALID_ARG) is the changed argument's doing; with one the made-up addresses
would be refused as well."""
import ctypes

import pytest
import torch

from block_diffusion_speculative_injection_gb300 import capi
from test_kvq_host import cache
from test_packed_host import A, attention, lib, page_calls, pages_struct  # noqa: F401  (lib: a fixture)

CUDA = 4

needs_no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses are refused where there is a GPU")


@needs_no_gpu
@pytest.mark.parametrize("kw", [
    {}, {"lse": None}, {"causal": 0}, {"batch": (1 << 26) - 1}, {"H": 128, "qs": 128 * 128}, {"H": 2}, {"qs": 1032},
    {"rows": 100000},
])
def test_attention(lib, kw):  # noqa: F811
    assert attention(lib, **kw) == CUDA


@needs_no_gpu
@pytest.mark.parametrize("kw", [
    {}, {"batch": 4096}, {"ids": None}, {"start": None}, {"rs": None}, {"rp": None}, {"rl": None}, {"n_rows": 0},
])
def test_pages(lib, kw):  # noqa: F811
    assert set(page_calls(lib, pages_struct(), **kw)) == {CUDA}


@needs_no_gpu
@pytest.mark.parametrize("heads,kw", [(2, {}), (2, {"ids": A}), (2, {"batch": (1 << 26) - 1}),
                                      (2, {"rows": 1 << 20, "ks": 264, "vs": (1 << 31) - 8}), (16, {"ks": 2048, "vs": 2048})])
def test_packed_append(lib, heads, kw):  # noqa: F811
    d = dict(batch=2, rows=10, ids=None, start=A, off=A, k=A, v=A, ks=256, vs=256)
    d.update(kw)
    assert lib.dflash_kvq_append_packed(ctypes.byref(cache(n_kv_heads=heads)), *d.values(), None) == CUDA


@needs_no_gpu
@pytest.mark.parametrize("kw", [
    {}, {"dtype": 1}, {"top": 32}, {"top": 0, "ids": None, "best": None}, {"lp": None, "tokens": None}, {"en": None},
    {"stride": 101}, {"dtype": 1, "x": A + 2}, {"rows": 1},
])
def test_logprobs(lib, kw):  # noqa: F811
    d = dict(rows=3, vocab=100, dtype=0, x=A, stride=100, tokens=2 * A, top=4, lp=3 * A, en=4 * A, ids=5 * A,
             best=6 * A)
    d.update(kw)
    assert lib.dflash_token_logprobs(*d.values(), None) == CUDA


@needs_no_gpu
def test_status_check(lib):  # noqa: F811
    assert lib.dflash_status_check(A, None) == CUDA
