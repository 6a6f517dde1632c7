"""Calls of the 8-bit KV cache whose arrays overlap, without a GPU: the refusals
are made before any device call, so made-up addresses do."""
import ctypes

import pytest
import torch

from block_diffusion_speculative_injection_gb300 import capi

A = 1 << 20
SRC, DST, LENS, KEPT, NEW, SCORE, TABLE = (A + (i << 16) for i in range(1, 8))
POOL = 1 << 40


@pytest.fixture(scope="module")
def lib():
    try:
        return capi.load()
    except FileNotFoundError:
        pytest.skip("libdflash.so not built (run __graft_entry__.build())")


def evict(lib, n_seqs=3, **kw):
    """Status of an eviction: 3 sequences of 4 pages, 2 heads, a batch of 2, 64 of 512 slots."""
    c = capi._KvqCacheStruct(POOL, POOL, POOL, POOL, TABLE, POOL, 10, 2, n_seqs, 4)
    a = dict(src=SRC, dst=DST, lens=LENS, score=SCORE, kept=KEPT, new=NEW)
    a.update(kw)
    return lib.dflash_kvq_evict(ctypes.byref(c), 2, a["src"], a["dst"], a["lens"], 500, 64, 8, a["score"],
                                a["kept"], a["new"], None)


def goes_on(status):
    """Past the checks that need no device: there the pool's made-up address is refused as no
    device memory, or no device is found; a refusal before that is status 1."""
    return status != 1 or torch.cuda.is_available()


def test_distinct_arrays_and_lengths_in_place_pass(lib):
    assert goes_on(evict(lib))
    assert goes_on(evict(lib, new=LENS))
    assert goes_on(evict(lib, src=LENS))                    # two inputs may be one array
    assert goes_on(evict(lib, kept=NEW + 8, score=NEW + 8 + 2 * 2 * 64 * 4))  # side by side


@pytest.mark.parametrize("kw", [
    {"new": SRC}, {"new": DST}, {"new": LENS + 4}, {"new": LENS - 4}, {"new": TABLE + 40},
    {"new": LENS, "src": LENS}, {"new": LENS, "dst": LENS + 4},
    {"kept": LENS}, {"kept": LENS - 2 * 2 * 64 * 4 + 4}, {"kept": SRC + 4}, {"kept": DST}, {"kept": NEW},
    {"kept": NEW - 4}, {"kept": TABLE}, {"score": KEPT + 1020}, {"score": NEW}, {"score": LENS},
    {"score": SRC - 4 * (3 * 2 * 512 - 1)}, {"score": TABLE + 44}, {"n_seqs": 2 ** 31 - 1, "score": SRC - 4},
])
def test_evict_refuses_overlaps(lib, kw):
    assert evict(lib, **kw) == 1
