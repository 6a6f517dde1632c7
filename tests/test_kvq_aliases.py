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


def test_workspace_has_to_be_contiguous(monkeypatch):
    """A strided or expanded view is refused before the library sees its address."""
    calls = []

    class Lib:
        def dflash_kvq_attention(self, *args):
            calls.append(args)
            return 0
    monkeypatch.setattr(capi, "load", Lib)
    k8 = torch.zeros(4, 2, 128, 128, dtype=torch.uint8)
    e = torch.zeros(4, 2, 8, dtype=torch.int8)
    c = capi.KvqCache(k8, k8.clone(), e, e.clone(), torch.zeros(1, 4, dtype=torch.int32),
                      torch.zeros(1, dtype=torch.int32))
    q = torch.zeros(1, 3, 4, 128, dtype=torch.bfloat16)
    lens = torch.zeros(1, dtype=torch.int32)

    def run(ws):
        capi.dflash_kvq_attention(c, 1, 4, 3, 0, None, lens, None, None, 500, q, q.clone(), None, ws, stream=0)
    room = torch.zeros(1 << 16)
    for bad in (room[::2], room[:1].expand(1 << 20), room.view(256, 256)[:, :128], room.view(256, 256).t()):
        with pytest.raises(capi.DFlashError, match="workspace"):
            run(bad)
    assert not calls
    for good in (room, room[64:], room.view(256, 256)[:16], torch.zeros(0)):
        run(good)
        assert calls[-1][-2] == good.numel() * 4
