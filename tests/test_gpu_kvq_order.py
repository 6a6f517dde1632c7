"""Passes whose warps run ahead of one another as far as the barriers let them."""
import numpy as np
import pytest
import torch

from kvq_util import HD, Cache, bf16
from test_gpu_kvq import capi, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("block,g,n", [(2, 64, 130), (5, 33, 90), (65, 4, 700), (130, 1, 200), (33, 2, 128)])
@pytest.mark.parametrize("mask", ["none", "causal"])
def test_score_of_several_q_tiles_repeats(block, g, n, mask):
    """The first q tiles are converted one after another while the tensor cores' warp may not have
    started: every one of many launches at once finishes and gives the same bits."""
    B, heads = 24, 8
    c = Cache(heads, B, (n + 127) // 128, seed=1)
    rng = np.random.default_rng(block)
    rows = rng.normal(size=(1, n, heads, HD))
    for b in range(B):
        c.append([0], rows, rows, seqs=[b], oracle=False)
    t, _ = bf16(rng.normal(size=(1, block, heads * g, HD)))
    t = t.expand(B, -1, -1, -1).contiguous()
    lse = torch.full((B, block, heads * g), 7.0, device="cuda")
    code = {"none": 0, "causal": 1}[mask]
    outs = [torch.zeros(B, heads, c.pages * 128, device="cuda") for _ in range(20)]
    for o in outs:
        capi().dflash_kvq_score(c.h, B, heads * g, block, code, None, i32([n] * B), None, None, n, t, lse,
                                1.0, None, o)
    capi().dflash_kvq_check(c.h)
    assert (outs[0][:, :, :n] > 0).all() and (outs[0][:, :, n:] == 0).all()
    assert torch.equal(outs[0][1:], outs[0][:-1])
    for o in outs[1:]:
        assert torch.equal(o, outs[0])
