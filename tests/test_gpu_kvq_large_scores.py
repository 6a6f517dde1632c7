"""Scores so large that fp32 holds them to whole numbers or worse: the softmax is one slot's, and
its value comes out, not an overflow of weights taken relative to a rounded maximum.

Tolerance: the largest score exceeds the others of its row by far more than any rounding (checked
per row), so the result is that slot's V, rounded to bf16 (2^-8 of it); the weight itself cancels.
"""
import numpy as np
import pytest

from kvq_util import HD, Cache
from test_gpu_kvq import run_attention

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("k_scale", [1.0, 2.0 ** 12])
@pytest.mark.parametrize("log2", [8, 14, 16, 18, 20, 24, 30, 40, 60])
def test_attention_of_large_scores(log2, k_scale):
    rng = np.random.default_rng(log2)
    n, rows = 400, 16
    c = Cache(1, 1, 4)
    # V's blocks differ in their exponents too
    v = rng.normal(size=(1, n, 1, HD)) * 2.0 ** np.repeat(rng.integers(-9, 10, n // 16), 16)[:, None, None]
    c.append([0], rng.normal(size=(1, n, 1, HD)) * k_scale, v)
    q = rng.normal(size=(1, rows, 4, HD)) * 2.0 ** log2
    for ws in (True, False):
        got, lse, qe = run_attention(c, q, "none", [n], ws=ws)
        s = np.einsum("jhd,kd->jhk", qe[0], c.val["k"][0, :n, 0]) / np.sqrt(HD)
        order = np.sort(s, axis=-1)
        # fp32 sums of 256 products, and q to 2^-18 of its largest
        err = 2.0 ** -15 * np.abs(qe[0]).max() * np.abs(c.val["k"][0, :n, 0]).sum(axis=-1).max() / np.sqrt(HD)
        clear = order[..., -1] - order[..., -2] > 2 * err + 60
        assert clear.sum() >= rows
        want = c.val["v"][0, s.argmax(axis=-1), 0]
        assert (np.abs(got[0] - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -40)[clear].all()
        assert np.isfinite(got).all()
        top = order[..., -1]
        assert (np.abs(lse[0] - top) <= err + 2.0 ** -20 * np.abs(top) + 7).all()
    c.capi.dflash_kvq_check(c.h)
