"""Small softmax weights beside a dominant slot in the 8-bit cache's attention.

Tolerance: a weight is held in fp16, off by at most 2^-11 of itself or, in the units of the
largest weight times 2^eV (the power of two of its block of V) that its row sees, by 2^-36;
a score by 2^-17 of sum |q_d k_d| / sqrt(128) (as the log-sum-exp's test), twice (weight and
sum); bf16 rounds the result by at most 2^-8 of itself.  V is one value of [1, 2] a slot, in
dim slot % 128, so that nothing cancels and the bound is relative to the result.
"""
import numpy as np
import pytest

from kvq_util import HD, PAGE, Cache
from test_gpu_kvq import run_attention
from oracle import kvq as ok

pytestmark = pytest.mark.gpu


def one_hot_values(rng, n, heads=1):
    v = np.zeros((1, n, heads, HD))
    v[0, np.arange(n), :, np.arange(n) % HD] = rng.uniform(1, 2, size=(n, heads))
    return v


def sink_case(rng, n, log2, spread, sink, rows=1, g=2):
    """q [1][rows][g][128] and K [1][n][1][128]: the sink's weight is 2^log2 times the others',
    which spread by about `spread` binades."""
    sign = rng.choice([-1.0, 1.0], size=HD)
    q = sign * rng.uniform(4, 8, size=(1, rows, g, HD))
    k = np.zeros((1, n, 1, HD))
    if spread:
        k[0, :, 0] = rng.normal(size=(n, HD)) * spread * np.log(2) / 6.0
    k[0, sink, 0] = sign * log2 * np.log(2) * np.sqrt(HD) / (6.0 * HD)
    return q, k


def check(c, q, got, n, v_sink=0):
    k, v = c.val["k"][0, :n], c.val["v"][0, :n]
    e = np.repeat(c.exp["v"][0, :, 0], 16)[:n]
    for j in range(q.shape[1]):
        ref, lse, _ = ok.attend(q[0, j:j + 1], k, v, np.ones((1, n), dtype=bool))
        for h in range(q.shape[2]):
            p = np.exp(k[:, 0] @ q[0, j, h] / np.sqrt(HD) - lse[0, h])
            ds = 2.0 ** -17 * (np.abs(k[:, 0]) @ np.abs(q[0, j, h])).max() / np.sqrt(HD)
            floor = 2.0 ** -36 * (p * 2.0 ** e).max() * np.abs(v[:, 0] * 2.0 ** -e[:, None]).sum(axis=0)
            tol = (2.0 ** -8 + 2.0 ** -11 + 2 * ds + 2.0 ** -18) * ref[0, h] + floor
            err = np.abs(got[0, j, h] - ref[0, h])
            assert (err <= tol).all(), float((err / (tol + 1e-300)).max())


@pytest.mark.parametrize("n,log2,spread", [
    (2, 11, 0), (3, 10.6, 0), (9, 13.3, 1), (17, 16.2, 1), (140, 18.7, 1), (40, 21.4, 0),
    (1000, 10.6, 0), (4000, 12, 1), (16000, 14, 1), (16000, 16, 1), (32000, 18, 0), (6000, 24.4, 1),
])
@pytest.mark.parametrize("rows,g", [(1, 2), (3, 16)])
def test_weights_beside_a_sink(n, log2, spread, rows, g):
    rng = np.random.default_rng(n + int(log2 * 10))
    sink = n // 3
    q, k = sink_case(rng, n, log2, spread, sink, rows, g)
    v = one_hot_values(rng, n)
    v[0, sink] = 0
    c = Cache(1, 1, (n + PAGE - 1) // PAGE, seed=n)
    c.append([0], k, v)
    for ws in (True, False):
        got, _, qe = run_attention(c, q, "none", [n], ws=ws)
        check(c, qe, got, n)
    c.capi.dflash_kvq_check(c.h)


@pytest.mark.parametrize("log2", [22.6, 24])
def test_a_long_tail_of_tiny_weights(log2):
    """131,072 slots below 2^-22 of the largest still make up their share."""
    n = 131072
    rng = np.random.default_rng(int(log2))
    q, k = sink_case(rng, n, log2, 0, 5, 1, 1)
    v = one_hot_values(rng, n)
    v[0, 5] = 0
    c = Cache(1, 1, n // PAGE, seed=1)
    c.append([0], k, v)
    got, _, qe = run_attention(c, q, "none", [n])
    check(c, qe, got, n)


@pytest.mark.parametrize("late", [3, 14, 18, 30])
def test_weights_before_a_growing_maximum(late):
    """The maximum grows page by page: what was summed before is rescaled, not lost."""
    n = 6 * PAGE
    rng = np.random.default_rng(late)
    q, k = sink_case(rng, n, 1, 1, 0, 2, 8)
    sign = np.sign(q[0, 0, 0])
    for page in range(6):
        k[0, page * PAGE + 7, 0] = sign * late * page / 5 * np.log(2) * np.sqrt(HD) / (6.0 * HD)
    v = one_hot_values(rng, n)
    v[0, 7::PAGE] = 0
    c = Cache(1, 1, 6, seed=2)
    c.append([0], k, v)
    for ws in (True, False):
        got, _, qe = run_attention(c, q, "none", [n], ws=ws)
        check(c, qe, got, n)
