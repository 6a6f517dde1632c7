"""Log probabilities, entropy and alternatives (dflash_token_logprobs) against the fp64 oracle.

Tolerances.  Ids are exact.  S = sum e^(x - m) is an fp32 sum in which a thread adds at most
n / 256 + 16 terms one after the other (n the vocabulary), each off by 2^-22 and the rounding of
its argument, 2^-23 |x - m| e^(x - m) (a term of at most 2^-1.5 absolute for any x); so log S is
off by at most 2^-24 (n / 256 + 64) + 2^-20, and a log probability by that and the
rounding of its two subtractions, 2^-23 (|x - m| + |lp|).  T adds terms d e^d of one sign the same
way, so the entropy is off by that relative to log S and to |T| / S: twice the above times
(1 + |T| / S).
"""
import numpy as np
import pytest
import torch

from oracle import packed as op

pytestmark = pytest.mark.gpu


def capi():
    from block_diffusion_speculative_injection_gb300 import capi as c
    return c


def run(x, tokens, top, stride=None, entropy=True):
    """Outputs as numpy, from junk."""
    R = x.shape[0]
    lp, en = torch.full((R,), 5.0, device="cuda"), torch.full((R,), 5.0, device="cuda")
    ids = torch.full((R, top), 5, dtype=torch.int32, device="cuda")
    best = torch.full((R, top), 5.0, device="cuda")
    capi().dflash_token_logprobs(x, tokens, top, lp if tokens is not None else None,
                                 en if entropy else None, ids if top else None, best if top else None)
    torch.cuda.synchronize()
    return [t.double().cpu().numpy() for t in (lp, en)] + [ids.cpu().numpy(), best.double().cpu().numpy()]


def check(x, tokens, top, got):
    V = x.shape[1]
    rel = 2.0 ** -24 * (V / 256 + 64) + 2.0 ** -20
    xs, ts = x.double().cpu().numpy(), tokens.tolist()
    for r, t in enumerate(ts):
        if t < 0:
            assert got[0][r] == got[1][r] == 5.0 and (got[2][r] == 5).all() and (got[3][r] == 5).all()
            continue
        lp, en, ids, vals = op.logprobs(xs[r], t, top)
        m = xs[r].max() if np.isfinite(xs[r].max()) else 0.0

        def near(a, b):
            if np.isinf(b):
                return a == b
            return abs(a - b) <= rel + 2.0 ** -22 * abs(b)
        assert near(got[0][r], lp), (r, got[0][r], lp)
        assert list(got[2][r]) == ids, r
        assert all(near(a, b) for a, b in zip(got[3][r], vals)), r
        span = en + abs(np.log(np.exp(xs[r][xs[r] > -np.inf] - m).sum())) if ids != [-1] * top or top == 0 else 0
        assert abs(got[1][r] - en) <= 2 * rel * (1 + span), (r, got[1][r], en)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,vocab,top", [
    (1, 1, 1), (3, 2, 2), (2, 7, 32), (5, 31, 3), (1, 255, 5), (4, 1000, 32), (3, 4095, 20),
    (2, 4097, 8), (9, 5000, 1), (1, 32003, 32), (40, 9001, 20), (1, 151936, 20), (7, 128257, 5),
    (160, 6000, 4), (2, 8192, 0),
])
def test_against_oracle(rows, vocab, top, dtype):
    gen = torch.Generator(device="cuda").manual_seed(vocab + top)
    x = (torch.randn(rows, vocab, device="cuda", generator=gen) * 3).to(dtype)
    tokens = torch.randint(0, vocab, (rows,), device="cuda", generator=gen).to(torch.int32)
    tokens[rows // 2] = -1 if rows > 2 else 0
    if rows > 3:
        tokens[1] = vocab  # no such id: log probability -inf
    check(x, tokens, top, run(x, tokens, top))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("top", [16, 17, 31, 32])
def test_long_rows_of_a_cta_each(top, dtype):
    """The list of alternatives is cut several times: scattered logits, a few values many times,
    and a list that overflows."""
    R, vocab = 310, 70001
    gen = torch.Generator(device="cuda").manual_seed(top)
    x = (torch.randn(R, vocab, device="cuda", generator=gen) * 2).to(dtype)
    x[1] = torch.randint(-5, 6, (vocab,), device="cuda", generator=gen).to(dtype)
    x[2] = (torch.arange(vocab, device="cuda") * 2.0 ** -8).to(dtype)
    x[3] += (torch.arange(vocab, device="cuda") * 2.0 ** -12).to(dtype)
    x[4, 5000:] += 9
    x[5] = torch.arange(vocab, device="cuda") // 9000
    x[6] = -float("inf")
    x[6, 9000:] = torch.arange(vocab - 9000, device="cuda") % 1000 * 0.01
    x[7] = 1
    tokens = torch.randint(0, vocab, (R,), device="cuda", generator=gen).to(torch.int32)
    got = run(x, tokens, top)
    check(x[:12], tokens[:12], top, [g[:12] for g in got])
    check(x[-3:], tokens[-3:], top, [g[-3:] for g in got])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("pad", [1, 2, 3, 5])
def test_strides_and_misaligned_rows(pad, dtype):
    gen = torch.Generator(device="cuda").manual_seed(pad)
    wide = torch.full((5, 4500 + pad), float("nan"), device="cuda", dtype=dtype)
    x = wide[:, pad - 1:pad - 1 + 4500]
    x.copy_(torch.randn(5, 4500, device="cuda", generator=gen) * 4)
    tokens = torch.tensor([0, 4499, 3, 17, 2222], dtype=torch.int32, device="cuda")
    check(x, tokens, 9, run(x, tokens, 9))


def test_elements_past_32_bits():
    wide = torch.empty(1100, 2 ** 21 + 3, dtype=torch.bfloat16, device="cuda")
    assert wide.numel() > 2 ** 31
    x = wide[:, -5001:]
    x[1080:] = torch.randn(20, 5001, device="cuda", generator=torch.Generator(device="cuda").manual_seed(0))
    tokens = torch.full((1100,), -1, dtype=torch.int32, device="cuda")
    tokens[1080:] = torch.arange(20, device="cuda") * 250
    got = run(x, tokens, 6)
    check(x[1070:], tokens[1070:], 6, [g[1070:] for g in got])


def patterns(vocab):
    i = torch.arange(vocab, device="cuda").float()
    yield torch.zeros(vocab, device="cuda")                       # all equal
    yield i * 1e-3                                                # rising: everything is a candidate
    yield -i * 1e-3                                               # falling
    yield torch.where(i < vocab - 50, -float("inf"), i * 0.01)    # only the last ids
    yield torch.where(i % 97 == 5, (i * 37) % 11, torch.tensor(-float("inf"), device="cuda"))
    yield torch.where(i == vocab // 2, 3.0, -float("inf"))        # one id
    yield torch.full((vocab,), -float("inf"), device="cuda")      # none
    yield torch.where(i % 2 == 0, 0.0, -0.0)                      # zeros of both signs are equal
    yield torch.full((vocab,), -3e38, device="cuda")
    yield torch.where(i == 7, 1e30, i)
    yield (i * 2654435761.0) % 1000 * -1e-2
    yield torch.where(i > 5000, 1.0, -float("inf")) + (i % 3)


@pytest.mark.parametrize("vocab", [40, 5000, 20011])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("copies", [1, 30])
def test_patterns(vocab, dtype, copies):
    """copies: rows split over a cluster, or a CTA each."""
    x = torch.stack(list(patterns(vocab)) * copies).to(dtype)
    tokens = torch.full((x.shape[0],), vocab // 2, dtype=torch.int32, device="cuda")
    got = run(x, tokens, 12)
    n = x.shape[0] // copies
    check(x[:n], tokens[:n], 12, [g[:n] for g in got])
    for g in got:  # and equal rows give equal results
        np.testing.assert_array_equal(g, np.concatenate([g[:n]] * copies))


def test_nan_and_infinity():
    gen = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn(4, 6000, device="cuda", generator=gen)
    x[1, 100], x[2, 5999], x[3, 0] = float("nan"), float("inf"), float("nan")
    tokens = torch.tensor([3, 3, 3, 3], dtype=torch.int32, device="cuda")
    lp, en, ids, best = run(x, tokens, 4)
    assert np.isfinite([lp[0], en[0]]).all() and np.isfinite(best[0]).all()
    for r in (1, 2, 3):
        assert np.isnan(lp[r]) and np.isnan(en[r]) and np.isnan(best[r]).all()


def test_some_of_the_outputs():
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(6, 7000, device="cuda", generator=gen)
    tokens = torch.arange(6, dtype=torch.int32, device="cuda")
    whole = run(x, tokens, 5)
    none = run(x, None, 5, entropy=False)
    assert (none[0] == 5.0).all() and (none[1] == 5.0).all()
    np.testing.assert_array_equal(none[2], whole[2])
    only = run(x, tokens, 0, entropy=False)
    np.testing.assert_array_equal(only[0], whole[0])


def test_captured():
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(3, 9000, device="cuda", generator=gen)
    tokens = torch.tensor([1, 2, 3], dtype=torch.int32, device="cuda")
    lp = torch.zeros(3, device="cuda")
    ids, best = torch.zeros(3, 4, dtype=torch.int32, device="cuda"), torch.zeros(3, 4, device="cuda")
    capi().dflash_token_logprobs(x, tokens, 4, lp, None, ids, best)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        capi().dflash_token_logprobs(x, tokens, 4, lp, None, ids, best)
    x.copy_(torch.randn(3, 9000, device="cuda", generator=gen))
    tokens.copy_(torch.tensor([9, 8, 7], dtype=torch.int32, device="cuda"))
    g.replay()
    torch.cuda.synchronize()
    want = run(x, tokens, 4)
    np.testing.assert_array_equal(lp.double().cpu().numpy(), want[0])
    np.testing.assert_array_equal(ids.cpu().numpy(), want[2])
