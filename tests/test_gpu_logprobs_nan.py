"""Rows with a NaN or +inf in dflash_token_logprobs: NaN for every number, whatever else the row
holds, also where fewer than `top` alternatives are left or the token is no id of the vocabulary."""
import numpy as np
import pytest
import torch

from oracle import packed as op

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


def rows_of(vocab):
    """(row, whether it holds a NaN or +inf)."""
    gen = torch.Generator().manual_seed(vocab)
    x = torch.randn(vocab, generator=gen)
    at = [0, vocab // 2, vocab - 1]
    yield x, False
    yield torch.full((vocab,), NAN), True
    yield torch.full((vocab,), INF), True
    yield torch.full((vocab,), -INF), False
    for bad in (NAN, INF):
        for i in at:
            yield torch.where(torch.arange(vocab) == i, bad, x), True           # among finite ones
            yield torch.where(torch.arange(vocab) == i, bad, -INF), True        # the only one left
            few = torch.where(torch.arange(vocab) % 977 == 1, x, -INF)          # a mask that leaves a few
            few[i] = bad
            yield few, True
    few = torch.where(torch.arange(vocab) % 977 == 1, x, -INF)
    yield few, False
    both = x.clone()
    both[0], both[-1] = INF, NAN
    yield both, True
    # a vector whose other values are the row's best
    best = x - 50
    best[vocab // 3:vocab // 3 + 8] = 5
    best[vocab // 3] = NAN
    yield best, True


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab,top", [(1, 3), (2, 1), (3, 5), (40, 32), (6000, 4), (20011, 20)])
@pytest.mark.parametrize("copies", [1, 30])
@pytest.mark.parametrize("token", ["in", "out"])
def test_every_number_is_nan(vocab, top, dtype, copies, token):
    """copies: rows split over a cluster, or a CTA each."""
    from block_diffusion_speculative_injection_gb300 import capi
    rows = list(rows_of(vocab)) * copies
    x = torch.stack([r for r, _ in rows]).to(dtype).cuda()
    bad = np.array([b for _, b in rows])
    R = len(rows)
    tokens = torch.full((R,), vocab // 2 if token == "in" else vocab + 3, dtype=torch.int32, device="cuda")
    lp, en = torch.full((R,), 5.0, device="cuda"), torch.full((R,), 5.0, device="cuda")
    ids = torch.full((R, top), 5, dtype=torch.int32, device="cuda")
    best = torch.full((R, top), 5.0, device="cuda")
    capi.dflash_token_logprobs(x, tokens, top, lp, en, ids, best)
    torch.cuda.synchronize()
    lp, en, ids, best = lp.cpu().numpy(), en.cpu().numpy(), ids.cpu().numpy(), best.cpu().numpy()
    for name, got in (("logp", lp), ("entropy", en), ("top_logp", best)):
        nan = np.isnan(got)
        assert nan[bad].all(), (name, np.argwhere(~nan & (bad if nan.ndim == 1 else bad[:, None]))[:4])
        assert not nan[~bad].any(), name
    assert (ids >= -1).all() and (ids < vocab).all()
    for r in np.flatnonzero(~bad)[:3 * copies]:  # and its neighbours know nothing of it
        w = op.logprobs(x[r].double().cpu().numpy(), int(tokens[r]), top)
        assert ids[r].tolist() == w[2]
        # 2^-24 (n / 256 + 64) + 2^-20 for log S, and the rounding of the subtractions
        tol = 2.0 ** -24 * (vocab / 256 + 64) + 2.0 ** -20
        for a, b in [(lp[r], w[0])] + list(zip(best[r], w[3])):
            assert a == b or abs(a - b) <= tol + 2.0 ** -22 * abs(b)
    only = torch.full((R,), 5.0, device="cuda")
    capi.dflash_token_logprobs(x, tokens, 0, only, None, None, None)  # (the kernel without alternatives)
    np.testing.assert_array_equal(np.isnan(only.cpu().numpy()), bad)
