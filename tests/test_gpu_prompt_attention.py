"""Attention of packed prompts (dflash_prompt_attention) against the fp64 oracle.

Tolerances.  A weight is rounded to bf16 (half a step, 2^-8 of itself at most) and so is the
result; scores are fp32 sums of 128 products (2^-24 of sum |q_d k_d| for each of 128 additions at
most, 2^-17 of it in all, and here less than 2^-10 of a weight), the exponential and the sums add
less than 2^-18:
  |out - ref| <= 2^-8 |ref| + (2^-8 + 2^-10) sum_k p_k |v_k|.
lse: 2^-17 of the largest sum |q_d k_d| / sqrt(128), and 2^-18.
"""
import numpy as np
import pytest
import torch

from oracle import packed as op

pytestmark = pytest.mark.gpu
HD = 128


def capi():
    from block_diffusion_speculative_injection_gb300 import capi as c
    return c


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Case:
    """Packed Q, K and V as slices of one buffer, `lead` rows before and `pad` behind."""

    def __init__(self, lens, hkv, g, seed=0, lead=0, pad=0, q_scale=1.5, wide=0):
        rng = np.random.default_rng(seed)
        self.lens, self.hkv, self.H = lens, hkv, hkv * g
        self.T = lead + sum(lens) + pad
        x = rng.normal(size=(self.T, self.H + 2 * hkv + wide, HD))
        x[:, :self.H] *= q_scale
        x[:, self.H:self.H + hkv] *= np.exp(0.5 * rng.normal(size=(1, hkv, HD)))
        self.t = torch.from_numpy(x).to(torch.bfloat16).cuda()
        self.off = [lead]
        for n in lens:
            self.off.append(self.off[-1] + n)

    @property
    def qkv(self):
        h, k = self.H, self.hkv
        return self.t[:, :h], self.t[:, h:h + k], self.t[:, h + k:h + 2 * k]

    def run(self, causal, lse=True, offsets=None, status=None):
        q, k, v = self.qkv
        self.out = torch.full((self.T, self.H, HD), 7.0, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((self.T, self.H), 7.0, device="cuda") if lse else None
        self.status = i32([0]) if status is None else status
        self.offsets = i32(self.off) if offsets is None else offsets
        capi().dflash_prompt_attention(len(self.offsets) - 1, causal, self.offsets, q, k, v, self.out,
                                       self.lse, self.status)
        torch.cuda.synchronize()
        return self.out, self.lse

    def check(self, causal, skip=()):
        q, k, v = (x.double().cpu().numpy() for x in self.qkv)
        got = self.out.double().cpu().numpy()
        glse = None if self.lse is None else self.lse.double().cpu().numpy()
        used = np.zeros(self.T, dtype=bool)
        for b, n in enumerate(self.lens):
            a, e = self.off[b], self.off[b + 1]
            used[a:e] = True
            if n == 0 or b in skip:
                continue
            ref, lse, mag = op.attend(q[a:e], k[a:e], v[a:e], causal)
            tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -10) * mag
            assert (np.abs(got[a:e] - ref) <= tol).all(), (b, np.abs(got[a:e] - ref).max())
            if glse is not None:
                big = np.abs(q[a:e]).max() * np.abs(k[a:e]).sum(-1).max() / np.sqrt(HD)
                np.testing.assert_allclose(glse[a:e], lse, rtol=0,
                                           atol=2.0 ** -17 * big + 2.0 ** -18 * (1 + np.abs(lse).max()))
        assert (got[~used] == 7.0).all()  # rows of no sequence stay
        if glse is not None:
            assert (glse[~used] == 7.0).all()
        assert int(self.status) == 0


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,hkv,g,lead,pad", [
    ([1], 1, 1, 0, 0), ([1, 1, 1], 2, 4, 0, 3), ([5, 0, 2, 17], 2, 4, 0, 1), ([0, 0], 1, 2, 2, 2),
    ([31, 32, 33], 1, 4, 7, 0), ([127, 128, 129], 1, 1, 0, 0), ([64, 65, 255, 256, 257], 1, 2, 0, 200),
    ([300], 2, 3, 0, 0), ([130, 90], 1, 5, 1, 0), ([200, 3], 2, 7, 0, 0), ([140], 1, 16, 0, 1),
    ([70, 10], 1, 64, 0, 0), ([75], 1, 33, 0, 0), ([513], 1, 8, 0, 5),
])
def test_attention(lens, hkv, g, lead, pad, causal):
    c = Case(lens, hkv, g, seed=sum(lens) + g, lead=lead, pad=pad)
    c.run(causal)
    c.check(causal)


def test_many_prompts():
    rng = np.random.default_rng(5)
    c = Case([int(x) for x in rng.integers(0, 40, 300)], 2, 2, seed=5, pad=9)
    c.run(True)
    c.check(True)


def test_long_prompt():
    """Enough rows for two query tiles a CTA on every SM."""
    c = Case([1500, 1301], 8, 4, seed=3)
    c.run(True)
    q, k, v = (x.double() for x in c.qkv)
    for b in range(2):
        a, e = c.off[b], c.off[b + 1]
        for h in (0, 13, 31):
            s = q[a:e, h] @ k[a:e, h // 4].T / np.sqrt(HD)
            s = s.masked_fill(torch.ones_like(s).triu(1).bool(), -np.inf)
            p = torch.softmax(s, -1)
            ref, mag = p @ v[a:e, h // 4], p @ v[a:e, h // 4].abs()
            assert ((c.out[a:e, h] - ref).abs() <= 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -10) * mag).all()
            assert torch.allclose(c.lse[a:e, h].double(), torch.logsumexp(s, -1), rtol=0, atol=1e-4)


def test_elements_past_32_bits():
    hkv, g, off = 8192, 2, [1020, 1021, 1099]
    gen = torch.Generator(device="cuda").manual_seed(0)
    x = torch.empty(1100, hkv * (g + 2), HD, dtype=torch.bfloat16, device="cuda")
    x[1000:].normal_(generator=gen)
    q, k, v = x[:, :hkv * g], x[:, hkv * g:-hkv], x[:, -hkv:]
    out = torch.full((1100, hkv * g, HD), 7.0, dtype=torch.bfloat16, device="cuda")
    lse, status = torch.full((1100, hkv * g), 7.0, device="cuda"), i32([0])
    assert out.numel() > 2 ** 31
    capi().dflash_prompt_attention(2, True, i32(off), q, k, v, out, lse, status)
    capi().dflash_status_check(status)
    assert (out[1019] == 7).all() and (out[1099] == 7).all() and (lse[1019] == 7).all()
    for a, e in zip(off, off[1:]):
        for h in (0, 9001, hkv * g - 1):
            f = [t[a:e, i:i + 1].double().cpu().numpy() for t, i in ((q, h), (k, h // g), (v, h // g))]
            ref, ref_lse, mag = op.attend(*f, True)
            err = np.abs(out[a:e, h:h + 1].double().cpu().numpy() - ref)
            assert (err <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -10) * mag).all()
            np.testing.assert_allclose(lse[a:e, h:h + 1].cpu().numpy(), ref_lse, rtol=0, atol=1e-4)


def test_without_lse_and_wide_rows():
    c = Case([77, 140], 2, 4, seed=9, wide=3)
    c.run(True, lse=False)
    c.check(True)


def test_growing_scores():
    """Scores that rise along the keys: every tile raises the maximum by more than 2^8."""
    c = Case([700], 1, 4, seed=4)
    q, k, v = c.qkv
    q[:] = 1.0
    k[:] = (torch.arange(700, device="cuda")[:, None, None] * 0.25).to(torch.bfloat16)
    c.run(True)
    c.check(True)
    c.run(False)
    c.check(False)


@pytest.mark.parametrize("scale", [2.0 ** 12, 2.0 ** 18, 2.0 ** 24])
def test_large_scores(scale):
    """Scores far beyond fp32's integers keep their order: one key wins each row, or a tie."""
    c = Case([200], 1, 4, seed=6)
    q, k, v = c.qkv
    q *= scale
    k *= scale
    c.run(True)
    qd, kd, vd = (x.double() for x in c.qkv)
    for h in range(4):
        s = qd[:, h] @ kd[:, 0].T / np.sqrt(HD)
        s = s.masked_fill(torch.ones_like(s).triu(1).bool(), -np.inf)
        top = s.topk(2, dim=-1)
        # rows whose best key leads by more than the scores' own rounding
        clear = torch.ones(200, dtype=torch.bool, device="cuda")
        err = 2.0 ** -16 * (qd[:, h].abs() @ kd[:, 0].abs().T).amax(-1) / np.sqrt(HD)
        clear[1:] = (top.values[:, 0] - top.values[:, 1])[1:] > err[1:] + 40
        assert clear.sum() > 100
        assert (c.out[:, h].double()[clear] == vd[top.indices[:, 0], 0][clear]).all()


def test_nan_and_infinity_stay_where_they_are_seen():
    c = Case([40, 200, 60], 2, 4, seed=8)
    q, k, v = c.qkv
    a = c.off[1]
    v[a + 130, 1, 5] = float("nan")
    v[a + 131, 1, 6] = float("-inf")
    v[a + 3, 0, 7] = float("inf")
    v[a + 150:a + 152, 1, 9] = torch.tensor([float("inf"), float("-inf")], device="cuda")
    k[a + 140, 0] = float("nan")
    q[a + 20, 2] = float("nan")
    plain = c.t.clone()
    c.run(True)
    c.check(True, skip=(1,))  # the prompts beside it know nothing of it
    out = c.out[a:a + 200].float()
    g1 = out[:, 4:8]  # query heads of KV head 1
    assert torch.isfinite(g1[:130]).all()
    assert torch.isnan(g1[130:, :, 5]).all() and (g1[131:, :, 6] == -np.inf).all()
    assert (g1[150, :, 9] == np.inf).all() and torch.isnan(g1[151:, :, 9]).all()
    assert torch.isfinite(g1[:150, :, 9]).all()
    rest = [d for d in range(HD) if d not in (5, 6, 9)]
    assert torch.isfinite(g1[:, :, rest]).all()
    g0 = out[:, :4]
    assert torch.isfinite(g0[:3]).all() and (g0[3:20, :, 7] == np.inf).all()
    assert torch.isnan(g0[140:]).all() and torch.isnan(g0[20, 2]).all()
    assert torch.isfinite(g0[21:140, :, :7]).all()
    # and the finite part is what it would be without them
    c2 = Case([40, 200, 60], 2, 4, seed=8)
    c2.run(True)
    assert torch.equal(c2.out[a:a + 130, 4:8], c.out[a:a + 130, 4:8])
    assert torch.equal(c2.out[a:a + 200, 4:8][:, :, rest], c.out[a:a + 200, 4:8][:, :, rest])
    assert torch.equal(torch.isnan(plain), torch.isnan(c.t))


def test_neighbours_of_a_bad_prompt_bidirectional():
    c = Case([50, 30, 50], 1, 2, seed=2)
    c.t[c.off[1]:c.off[2]] = float("nan")
    c.run(False)
    c.check(False, skip=(1,))
    assert torch.isnan(c.out[c.off[1]:c.off[2]]).all()


def test_runs_are_equal():
    c = Case([700, 55], 2, 4, seed=1)
    first = [x.clone() for x in c.run(True)]
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, c.run(True)))


BAD = [[0, 50, 40, 90], [0, 50, 60, 91], [-1, 50, 60, 90], [60, 50, 40, 0], [0, -5, 20, 90], [0, 1 << 25, 3, 90],
       [0, 90, 10, 50], [-2 ** 31, 2 ** 31 - 1, -7, 90], [90, 90, 0, 90]]


@pytest.mark.parametrize("off", BAD)
def test_bad_offsets_set_the_status(off):
    """And nothing outside the arrays is written."""
    c = Case([50, 10, 30], 1, 4, seed=1)
    q, k, v = c.qkv
    wide = torch.full((c.T + 400, c.H, HD), 3.0, dtype=torch.bfloat16, device="cuda")
    wide_lse = torch.full((c.T + 400, c.H), 3.0, device="cuda")
    status = i32([0])
    capi().dflash_prompt_attention(3, True, i32(off), q, k, v, wide[200:200 + c.T], wide_lse[200:200 + c.T], status)
    with pytest.raises(capi().DFlashError) as e:
        capi().dflash_status_check(status)
    assert e.value.status == 5
    capi().dflash_status_check(status)  # and clears
    for w in (wide, wide_lse):
        assert (w[:200] == 3.0).all() and (w[200 + c.T:] == 3.0).all()


def test_many_bad_offsets():
    rng = np.random.default_rng(0)
    c = Case([300], 2, 4, seed=1)
    q, k, v = c.qkv
    wide = torch.full((c.T + 400, c.H, HD), 3.0, dtype=torch.bfloat16, device="cuda")
    for _ in range(20):
        off = rng.integers(-40, 360, 101)
        status = i32([0])
        capi().dflash_prompt_attention(100, True, i32(off), q, k, v, wide[200:200 + c.T], None, status)
        assert int(status) == 3
    assert (wide[:200] == 3.0).all() and (wide[200 + c.T:] == 3.0).all()


def test_captured_with_other_lengths_and_streams():
    """A captured call serves other lengths of the same number of rows; two streams at once."""
    c = Case([100, 60, 40], 2, 4, seed=7)
    q, k, v = c.qkv
    off = i32(c.off)
    outs = [torch.zeros(c.T, c.H, HD, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    status = i32([0])
    capi().dflash_prompt_attention(3, True, off, q, k, v, outs[0], None, status)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        capi().dflash_prompt_attention(3, True, off, q, k, v, outs[0], None, status)
    c.lens, c.off = [3, 0, 190], [0, 3, 3, 193]
    off.copy_(i32(c.off))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g.replay()
    with torch.cuda.stream(s):
        capi().dflash_prompt_attention(3, True, off, q, k, v, outs[1], None, status)
    torch.cuda.synchronize()
    assert torch.equal(outs[0][:193], outs[1][:193])
    c.run(True)
    assert torch.equal(c.out[:193], outs[0][:193])
    c.check(True)
