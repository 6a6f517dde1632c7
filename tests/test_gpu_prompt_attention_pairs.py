"""dflash_prompt_attention with two query tiles a CTA, and CTAs that take on the items of others:
the form that every batch of some size takes.

Tolerances (as for the one-tile form).  A weight is rounded to bf16 (half a step, 2^-8 of itself at
most) and so is the result; scores are fp32 sums of 128 products (2^-24 of sum |q_d k_d| for each of
128 additions at most, 2^-17 of it in all, and here less than 2^-10 of a weight), the exponential and the
sums add less than 2^-18:
  |out - ref| <= 2^-8 |ref| + (2^-8 + 2^-10) sum_k p_k |v_k|.
lse: 2^-17 of the largest sum |q_d k_d| / sqrt(128), and 2^-18 (1 + the largest).
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
HD = 128

# Lengths against the 2 * (128 / g) positions of a CTA: ending in its first tile, in its second, between
# them, whole; none, one; steps of 128 keys that the tiles have in different numbers.
CASES = {
    1: (16, [316, 456, 384, 512, 100, 0, 1]),
    2: (20, [128 + 40, 128 * 3 + 100, 64, 256, 0, 1, 130]),
    3: (12, [188, 312, 126, 168, 0, 1]),
    4: (8, [202, 306, 160, 192, 0, 300]),
    7: (6, [149, 210, 126, 144, 0, 260]),
    16: (5, [133, 142, 136, 144, 1]),
    33: (3, [61, 94, 135, 0, 132]),
    64: (2, [41, 63, 130, 128]),
}


def capi():
    from block_diffusion_speculative_injection_gb300 import capi as c
    return c


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Batch:
    """Packed Q, K and V as slices of one buffer, `lead` rows before and `pad` behind."""

    def __init__(self, g, hkv, lens, seed=0, lead=3, pad=5, q_scale=1.5):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.g, self.hkv, self.H, self.lens = g, hkv, hkv * g, lens
        self.T = lead + sum(lens) + pad
        x = torch.randn(self.T, self.H + 2 * hkv, HD, device="cuda", generator=gen)
        x[:, :self.H] *= q_scale
        x[:, self.H:self.H + hkv] *= torch.exp(0.5 * torch.randn(1, hkv, HD, device="cuda", generator=gen))
        self.t = x.to(torch.bfloat16)
        self.off = [lead]
        for n in lens:
            self.off.append(self.off[-1] + n)
        # the library's rule: two tiles as soon as some SM has more than one item, and here more
        # items than SMs
        sms = torch.cuda.get_device_properties(0).multi_processor_count
        self.items = (self.T // (2 * (128 // g)) + len(lens)) * hkv
        assert 2 * self.items > sms and self.items > sms

    @property
    def qkv(self):
        h, k = self.H, self.hkv
        return self.t[:, :h], self.t[:, h:h + k], self.t[:, h + k:]

    def run(self, causal):
        self.out = torch.full((self.T, self.H, HD), 7.0, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((self.T, self.H), 7.0, device="cuda")
        status = i32([0])
        capi().dflash_prompt_attention(len(self.lens), causal, i32(self.off), *self.qkv, self.out, self.lse, status)
        capi().dflash_status_check(status)
        return self.out, self.lse

    def prompts(self):
        for a, e in zip(self.off, self.off[1:]):
            if e > a:
                yield slice(a, e)

    def scores(self, r, causal):
        """[H][n][n] of a prompt, -inf where a row does not see the key."""
        q, k, _ = (x[r].double().transpose(0, 1) for x in self.qkv)
        s = q @ k.repeat_interleave(self.g, 0).transpose(1, 2) / math.sqrt(HD)
        if causal:
            s.masked_fill_(torch.ones_like(s[0], dtype=torch.bool).triu(1), -math.inf)
        return s

    def values(self, r):
        return self.qkv[2][r].double().transpose(0, 1).repeat_interleave(self.g, 0)

    def check_rest(self):
        """Rows of no sequence stay."""
        used = torch.zeros(self.T, dtype=torch.bool, device="cuda")
        used[self.off[0]:self.off[-1]] = True
        assert (self.out[~used] == 7.0).all() and (self.lse[~used] == 7.0).all()

    def check(self, causal):
        for r in self.prompts():
            s, v = self.scores(r, causal), self.values(r)
            p = torch.softmax(s, -1)
            ref, mag = p @ v, p @ v.abs()
            err = (self.out[r].double().transpose(0, 1) - ref).abs()
            tol = 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -10) * mag
            assert (err <= tol).all(), (r, (err - tol).max(), torch.nonzero(err > tol)[:4])
            q, k, _ = (x[r].double() for x in self.qkv)
            big = float(q.abs().max() * k.abs().sum(-1).max()) / math.sqrt(HD)
            lse = torch.logsumexp(s, -1)
            err = (self.lse[r].double().T - lse).abs().max()
            assert err <= 2.0 ** -17 * big + 2.0 ** -18 * (1 + float(lse.abs().max())), (r, err)
        self.check_rest()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("g", CASES)
def test_values(g, causal):
    c = Batch(g, *CASES[g], seed=g)
    c.run(causal)
    c.check(causal)


@pytest.mark.parametrize("causal", [True, False])
def test_many_items_a_cta(causal):
    """A dozen items a CTA, long and short prompts in either order."""
    for lens in ([900, 300, 40, 0, 700, 1, 64], [1, 64, 0, 700, 40, 300, 900]):
        c = Batch(2, 96, lens, seed=7)
        assert c.items > 12 * torch.cuda.get_device_properties(0).multi_processor_count
        c.run(causal)
        c.check(causal)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("g", [1, 3, 4])
def test_scores_that_rise_and_fall(g, causal):
    """Scores rise along the keys for some heads and fall for others: rows of one warp raise their maximum
    by more than 2^8 at every step while others never do."""
    hkv, lens = CASES[g]
    c = Batch(g, hkv, lens, seed=g)
    q, k, _ = c.qkv
    sign = torch.tensor([1.0, -1.0, 0.01], device="cuda")[torch.arange(c.H, device="cuda") * 7 % 5 % 3]
    q[:] = sign[None, :, None]
    for r in c.prompts():
        k[r] = (torch.arange(r.stop - r.start, device="cuda")[:, None, None] * 0.25).to(torch.bfloat16)
    c.run(causal)
    c.check(causal)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("scale", [2.0 ** 12, 2.0 ** 18, 2.0 ** 24])
@pytest.mark.parametrize("g", [3, 4])
def test_large_scores(g, scale, causal):
    """Scores far beyond fp32's integers keep their order: one key wins each row, or a tie.  The
    winner's weight is 1 but for the rounding of the maximum times log2(e) / sqrt(128) (below 2^20 in
    binades, so up to 2^-4 of one, the same in the sum of weights); what is rounded to bf16 then, by half a
    step, is the weight and not the sum, so the row is v (1 + 2^-8), rounded once more."""
    c = Batch(g, *CASES[g], seed=g + 100)
    q, k, v = c.qkv
    q *= scale
    k *= scale
    c.run(causal)
    c.check_rest()
    n_clear = n = 0
    for r in c.prompts():
        s = c.scores(r, causal)
        if s.shape[-1] < 2:
            continue
        top = s.topk(2, dim=-1)
        q, k, _ = (x[r].double().abs().transpose(0, 1) for x in c.qkv)
        # rows whose best key leads by more than the scores' own rounding
        err = 2.0 ** -16 * (q @ k.repeat_interleave(g, 0).transpose(1, 2)).amax(-1) / math.sqrt(HD)
        clear = top.values[..., 0] - top.values[..., 1] > err + 40
        if causal:
            clear[:, 0] = True  # one key
        best = torch.gather(c.values(r), 1, top.indices[..., :1].expand(-1, -1, HD))
        err = (c.out[r].double().transpose(0, 1) - best)[clear].abs()
        assert (err <= (2 * 2.0 ** -8 + 2.0 ** -10) * best[clear].abs()).all()
        n, n_clear = n + clear.numel(), n_clear + int(clear.sum())
    assert n_clear > n // 2


@pytest.mark.parametrize("causal", [True, False])
def test_nan_and_infinity_stay_where_they_are_seen(causal):
    """In V, K and Q of some heads and prompts; the other items of the same CTAs do not notice."""
    g, hkv, lens = 2, 48, [128 + 40, 128 * 3 + 100, 64, 256, 0, 1, 130, 300]
    c, plain = (Batch(g, hkv, lens, seed=11) for _ in range(2))
    assert c.items > 4 * torch.cuda.get_device_properties(0).multi_processor_count
    q, k, v = c.qkv
    gen = torch.Generator().manual_seed(1)
    for h in range(0, hkv, 3):  # a few elements of V, in any tile
        for b in (0, 1, 3, 7):
            for _ in range(3):
                at, d = (int(torch.randint(0, m, (1,), generator=gen)) for m in (lens[b], HD))
                v[c.off[b] + at, h, d] = [math.nan, math.inf, -math.inf][(h // 3 + b) % 3]
    v[c.off[1] + 300, 4, 9], v[c.off[1] + 301, 4, 9] = math.inf, -math.inf
    v[c.off[2]:c.off[3], 7] = math.nan  # a whole prompt of a head
    k[c.off[1] + 200, 10] = math.nan
    q[c.off[3] + 77, 23] = math.nan
    c.run(causal)
    plain.run(causal)
    c.check_rest()
    for r in c.prompts():
        n = r.stop - r.start
        seen = torch.ones(n, n, dtype=torch.bool, device="cuda")
        if causal:
            seen = seen.tril()
        V = c.values(r)

        def any_seen(bad):  # [H][n keys][..] -> [H][n rows][..]
            return (seen.double() @ bad.double()) > 0
        nan = any_seen(V.isnan()) | (any_seen(V == math.inf) & any_seen(V == -math.inf))
        bad = any_seen(~V.isfinite())
        qd, kd, _ = (x[r].double().transpose(0, 1) for x in c.qkv)
        whole = any_seen(kd.repeat_interleave(g, 0).isnan().any(-1, keepdim=True)) | qd.isnan().any(-1, keepdim=True)
        got, want = (x.out[r].double().transpose(0, 1) for x in (c, plain))
        assert got[whole.expand_as(got) | nan].isnan().all()
        rest = ~whole.expand_as(got)
        assert (~got[rest & bad].isfinite()).all()
        only = rest & bad & ~nan & got.isinf()  # infinities have the sign of those seen
        sign = torch.where(any_seen(V == math.inf), math.inf, -math.inf)
        assert (got[only] == sign[only]).all()
        assert torch.equal(got[rest & ~bad], want[rest & ~bad])
        lse, want = c.lse[r].T, plain.lse[r].T
        assert lse[whole[..., 0]].isnan().all() and torch.equal(lse[~whole[..., 0]], want[~whole[..., 0]])


def test_runs_are_equal():
    c = Batch(4, 32, [700, 55, 0, 400, 129, 640], seed=1)
    for causal in (True, False):
        first = [x.clone() for x in c.run(causal)]
        for _ in range(6):
            assert all(torch.equal(a, b) for a, b in zip(first, c.run(causal)))


def test_captured_with_other_lengths_beside_another_stream():
    c = Batch(4, 16, [300, 200, 100], seed=5, lead=0, pad=0)
    off, status = i32(c.off), i32([0])
    outs = [torch.zeros(c.T, c.H, HD, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    call = lambda o: capi().dflash_prompt_attention(3, True, off, *c.qkv, o, None, status)
    call(outs[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(outs[0])
    side = torch.cuda.Stream()
    for lens in ([3, 0, 590], [0, 600, 0], [129, 255, 128], [1, 1, 1]):
        c.lens, c.off = lens, [0, lens[0], lens[0] + lens[1], sum(lens)]
        off.copy_(i32(c.off))
        for o in outs:
            o.fill_(7.0)
        side.wait_stream(torch.cuda.current_stream())
        graph.replay()
        with torch.cuda.stream(side):
            call(outs[1])
        torch.cuda.synchronize()
        capi().dflash_status_check(status)
        assert torch.equal(outs[0], outs[1])
        c.run(True)
        assert torch.equal(c.out[:c.off[-1]], outs[0][:c.off[-1]])
        c.check(True)


def test_millions_of_empty_prompts():
    """Two prompts with 2^26 - 3 empty ones between: 3.5 million empty items in a row for each CTA, for
    longer than a wait within the kernel may take."""
    B, hkv, lens = (1 << 26) - 1, 8, (100, 60)
    gen = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn(160, 3 * hkv, HD, device="cuda", generator=gen).to(torch.bfloat16)
    q, k, v = x[:, :hkv], x[:, hkv:2 * hkv], x[:, 2 * hkv:]
    off = torch.full((B + 1,), lens[0], dtype=torch.int32, device="cuda")
    off[0], off[B] = 0, 160
    out, few = (torch.zeros(160, hkv, HD, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    status = i32([0])
    capi().dflash_prompt_attention(B, True, off, q, k, v, out, None, status)
    capi().dflash_status_check(status)
    capi().dflash_prompt_attention(2, True, i32([0, 100, 160]), q, k, v, few, None, status)
    capi().dflash_status_check(status)
    assert torch.equal(out, few)
