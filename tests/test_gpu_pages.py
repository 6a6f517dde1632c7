"""Pages mapped and given back on the GPU (dflash_pages_map, dflash_pages_release) against the
list oracle.  Everything is integers and exact."""
import numpy as np
import pytest
import torch

from oracle import packed as op

pytestmark = pytest.mark.gpu
PAGE = 128
CODE = {"check": 5, "capacity": 2}


def capi():
    from block_diffusion_speculative_injection_gb300 import capi as c
    return c


def i32(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")


class Pool:
    def __init__(self, n_pages, n_seqs, pps):
        self.o = op.Pages(n_pages, n_seqs, pps)
        self.h = capi().Pages.empty(n_pages, n_seqs, pps)
        self.table, self.mapped, self.free, self.n_free, self.status = self.h.tensors

    def same(self):
        o = self.o
        assert self.table.tolist() == o.table
        assert self.mapped.tolist() == o.mapped
        assert int(self.n_free) == len(o.free)
        assert self.free.tolist() == o.free + [-1] * (o.n_pages - len(o.free))

    def failed(self, wrong):
        """The status names one of the failures (whichever a thread met first), then clears."""
        if not wrong:
            capi().dflash_status_check(self.status)
            return
        with pytest.raises(capi().DFlashError) as e:
            capi().dflash_status_check(self.status)
        assert e.value.status in [CODE[w] for w in wrong]
        assert int(self.status) == 0

    def map(self, seqs, start, counts, n_rows=None):
        B = len(seqs)
        n_rows = sum(max(c, 0) for c in counts) if n_rows is None else n_rows
        off, lens = (torch.full((B + k,), -7, dtype=torch.int32, device="cuda") for k in (1, 0))
        rows = [torch.full((n_rows,), -7, dtype=torch.int32, device="cuda") for _ in range(3)]
        capi().dflash_pages_map(self.h, B, n_rows, i32(seqs), i32(start), i32(counts), off, lens, *rows)
        want = self.o.map(seqs, start, counts, n_rows)
        assert off.tolist() == want[0]
        assert lens.tolist() == want[1]
        assert list(zip(*[r.tolist() for r in rows])) == want[2]
        self.same()
        self.failed(want[3])
        return off, lens, rows

    def release(self, seqs, keep):
        capi().dflash_pages_release(self.h, len(seqs), i32(seqs), i32(keep))
        wrong = self.o.release(seqs, keep)
        self.same()
        self.failed(wrong)


@pytest.mark.parametrize("seed,batch,hi", [(0, 1, 1), (1, 3, 300), (2, 40, 700), (3, 257, 20),
                                           (4, 1025, 3), (5, 7, 5000)])
def test_steps_of_a_server(seed, batch, hi):
    rng = np.random.default_rng(seed)
    n_seqs, pps = batch + 2, (3 * hi) // PAGE + 3
    p = Pool(n_seqs * pps - 1, n_seqs, pps)
    lens = [0] * n_seqs
    for step in range(4):
        seqs = [int(x) for x in rng.permutation(n_seqs)[:batch]]
        counts = [int(x) for x in rng.integers(0, hi + 1, batch)]
        start = [min(lens[q], pps * PAGE - hi) for q in seqs]
        p.release(seqs, start)  # what was rejected, or nothing
        _, got, _ = p.map(seqs, start, counts, sum(counts) + 3)
        for q, n in zip(seqs, got.tolist()):
            lens[q] = int(rng.integers(0, n + 1))
    before = [t.clone() for t in p.h.tensors]
    seqs = list(range(n_seqs))
    have = p.mapped.tolist()
    p.release(seqs, [0] * n_seqs)
    assert int(p.n_free) == n_seqs * pps - 1
    p.map(seqs, [0] * n_seqs, [m * PAGE for m in have])  # takes the same pages again
    assert all(torch.equal(a, b) for a, b in zip(before, p.h.tensors))


def test_pages_run_out_in_order():
    p = Pool(4, 6, 3)
    p.map([0, 1, 2, 3], [0, 0, 0, 0], [100, 300, 10, 0])  # 1 + 3, then none left
    assert p.mapped.tolist() == [1, 3, 0, 0, 0, 0]
    p.map([0, 4, 1], [100, 0, 300], [28, 1, 84])  # the rooms they have are used
    p.release([1], [1])
    p.map([4, 2, 5, 3], [0, 0, 0, 5], [129, 1, 0, 3])


def test_refused_entries_change_nothing():
    p = Pool(40, 8, 2)
    p.map([0, 1], [0, 0], [130, 5])
    for seqs, start, counts in (([0, 9, 2], [130, 0, 0], [1, 4, 4]), ([-1, 2], [0, 0], [4, 4]),
                                ([3, 3, 4, 3], [0, 0, 0, 7], [4, 5, 6, 7]), ([5, 6], [-1, 0], [3, 2]),
                                ([5, 6], [-3, 0], [3, 2]), ([5, 6], [0, 0], [-3, 2]),
                                ([7, 2], [200, 0], [57, 3]), ([7, 2], [2 ** 31 - 1, 0], [1, 3]),
                                ([7, 2], [0, 0], [2 ** 30 - 1, 3])):
        total = sum(c for c in counts if 0 <= c < 10 ** 6)
        p.map(seqs, start, counts, total)
    p.release([0, 9, 0, 1], [128, 0, 0, 0])
    p.release([2, 3], [-1, 0])


def test_more_rows_than_the_packed_batch_holds():
    p = Pool(20, 4, 3)
    p.map([0, 1, 2], [0, 0, 0], [100, 100, 100], 250)
    p.map([3], [0], [1], 0)


def test_counts_that_are_not_the_pools():
    p = Pool(6, 2, 3)
    p.n_free.fill_(5)
    before = [t.clone() for t in p.h.tensors[:4]]
    p.mapped.fill_(2)
    with pytest.raises(capi().DFlashError):
        capi().dflash_pages_release(p.h, 2, None, None)
        capi().dflash_status_check(p.status)
    p.mapped.zero_()
    assert all(torch.equal(a, b) for a, b in zip(before, p.h.tensors[:4]))
    p.mapped.fill_(4)
    off, lens = torch.zeros(3, dtype=torch.int32, device="cuda"), i32([9, 9])
    capi().dflash_pages_map(p.h, 2, 0, None, None, i32([1, 1]), off, lens)
    with pytest.raises(capi().DFlashError) as e:
        capi().dflash_status_check(p.status)
    assert e.value.status == 5 and lens.tolist() == [0, 0] and p.table.eq(-1).all()


@pytest.mark.parametrize("n_rows", [4096, 4097])
def test_both_forms_of_the_rows_maps(n_rows):
    p = Pool(64, 3, 40)
    p.map([2, 0], [5, 127], [2000, 2096], n_rows)
    q = Pool(64, 3, 40)  # some of the maps, and default ids and starts
    off, lens = torch.zeros(3, dtype=torch.int32, device="cuda"), i32([0, 0])
    slot = torch.zeros(n_rows, dtype=torch.int32, device="cuda")
    capi().dflash_pages_map(q.h, 2, n_rows, None, None, i32([2000, 2096]), off, lens, None, None, slot)
    want = q.o.map([0, 1], [0, 0], [2000, 2096], n_rows)
    assert slot.tolist() == [r[2] for r in want[2]]
    q.same()


@pytest.mark.parametrize("n_rows", [1023, 1024, 1025, 2049, 8193, 16385, 33000])
def test_rows_over_several_ctas(n_rows):
    """Empty and refused entries among long and short ones, and rows behind the last."""
    rng = np.random.default_rng(n_rows)
    B = 50
    counts = rng.integers(0, 2 * n_rows // B, B)
    counts[rng.permutation(B)[:20]] = 0
    counts[B // 2:B // 2 + 10] = rng.integers(0, 4, 10)
    start = rng.integers(0, 300, B)
    start[7] = -1
    p = Pool(sum(-(-(int(c) + 300) // PAGE) for c in counts), B, 2 * n_rows // B // PAGE + 5)
    p.map(rng.permutation(B).tolist(), start.tolist(), counts.tolist(), n_rows)


def test_ids_that_meet_in_a_table():
    """Ids whose multiples of the golden ratio lie together, some of them twice."""
    ids = [i for i in range(6000) if i * 2654435769 % 2 ** 32 < 2 ** 26][:40]
    assert len(ids) == 40
    p = Pool(100, 6000, 2)
    seqs = ids + [ids[3], ids[39]] + list(range(40, 60))
    p.map(seqs, [0] * len(seqs), [1 + i for i in range(len(seqs))])
    p.release(seqs[::-1], [0] * len(seqs))


def test_captured_and_replayed():
    p = Pool(64, 4, 8)
    seqs, start, counts = i32([1, 3]), i32([0, 0]), i32([16, 16])
    off, lens = i32([0, 0, 0]), i32([0, 0])
    slot = torch.zeros(32, dtype=torch.int32, device="cuda")
    p.map([0], [0], [1])  # (the kernels are loaded)
    p.release([0], [1])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        capi().dflash_pages_release(p.h, 2, seqs, start)
        capi().dflash_pages_map(p.h, 2, 32, seqs, start, counts, off, lens, None, None, slot)
    rng = np.random.default_rng(0)
    now = [0, 0]
    for _ in range(30):
        start.copy_(i32(now))
        g.replay()
        p.o.release([1, 3], now)
        want = p.o.map([1, 3], now, [16, 16], 32)
        assert lens.tolist() == want[1] and slot.tolist() == [r[2] for r in want[2]]
        p.same()
        now = [int(x) + int(rng.integers(1, 17)) for x in now]
    p.failed(set())
