"""Sequences that several entries of a call name: the first entry alone counts, refused or not."""
import pytest

from test_gpu_pages import Pool

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seqs,keep", [
    ([2, 2], [-1, 0]), ([2, 3, 2], [-1, 0, 0]), ([2, 3, 2], [0, -1, 128]), ([9, 2, -1, 2, 9], [0, -5, 0, 1, 0]),
    ([3, 3, 2, 2], [200, 0, -2 ** 31, 2 ** 31 - 1]),
])
def test_release(seqs, keep):
    p = Pool(8, 4, 2)
    p.map([2, 3], [0, 0], [200, 200])
    p.release(seqs, keep)


@pytest.mark.parametrize("seqs,start,counts", [
    ([2, 2], [-1, 0], [5, 5]), ([2, 3, 2], [0, 0, 0], [-5, 5, 5]), ([2, 2, 3], [0, 0, 0], [1000, 5, 5]),
    ([9, 2, 9, 2], [0, 0, 0, 0], [3, 4, 5, 6]),
])
def test_map(seqs, start, counts):
    p = Pool(8, 4, 2)
    p.map(seqs, start, counts, 2000)
