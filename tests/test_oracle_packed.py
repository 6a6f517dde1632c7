"""The oracle of the calls over packed batches against what the header says of them."""
import numpy as np
import pytest

from oracle import packed as op


@pytest.mark.parametrize("x", [[np.nan], [np.inf], [np.nan, -np.inf, -np.inf], [1.0, np.inf, -np.inf],
                               [0.0, 1.0, np.nan], [np.inf, np.nan]])
@pytest.mark.parametrize("token", [0, 7])
def test_rows_with_nan_or_infinity_have_no_numbers(x, token):
    lp, entropy, ids, best = op.logprobs(x, token, 4)
    assert np.isnan([lp, entropy]).all() and np.isnan(best).all() and len(best) == len(ids) == 4


def test_a_release_refuses_what_an_earlier_entry_names():
    """Also where that entry was refused itself."""
    p = op.Pages(8, 4, 2)
    p.map([2, 3], [0, 0], [200, 200], 400)
    table, free = [list(t) for t in p.table], list(p.free)
    assert p.release([2, 2], [-1, 0]) == {"check"}
    assert p.table == table and p.free == free and p.mapped == [0, 0, 2, 2]
    assert p.release([2, 3, 2], [-1, 0, 0]) == {"check"}
    assert p.mapped == [0, 0, 2, 0] and p.table[2] == table[2]
