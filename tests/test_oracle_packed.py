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
