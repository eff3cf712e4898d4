"""The oracle's choices for whole blocks of tokens against those by sorting tuples (no GPU)."""

import numpy as np
import pytest

from oracle import memory_oracle as mo


@pytest.mark.parametrize("fn", ["sigmoid", "softmax"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("E,K,groups,top,gt", [
    (1, 1, 1, 1, 2), (12, 5, 3, 2, 2), (12, 8, 4, 3, 1), (32, 4, 32, 9, 2), (30, 12, 5, 5, 2)])
def test_choices_of_a_block_are_those_of_its_tokens(E, K, groups, top, gt, biased, fn):
    rng = np.random.default_rng(E + K)
    x = np.round(rng.standard_normal((60, E)) * 3) / 2  # many ties
    x[rng.random(x.shape) < 0.3] = -np.inf
    x[1] = -np.inf
    x[2, E // 2:] = np.nan
    if fn == "sigmoid":
        x[3, 0] = np.inf
    bias = np.round(rng.standard_normal(E) * 4) / 8 if biased else None
    args = (x, K, fn, bias, groups, top, gt)
    rows = [t for t in range(60) if not (fn == "softmax" and t == 2)]  # some K ids of NaN's row
    assert np.array_equal(mo.choose_rows(*args)[rows], mo.choose(*args)[rows])
