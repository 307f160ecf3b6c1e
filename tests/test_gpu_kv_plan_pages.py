"""Page numbers that are none (a table or a stack that holds something else): their slots never fall
on another page, so the cache's append skips them."""
import numpy as np
import pytest
import torch

from gpu_common import dev
from serving_common import PlanState, plan_oracle

import free_block_sparse_predict_b200 as fb

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens", [60, 40_000])      # one cluster of CTAs, a whole grid
@pytest.mark.parametrize("P", [1, 7, 16, 1024])
@pytest.mark.parametrize("near", [0, 2 ** 28, 2 ** 27, -2 ** 28, 2 ** 31 - 9, -2 ** 31, 2 ** 22])
def test_page_numbers_that_are_none(near, P, tokens):
    ids = np.clip(near + np.arange(40), -2 ** 31, 2 ** 31 - 1)
    table = np.full((3, 50), -1)
    table[:, 0] = ids[30:33]
    args = (np.array([5, 3 * P + 1, 20]), np.array([1, min(P, 3), 1]), table, ids[:30], 30, P)
    s = PlanState(*args, tokens, dev())
    s.call(fb)
    got, want = s.outputs(), plan_oracle(*args, tokens)
    fits = (want["slots"] >= -2 ** 31) & (want["slots"] < 2 ** 31)
    page_fits = fits & (want["slots"] // P * P + P <= 2 ** 31)
    for k in want:
        if k != "slots":
            assert np.array_equal(got[k], want[k]), k
    assert np.array_equal(got["slots"][page_fits], want["slots"][page_fits])
    assert (got["slots"][~fits] < 0).all()
