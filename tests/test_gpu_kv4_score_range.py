"""Scores far from zero: a row whose scores all lie below -1e30 (scales reach 2^100) is no row that
sees no key."""
import math

import pytest
import torch

import free_block_sparse_predict_b200 as fb

from gpu_common import dev
from serving_common import AttnCase
from test_gpu_kv4_light_keys import refill

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,m", [(40, 1), (20000, 1), (100, 70), (20000, 70)])
def test_rows_whose_scores_are_all_very_negative(n, m):
    """Keys of -1 under queries of 1: every score is -64 scale, all weights are alike, o is the mean
    of the values (2^-10 of them, weights being 1 and exact; values between 1 and 2) and lse the
    score itself, ln n being far below its last bit."""
    case = AttnCase(fb, dev(), [n], [m], 2, 1, 64, 64, 16, torch.bfloat16)
    g = torch.Generator(device=dev()).manual_seed(4)
    v = 1 + torch.rand(n, 1, 64, generator=g, device=dev())
    refill(case, torch.full((n, 1, 64), -1.0, device=dev()), v)
    case.q[:] = 1.0
    assert bool((case.k + 1).abs().max() < 2.0 ** -10)
    scale = 2.0 ** 100
    o, lse = case.run(scale=scale)
    torch.cuda.synchronize()
    assert fb.sparge_device_status(case.ws) == 0
    sums = case.v.double().cumsum(0)[n - m:, 0]
    want = sums / torch.arange(n - m + 1, n + 1, device=dev())[:, None]
    off = (o.double() - want[:, None]).abs()
    # steps of up to n / 8 sums of the same size round by 2^-22 each: 2^-10.7 for 20,000 keys
    assert bool((off <= (2.0 ** -8 + 2.0 ** -10 + 2.0 ** -10.7) * want[:, None]).all()), float(off.max())
    score = -64 * scale * float(-case.k.double().mean())
    # of 140 rows for the KV head K is rounded to fp16 in bf16 calls: 2^-11 of every product
    assert bool(((lse.double() - score).abs() <= (2.0 ** -18 + 2.0 ** -11 * (m > 32)) * math.fabs(score)).all())
