"""Requests with more than 64 rows for a KV head and scales of the cache at either end of fp16: the
values of fp16 rows enter as they are, those of bf16 rows rounded by 2^-11 at most.

Tolerance, relative to size = sum p |v| of each output.  P is rounded to fp16: 2^-11 of it, or
2^-25 where the weight (at least its ratio to the row's largest) is below 2^-14, but never more
than the weight.  For bf16 rows the values of V are rounded by 2^-11 and those of K too, so that
scores are off by 2^-11 scale max sum |q||k|; with the float32 sums w = 2^-17 (E + 1) more (E: see
serving_common.check_attn), each relatively in the weights and in their sum.  Sums: 2^-22 of the
running size for each of the eight products of a 64-key step.  Then the output's own rounding."""
import numpy as np
import pytest
import torch

import free_block_sparse_predict_b200 as fb

from gpu_common import dev
from serving_common import AttnCase
from test_gpu_kv4_light_keys import refill

pytestmark = pytest.mark.gpu

TINY = 2.0 ** -24
LEAST = 2.0 ** -14      # weights from here on keep 11 bits


def check_pieces(case, scale=None, least=LEAST):
    """One request per case; see above.  least: the smallest weight with 11 bits."""
    got = case.run(scale=scale)
    torch.cuda.synchronize()
    assert fb.sparge_device_status(case.ws) == 0
    (o, lse), (wo, wl, size, err, keys, sums, many) = got, case.exact(scale=scale)
    assert bool(many.all())
    n, m, d = case.lens[0], case.news[0], case.q.shape[2]
    Hq, bf16 = case.q.shape[1], case.q.dtype is torch.bfloat16
    w = 2.0 ** -17 * (err + 1) + 2.0 ** -11 * sums
    k, v = (x.double().repeat_interleave(Hq // case.c.Hkv, 1) for x in (case.k, case.v))
    s = torch.einsum("ihd,nhd->ihn", case.q.double(), k) * (d ** -0.5 if scale is None else scale)
    see = torch.arange(n, device=dev())[None] <= (n - m + torch.arange(m, device=dev()))[:, None]
    s = s.masked_fill(~see[:, None], -np.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True))
    light = torch.where(p < least, p.clamp(max=least * 2.0 ** -11), torch.zeros_like(p))
    loose = torch.einsum("ihn,nhd->ihd", light, v.abs())
    tol = (2.0 ** -11 * (2 if bf16 else 1) + 2 * w + 8 * (keys / 64 + 2) * 2.0 ** -22)[..., None] * size
    tol = tol * (1 + 2.0 ** -8) + loose
    tol = tol + torch.finfo(o.dtype).eps / 2 * (wo.abs() + tol)
    if not bf16:
        tol = tol + 2.0 ** -25
    off = (o.double() - wo).abs()
    assert bool((off <= tol).all()), (float((off / tol).max()), float((off / size).max()))
    assert bool(((lse.double() - wl).abs() <= w + 2.0 ** -22 * wl.abs()).all())


def case_of(dtype, d, group, n=150, m=70, **kw):
    return AttnCase(fb, dev(), [n], [m], 2, 2, d, group, 16, dtype, **kw)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("d,group", [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128)])
def test_the_smallest_scales(d, group, dtype):
    """Scales that are odd multiples of 2^-24, 2^-24 itself among them: of V, whose rows all hold one
    value; then of K, with scores of a few units."""
    for steps in (1, 3, 5, 25, 1023):
        case = case_of(dtype, d, group)
        refill(case, case.k, torch.full((150, 2, d), 7 * steps * TINY, device=dev()))
        assert bool((case.v > 0).all())
        check_pieces(case)
    for kscale in (1e-6, 1e-5, 3e-4):
        case = case_of(dtype, d, group, q_scale=2e4, kscale=kscale)
        case.q.clamp_(-6e4, 6e4)                     # 3.3 deviations would be infinite in fp16
        check_pieces(case, scale=0.3 / (2e4 * kscale))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("vscale", [1e-6, 1e-5, 1e-4, 3e-4])
def test_small_values(vscale, dtype):
    case = case_of(dtype, 128, 32)
    g = torch.Generator(device=dev()).manual_seed(1)
    refill(case, case.k, vscale * (1 + 0.3 * torch.randn(150, 2, 128, generator=g, device=dev())))
    check_pieces(case)


@pytest.mark.parametrize("n", [150, 3000])
def test_large_and_small_scales_in_one_call(n):
    """Tokens whose scale is near the largest beside tokens whose scale is near the smallest: each keeps
    its own value, in K and in V."""
    g = torch.Generator(device=dev()).manual_seed(2)
    for dtype, top in ((torch.float16, 6e4), (torch.bfloat16, 1.1e5)):
        case = case_of(dtype, 128, 64, n=n, q_scale=1.0)
        k, v = (torch.randn(n, 2, 128, generator=g, device=dev()) for _ in "kv")
        large = torch.arange(n, device=dev()) % 7 == 3
        size = torch.where(large, top, 3e-6)[:, None, None]
        # K: scores of a few units from the large, next to none from the small
        refill(case, k.clamp(-1, 1) * size, case.v)
        check_pieces(case, scale=1e-5)
        # V: every row meets large values
        refill(case, torch.randn(n, 2, 128, generator=g, device=dev()), v.clamp(-1, 1) * size)
        check_pieces(case)
        # and none of them weighs anything
        case.q[..., 0] = 16.0
        k = torch.randn(n, 2, 128, generator=g, device=dev())
        k[..., 0] = torch.where(large, -40.0, 0.0)[:, None]
        refill(case, k, v.clamp(-1, 1) * size)
        check_pieces(case)
