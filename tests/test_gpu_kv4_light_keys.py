"""Attention over the 4-bit cache where many light keys carry the answer: a few keys far above the
rest whose own values are near zero, at every size of V.

Tolerance, relative to size = sum p |v| of each output, without an absolute part for keys that the
kernel holds in full.  A weight p (at least its ratio to the row's largest) is held times 2^10 and
a scale s of V times 2^b, b = min(15, 3 - floor(log2 S)), S the largest scale of the KV head (a warp
that has met smaller ones only has a larger b); both, and their product, are rounded to fp16: 2^-11
each for p and the product where they are normal, s exactly.  Below, with codes of up to 7:
  p < 2^-24          off by 2^-35, o by 7 s 2^-35
  p s < 2^-(24 + b)  off by 2^-(35 + b), o by 7 2^-(35 + b)
  s < 2^-(14 + b)    off by 2^-(25 + b), o by 7 p 2^-(25 + b)
each in units of a sum of weights that is at least 1.  Scores are off by w = 2^-17 (E + 1),
relatively in the weight, in the sum of weights too (E: see serving_common.check_attn).  Sums:
2^-22 of the running size per step.  Then the output's own rounding."""
import numpy as np
import pytest
import torch

import free_block_sparse_predict_b200 as fb

from gpu_common import dev
from serving_common import AttnCase

pytestmark = pytest.mark.gpu


def refill(case, k, v):
    """Writes k, v [tokens, Hkv, d] in place of what the cache holds, and reads back what it keeps."""
    slots = torch.cat(case.slots)
    fb.sparge_kv4_append(case.c, k.to(case.q.dtype), v.to(case.q.dtype), slots, case.cache)
    fb.sparge_kv4_read(case.c, case.cache, slots, case.k, case.v)


def check_relative(case, got, scale=None):
    """One request per case; see above."""
    (o, lse), (wo, wl, size, err, keys, sums, many) = got, case.exact(scale=scale)
    n, m, d = case.lens[0], case.news[0], case.q.shape[2]
    Hq, group = case.q.shape[1], case.c.group
    scale = d ** -0.5 if scale is None else scale
    assert not bool(many.any())
    w = 2.0 ** -17 * (err + 1)
    # keys that a row holds in fewer bits: by how much each channel may be off
    k, v = (x.double().repeat_interleave(Hq // case.c.Hkv, 1) for x in (case.k, case.v))
    s = torch.einsum("ihd,nhd->ihn", case.q.double(), k) * scale
    see = torch.arange(n, device=dev())[None] <= (n - m + torch.arange(m, device=dev()))[:, None]
    s = s.masked_fill(~see[:, None], -np.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True))
    loose = torch.zeros_like(wo)
    for h in range(Hq):
        step = v[:, h].view(n, d // group, group).abs().amax(-1) / 7          # [n, groups]
        b = min(15, 3 - int(torch.floor(torch.log2(step.max()))))
        for i in range(m):
            q = p[i, h][:, None]
            part = 7 * 2.0 ** -35 * step * (q < 2.0 ** -24)
            part += 7 * 2.0 ** -(35 + b) * ((q * step < 2.0 ** -(24 + b)) & (step > 0))
            part += 7 * 2.0 ** -(25 + b) * q * ((step < 2.0 ** -(14 + b)) & (step > 0))
            loose[i, h] = part.sum(0).repeat_interleave(group)
    steps = (keys / 64 + 2).clamp(max=514)
    tol = (2.0 ** -10 + 2 * w + steps * 2.0 ** -22)[..., None] * size * (1 + 2.0 ** -8) + loose
    tol = tol + torch.finfo(o.dtype).eps / 2 * (wo.abs() + tol)
    if o.dtype is torch.float16:
        tol = tol + 2.0 ** -25
    off = (o.double() - wo).abs()
    assert bool((off <= tol).all()), (float((off / tol).max()), float((off / size).max()))
    tl = w + 2.0 ** -22 * wl.abs()
    assert bool(((lse.double() - wl).abs() <= tl).all())
    return float((off / size).max())


def heavy_case(n, m, Hq, Hkv, d, group, dtype, nats, vscale, every=32, left=0.0, seed=0):
    """m new tokens after n - m others; each `every`-th key stands `nats` above the rest, and its
    values are `left` times theirs."""
    case = AttnCase(fb, dev(), [n], [m], Hq, Hkv, d, group, 64, dtype, seed=seed, q_scale=0.5)
    g = torch.Generator(device=dev()).manual_seed(seed + 1)
    case.q[..., 0] = 8.0
    k, v = (torch.randn(n, Hkv, d, generator=g, device=dev()) for _ in "kv")
    v = vscale * (v + 0.5)
    heavy = torch.arange(n, device=dev()) % every == 5
    k[..., 0] = 0.0
    k[heavy, :, 0] = nats * d ** 0.5 / 8.0
    v[heavy] *= left
    refill(case, k, v)
    return case


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("vscale", [1.0, 0.1, 0.02, 0.002, 0.0001])
@pytest.mark.parametrize("nats", [0.0, 8.0, 12.0, 14.0])
def test_light_keys_count_whatever_the_size_of_v(nats, vscale, dtype):
    """A heavy key in every 32, so that each warp has one from its first step on."""
    check_relative(*run(heavy_case(8192, 1, 8, 2, 128, 32, dtype, nats, vscale)))
    check_relative(*run(heavy_case(1009, 3, 6, 2, 64, 64, dtype, nats, vscale, left=1e-3)))


@pytest.mark.parametrize("vscale", [1.0, 0.1, 0.02, 0.002])
@pytest.mark.parametrize("nats,every", [(8.0, 1024), (12.0, 1024), (14.0, 64)])
def test_light_keys_of_a_long_context(nats, every, vscale):
    check_relative(*run(heavy_case(131072, 1, 8, 2, 128, 32, torch.bfloat16, nats, vscale, every=every,
                                   left=0.02)))
    check_relative(*run(heavy_case(131072, 2, 4, 2, 128, 128, torch.bfloat16, nats, vscale, every=every)))


def test_sizes_of_v_that_grow_and_shrink_along_the_keys():
    """The largest scale met so far sets the operands' size: it may come last, or first."""
    for last in (True, False):
        case = heavy_case(4000, 1, 4, 1, 128, 64, torch.bfloat16, 0.0, 1.0)
        g = torch.Generator(device=dev()).manual_seed(3)
        size = torch.logspace(-3, 2, 4000, device=dev())
        v = torch.randn(4000, 1, 128, generator=g, device=dev()) * (size if last else size.flip(0))[:, None, None]
        refill(case, case.k, v)
        check_relative(*run(case))


def run(case, **kw):
    got = case.run(**kw)
    torch.cuda.synchronize()
    assert fb.sparge_device_status(case.ws) == 0
    return case, got
