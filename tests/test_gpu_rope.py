"""Rotary positions with several axes against the formula in 64 bits.

Tolerance.  With |u|, |v| the pair's inputs, the fraction of a turn is rounded
to float32 (an angle error of pi 2^-24), sincospi is within 2 ulp (2^-23 for
values up to 1), and two products and one sum round at 2^-24 each: below
(|u| + |v|) (pi + 2 + 2) 2^-24 < 2^-21 (|u| + |v|).  The result is then rounded
once: eps/2 of its value (2^-25 for fp16 below its normal range)."""
import numpy as np
import pytest
import torch

import free_block_sparse_predict_b200 as fb
from free_block_sparse_predict_b200.graph import SpargeGraph
from oracle import sparge_oracle as orc

from gpu_common import dev, params_for, to_dev, workload

pytestmark = pytest.mark.gpu


def exact(x, pos, inv_freq, axis, interleaved, inverse=False):
    """x [B, H, N, d] in float64 turned by the formula, and |u| + |v| of every channel."""
    x = x.double()
    n = inv_freq.numel()
    i = torch.arange(n, device=x.device)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
    pos = pos if pos.dim() == 3 else pos[None]
    ang = pos.double()[:, axis.long()] * inv_freq[None, :, None]            # [B, pairs, N]
    ang = ang.transpose(1, 2)[:, None] * (-1 if inverse else 1)
    y, size = x.clone(), torch.zeros_like(x)
    y[..., a] = x[..., a] * ang.cos() - x[..., b] * ang.sin()
    y[..., b] = x[..., a] * ang.sin() + x[..., b] * ang.cos()
    size[..., a] = size[..., b] = x[..., a].abs() + x[..., b].abs()
    return y, size


def check(got, want, size):
    tol = 2.0 ** -21 * size + torch.finfo(got.dtype).eps / 2 * want.abs()
    if got.dtype == torch.float16:
        tol = tol + 2.0 ** -25
    err = (got.double() - want).abs()
    assert bool((err <= tol).all()), float((err - tol).max())


def inputs(B, H, N, d, pairs, axes, dtype, far=100000, seed=0, batched=False):
    g = torch.Generator(device=dev()).manual_seed(seed)
    x = torch.randn(B, H, N, d, generator=g, device=dev()).to(dtype)
    pos = torch.randint(-50, far, (B, axes, N) if batched else (axes, N), generator=g,
                        device=dev()).int()
    share = [pairs // axes + (a < pairs % axes) for a in range(axes)]
    return x, pos, *fb.rope_frequencies(share, device=dev())


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,H,N,d,pairs,axes", [
    (1, 1, 1, 16, 8, 1), (2, 3, 77, 64, 32, 3), (1, 40, 5, 128, 64, 3), (3, 9, 130, 128, 32, 2),
    (1, 2, 1000, 80, 24, 4), (1, 33, 257, 256, 128, 1)])
def test_turns_and_turns_back(B, H, N, d, pairs, axes, interleaved, dtype):
    x, pos, f, ax = inputs(B, H, N, d, pairs, axes, dtype, seed=N, batched=B > 1)
    y = torch.full_like(x, 7)
    fb.sparge_rope_apply(x, y, pos, f, ax, interleaved=interleaved)
    check(y, *exact(x, pos, f, ax, interleaved))
    assert torch.equal(y[..., 2 * pairs:], x[..., 2 * pairs:])
    z = torch.full_like(x, 7)
    fb.sparge_rope_inverse(y, z, pos, f, ax, interleaved=interleaved)
    check(z, *exact(y, pos, f, ax, interleaved, inverse=True))


def test_far_positions_keep_their_angle():
    """Positions up to 2^30: the angle's own error (2^-23 of a turn, 2^-20.3 rad, by the
    documented bound) joins the tolerance."""
    x, _, f, ax = inputs(1, 2, 64, 64, 32, 1, torch.float32)
    pos = (2 ** 30 - torch.arange(64, device=dev())).int()[None]
    y = torch.empty_like(x)
    fb.sparge_rope_apply(x, y, pos, f, ax)
    # the angle's remainder in whole numbers, scaled by 2^80 (pi has 256 bits behind its point)
    pi = int("3243F6A8885A308D313198A2E03707344A4093822299F31D0082EFA98EC4E6C89", 16)
    period = (2 * pi << 80) >> 256
    frac = [[int(q) * round(float(w) * 2 ** 80) for w in f.tolist()] for q in pos[0].tolist()]
    ang = torch.tensor([[(v % period) / 2.0 ** 80 for v in row] for row in frac],
                       dtype=torch.float64, device=dev())
    u, v = x.double()[..., :32], x.double()[..., 32:]
    want = torch.cat([u * ang.cos() - v * ang.sin(), u * ang.sin() + v * ang.cos()], -1)
    size = torch.cat([u.abs() + v.abs()] * 2, -1)
    err = (y.double() - want).abs()
    assert bool((err <= (2.0 ** -21 + 2.0 ** -20.3) * size + 2.0 ** -24 * want.abs()).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_table_strides_and_untouched_rows(dtype):
    B, H, N, d = 2, 5, 203, 64
    packed = torch.randn(B, N, H + 3, d, device=dev()).to(dtype)
    x = packed[:, :, 1:1 + H].transpose(1, 2)                       # heads inside a projection
    _, pos, f, ax = inputs(B, H, N, d, 32, 3, dtype)
    perm_np = np.random.default_rng(0).permutation(N).astype(np.int32)
    perm_np[::9] = -1
    perm_np[4::31] = N + 2
    ok = torch.from_numpy((perm_np >= 0) & (perm_np < N)).to(dev())
    perm = torch.from_numpy(perm_np).to(dev())
    src = perm.clamp(0, N - 1).long()
    y = torch.full((B, H, N, d), 3.0, device=dev(), dtype=dtype)
    before = packed.clone()
    fb.sparge_rope_apply(x, y, pos, f, ax, perm=perm, interleaved=True)
    want, size = exact(x, pos, f, ax, True)
    check(y[:, :, ok], want[:, :, src][:, :, ok], size[:, :, src][:, :, ok])
    assert bool((y[:, :, ~ok] == 3).all()) and torch.equal(packed, before)
    # back into the heads of another packed tensor: nothing beside the named rows changes
    into = torch.full_like(packed, 5)
    fb.sparge_rope_inverse(y, into[:, :, 1:1 + H].transpose(1, 2), pos, f, ax, perm=perm,
                           interleaved=True)
    back, bsize = exact(y, pos[:, src], f, ax, True, inverse=True)
    z = into[:, :, 1:1 + H].transpose(1, 2)
    check(z[:, :, src[ok]], back[:, :, ok], bsize[:, :, ok])
    rest = torch.ones(N, dtype=torch.bool, device=dev())
    rest[src[ok]] = False
    assert bool((z[:, :, rest] == 5).all()) and bool((into[:, :, 0] == 5).all())
    assert bool((into[:, :, 1 + H:] == 5).all())


def test_in_place_and_broadcast_source():
    x, pos, f, ax = inputs(2, 6, 91, 128, 64, 3, torch.float16)
    want, size = exact(x, pos, f, ax, False)
    part = x.clone()
    fb.sparge_rope_apply(part, part, pos, f, ax)
    check(part, want, size)
    one = x[:1, :1].expand(2, 6, 91, 128)
    y = torch.empty_like(x)
    fb.sparge_rope_apply(one, y, pos, f, ax)
    check(y, *exact(one, pos, f, ax, False))
    with pytest.raises(fb.SpargeError):
        fb.sparge_rope_inverse(y, one, pos, f, ax)


def test_gradient_is_the_inverse():
    """<dy, R x> differentiated: the formula's gradient R^T dy, and differences of the call."""
    x, pos, f, ax = inputs(1, 2, 9, 32, 12, 2, torch.float32, far=50)
    dy = torch.randn_like(x)
    dx = torch.empty_like(x)
    fb.sparge_rope_inverse(dy, dx, pos, f, ax)
    leaf = x.double().requires_grad_()
    n = f.numel()
    ang = (pos.double()[ax.long()] * f[:, None]).t()
    u, v = leaf[..., :n], leaf[..., n:2 * n]
    out = torch.cat([u * ang.cos() - v * ang.sin(), u * ang.sin() + v * ang.cos(),
                     leaf[..., 2 * n:]], -1)
    grad, = torch.autograd.grad((out * dy.double()).sum(), leaf)
    check(dx, grad, exact(dy, pos, f, ax, False, inverse=True)[1])
    step, y0, y1 = 0.5, torch.empty_like(x), torch.empty_like(x)
    e = torch.zeros_like(x)
    e[0, 1, 4, 3] = step                                             # linear: any step is exact
    fb.sparge_rope_apply(x - e, y0, pos, f, ax)
    fb.sparge_rope_apply(x + e, y1, pos, f, ax)
    slope = float(((y1.double() - y0.double()) * dy.double()).sum()) / (2 * step)
    # each of the 2 * 32 values involved is within 2^-20 (|u| + |v| < 8, and its rounding)
    assert abs(slope - float(dx[0, 1, 4, 3])) <= 64 * 2.0 ** -18 * float(dy.abs().max())


def test_unknown_axis_does_not_turn():
    x, pos, f, ax = inputs(1, 2, 20, 64, 32, 2, torch.float32)
    ax = ax.clone()
    ax[3], ax[5] = -1, 2
    y = torch.empty_like(x)
    fb.sparge_rope_apply(x, y, pos, f, ax)
    for pair in (3, 5):
        assert torch.equal(y[..., [pair, pair + 32]], x[..., [pair, pair + 32]])


def test_two_streams_and_a_side_stream():
    x, pos, f, ax = inputs(1, 8, 4000, 64, 32, 3, torch.bfloat16)
    want, size = exact(x, pos, f, ax, False)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    ys = [torch.empty_like(x) for _ in range(2)]
    torch.cuda.synchronize()
    fb.sparge_rope_apply(x, ys[0], pos, f, ax, stream=s1)
    with torch.cuda.stream(s2):
        fb.sparge_rope_apply(x, ys[1], pos, f, ax)
    torch.cuda.synchronize()
    for y in ys:
        check(y, want, size)


def test_binding_refusals():
    x, pos, f, ax = inputs(2, 2, 10, 64, 32, 2, torch.bfloat16)
    y = torch.empty_like(x)
    bad = [
        dict(y=y[:, :1]), dict(y=y.float()), dict(y=y.cpu()), dict(x=x.cpu()),
        dict(x=x.transpose(2, 3).contiguous().transpose(2, 3)), dict(pos=pos[:, :9]),
        dict(pos=pos.long()), dict(pos=pos.t().contiguous().t()), dict(pos=pos[None].repeat(3, 1, 1)),
        dict(inv_freq=f.float()), dict(axis=ax[:-1]), dict(axis=ax.long()),
        dict(perm=torch.zeros(9, dtype=torch.int32, device=dev())),
        dict(inv_freq=f.cpu()), dict(pos=pos.cpu()),
    ]
    for kw in bad:
        args = dict(x=x, y=y, pos=pos, inv_freq=f, axis=ax)
        args.update(kw)
        with pytest.raises(fb.SpargeError):
            fb.sparge_rope_apply(**args)
    with pytest.raises(fb.SpargeError) as e:
        fb.sparge_rope_apply(x[..., :24], y[..., :24], pos, f[:12], ax[:12])   # 48 bytes turn
    assert e.value.code == 2


@pytest.mark.parametrize("name", ["image_dit", "llm_32k"])
def test_forward_and_graph_with_rope(name):
    """sparge_forward(rope=...) is the plain chain: turn, permute, forward, put back; and the
    captured path replays it bit for bit."""
    over = {"N": 2112, "Hq": 4, "Hkv": 2} if name == "llm_32k" else {"Hq": 2, "Hkv": 2}
    w, t = workload(name, **over)
    p = params_for(w, o_dtype={"f16": torch.float16, "bf16": torch.bfloat16}[w.dtype])
    q, k, v = (to_dev(t[x], w.dtype) for x in ("q", "k", "v"))
    pos = fb.grid_positions(w.N, w.prefix_len, *w.grid) if w.grid else \
        torch.arange(w.N, dtype=torch.int32, device=dev())[None]
    r = fb.Rope(pos, *fb.rope_frequencies((16, 24, 24) if w.grid else (64,)), False)
    perm = None
    if w.grid:
        perm = torch.from_numpy(orc.hilbert_permutation(w.N, w.prefix_len, *w.grid).astype(np.int32)).to(dev())
    qt, kt = torch.empty_like(q), torch.empty_like(k)
    fb.sparge_rope_apply(q, qt, *r[:3])
    fb.sparge_rope_apply(k, kt, *r[:3])
    o0, m0, _, c0 = fb.sparge_forward(p, qt, kt, v, perm=perm)
    strided = q.transpose(1, 2).contiguous().transpose(1, 2)
    o1, m1, _, c1 = fb.sparge_forward(p, strided, k, v, perm=perm, rope=r)
    assert torch.equal(m0, m1) and torch.equal(c0, c1) and torch.equal(o0, o1)
    g = SpargeGraph(p, grid=(w.prefix_len, *w.grid) if w.grid else None, device=dev(), rope=r)
    assert torch.equal(g.run(q, k, v), o0)
    assert fb.sparge_device_status(g.ws) == 0
