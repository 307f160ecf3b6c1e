"""The 4-bit cache, written and read: its bytes against the documented layout
and rounding rule, bit for bit, and the values read back."""
import numpy as np
import pytest
import torch

import free_block_sparse_predict_b200 as fb

from gpu_common import dev
from serving_common import MAX_SCALE, kv4_quantise, kv4_values, kv4_write

pytestmark = pytest.mark.gpu

SHAPES = [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128)]


def rows(T, H, d, dtype, seed=0, spread=3.0):
    g = torch.Generator(device=dev()).manual_seed(seed)
    size = torch.exp(spread * torch.randn(T, H, 1, generator=g, device=dev()))
    return (torch.randn(T, H, d, generator=g, device=dev()) * size).to(dtype)


def f32(x):
    return x.float().cpu().numpy()


def slots_of(n, total, seed=0):
    return torch.randperm(total, generator=torch.Generator().manual_seed(seed))[:n].int()


def check_bytes(c, cache, before, slots, k, v):
    kc, ks, _ = kv4_quantise(f32(k), c.group)
    vc, vs, _ = kv4_quantise(f32(v), c.group)
    want = before.cpu().numpy()
    for t, s in enumerate(slots.tolist()):
        if 0 <= s < c.num_pages * c.page_size:
            kv4_write(want, s, c.page_size, kc[t], ks[t], vc[t], vs[t])
    got = cache.cpu().numpy()
    # scales as fp16 values (a NaN has many bit patterns), codes as bytes
    a, b = (np.ascontiguousarray(x[..., 16 * c.d:]).view(np.float16) for x in (got, want))
    assert np.array_equal(a, b, equal_nan=True), np.argwhere(a != b)[:5]
    got, want = got[..., :16 * c.d], want[..., :16 * c.d]
    assert np.array_equal(got, want), np.argwhere(got != want)[:5]
    return (kc, ks), (vc, vs)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("d,group", SHAPES)
@pytest.mark.parametrize("Hkv,page,pages,T", [(1, 16, 1, 1), (3, 48, 5, 101), (8, 64, 3, 33)])
def test_bytes_and_values(Hkv, page, pages, T, d, group, dtype):
    c = fb.make_kv4(Hkv, d, group, page, pages)
    cache = fb.kv4_cache(c, dev())
    assert cache.numel() == fb.sparge_kv4_bytes(c)
    cache.copy_(torch.randint(0, 256, cache.shape, dtype=torch.uint8, device=dev()))
    before = cache.clone()
    k, v = rows(T, Hkv, d, dtype, 1), rows(T, Hkv, d, dtype, 2)
    slots = slots_of(T, page * pages)
    if T > 30:
        slots[::11], slots[5], slots[7] = -1, page * pages, 2 ** 31 - 1
    # three heads of a wider projection, token and head strides of their own
    kv = torch.zeros(T, 2 * Hkv + 1, 2 * d, dtype=dtype, device=dev())
    kv[:, :Hkv, :d], kv[:, Hkv + 1:, d:] = k, v
    fb.sparge_kv4_append(c, kv[:, :Hkv, :d], kv[:, Hkv + 1:, d:], slots.to(dev()), cache)
    coded = check_bytes(c, cache, before, slots, k, v)
    ok = ((slots >= 0) & (slots < page * pages)).numpy()
    for out in (dtype, torch.float32):
        got = [torch.full((T, Hkv, d), 9.0, dtype=out, device=dev()) for _ in "kv"]
        fb.sparge_kv4_read(c, cache, slots.to(dev()), *got)
        for x, (code, s) in zip(got, coded):
            want = torch.from_numpy(kv4_values(code, s)).to(dev()).to(out)
            assert torch.equal(x[ok], want[ok]) and bool((x[~ok] == 9).all())
    # K or V alone, into a [1, Hkv, T, d] tensor
    alone = torch.full((1, Hkv, T, d), 9.0, dtype=dtype, device=dev())
    fb.sparge_kv4_read(c, cache, slots.to(dev()), None, alone[0].transpose(0, 1))
    want = torch.from_numpy(kv4_values(*coded[1])).to(dev()).to(dtype)
    assert torch.equal(alone[0].transpose(0, 1)[ok], want[ok])


def test_values_are_within_half_a_step():
    """|x - value| <= s/2 for codes inside, and s is at most absmax/7 + half its own step: the
    code 7 may be off by 7 * 2^-11 s more where the scale was rounded down."""
    c = fb.make_kv4(2, 128, 32, 16, 8)
    cache, k = fb.kv4_cache(c, dev()), rows(100, 2, 128, torch.bfloat16, 3, spread=1.0)
    slots = slots_of(100, 128).to(dev())
    fb.sparge_kv4_append(c, k, k, slots, cache)
    got = [torch.empty(100, 2, 128, device=dev()) for _ in "kv"]
    fb.sparge_kv4_read(c, cache, slots, *got)
    s = (k.float().view(100, 2, 4, 32).abs().amax(-1, keepdim=True) / 7) * (1 + 2.0 ** -11)
    err = (got[0] - k.float()).view(100, 2, 4, 32).abs()
    assert bool((err <= s * (0.5 + 7 * 2.0 ** -11 + 2.0 ** -20)).all())
    assert torch.equal(got[0], got[1])


def test_special_values():
    c = fb.make_kv4(1, 64, 32, 16, 1)
    cache = torch.zeros_like(fb.kv4_cache(c, dev()))
    k = torch.zeros(8, 1, 64, dtype=torch.bfloat16, device=dev())
    k[1, 0, 3] = float("nan")                      # one group NaN, the other not
    k[1, 0, 40] = 3.0
    k[2, 0, 0], k[2, 0, 1] = float("inf"), -1e5    # saturated, the finite one keeps its value
    k[3, 0, 5], k[3, 0, 6] = 1e30, -float("inf")
    k[4] = 1e-6                                    # the scale is an fp16 subnormal
    k[5] = 1e-30                                   # the scale is 0
    k[6, 0, 0] = 7 * 16376.0                       # rounds to the largest scale
    k[7] = -0.0
    v = torch.full_like(k, 0.5)
    slots = torch.arange(8, dtype=torch.int32, device=dev())
    status = torch.zeros(64, dtype=torch.int32, device=dev())
    fb.sparge_kv4_append(c, k[4:], v[4:], slots[4:], cache, status)
    assert int(status[0]) == (6 if float(k[6, 0, 0]) / 7 > 16376 else 0)
    status.zero_()
    fb.sparge_kv4_append(c, k, v, slots, cache, status)
    assert int(status[0]) == 6 and int(status[1:].abs().sum()) == 0
    check_bytes(c, cache, torch.zeros_like(cache), slots, k, v)
    got = torch.empty(8, 1, 64, device=dev())
    fb.sparge_kv4_read(c, cache, slots, got, None)
    assert bool(got[1, 0, :32].isnan().all()) and bool(got[1, 0, 32:].isfinite().all())
    assert got[2, 0, 0].item() == 7 * float(MAX_SCALE) and got[3, 0, 6].item() == -7 * float(MAX_SCALE)
    assert bool((got[[0, 5, 7]] == 0).all())


def test_neighbours_keep_their_bytes():
    """Tokens written one call at a time, in any order, give what one call gives."""
    c = fb.make_kv4(2, 64, 64, 32, 2)
    k, v = rows(64, 2, 64, torch.float16, 4), rows(64, 2, 64, torch.float16, 5)
    slots = slots_of(64, 64, 6).to(dev())
    one, many = (torch.zeros_like(fb.kv4_cache(c, dev())) for _ in range(2))
    fb.sparge_kv4_append(c, k, v, slots, one)
    for t in slots_of(64, 64, 7).tolist():
        fb.sparge_kv4_append(c, k[t:t + 1], v[t:t + 1], slots[t:t + 1], many)
    assert torch.equal(one, many)


def test_one_slot_named_twice():
    c = fb.make_kv4(1, 128, 128, 16, 1)
    k, v = rows(2, 1, 128, torch.float16, 8), rows(2, 1, 128, torch.float16, 9)
    a, b, both = (torch.zeros_like(fb.kv4_cache(c, dev())) for _ in range(3))
    at = torch.full((2,), 11, dtype=torch.int32, device=dev())
    fb.sparge_kv4_append(c, k[:1], v[:1], at[:1], a)
    fb.sparge_kv4_append(c, k[1:], v[1:], at[1:], b)
    fb.sparge_kv4_append(c, k, v, at, both)
    assert bool(((both == a) | (both == b)).all())


def test_offsets_past_32_bits():
    """4.8 GB of cache: the last page, the first, and one behind 2^32 bytes."""
    c = fb.make_kv4(1, 128, 32, 1024, 1 << 15)
    cache = fb.kv4_cache(c, dev())
    assert cache.numel() > 2 ** 32
    n = c.num_pages * c.page_size
    slots = torch.tensor([0, n - 1, n - 16, 2 ** 32 // 144 + 5, 17, n], dtype=torch.int32, device=dev())
    k, v = rows(6, 1, 128, torch.bfloat16, 1), rows(6, 1, 128, torch.bfloat16, 2)
    fb.sparge_kv4_append(c, k, v, slots, cache)
    got = [torch.zeros(6, 1, 128, device=dev()) for _ in "kv"]
    fb.sparge_kv4_read(c, cache, slots, *got)
    for x, y in zip(got, (k, v)):
        want = torch.from_numpy(kv4_values(*kv4_quantise(f32(y), 32)[:2])).to(dev())
        want[5] = 0
        assert torch.equal(x, want)


def test_binding_refusals():
    c = fb.make_kv4(2, 64, 32, 16, 4)
    cache, slots = fb.kv4_cache(c, dev()), torch.arange(5, dtype=torch.int32, device=dev())
    k = torch.zeros(5, 2, 64, dtype=torch.float16, device=dev())
    good = dict(c=c, k=k, v=k, slot_map=slots, cache=cache)
    fb.sparge_kv4_append(**good)
    bad = [dict(k=k[:4]), dict(v=k.bfloat16()), dict(k=k.float(), v=k.float()), dict(v=k.cpu()),
           dict(k=k.transpose(1, 2).contiguous().transpose(1, 2)), dict(slot_map=slots.long()),
           dict(slot_map=slots.cpu()), dict(cache=cache[:3]), dict(cache=cache.cpu()),
           dict(cache=cache.view(torch.int8)), dict(c=fb.make_kv4(2, 96, 32, 16, 4)),
           dict(c=fb.make_kv4(2, 64, 128, 16, 4)), dict(c=fb.make_kv4(2, 64, 32, 24, 4)),
           dict(status=slots[:0])]
    for kw in bad:
        with pytest.raises(fb.SpargeError):
            fb.sparge_kv4_append(**{**good, **kw})
    wide = torch.zeros(5, 2, 68, dtype=torch.float16, device=dev())[:, :, :64]
    with pytest.raises(fb.SpargeError) as e:
        fb.sparge_kv4_append(**{**good, "k": wide})          # 136-byte steps
    assert e.value.code == 2
    one = torch.zeros(1, 2, 64, device=dev()).expand(5, 2, 64)
    with pytest.raises(fb.SpargeError):
        fb.sparge_kv4_read(c, cache, slots, one, None)       # five rows on top of one another
    with pytest.raises(fb.SpargeError):
        fb.sparge_kv4_read(c, cache, slots, k.double(), None)
