"""Attention over the 4-bit cache against the definition in 64 bits, on the
values that the cache holds.  The tolerance is derived in serving_common."""
import numpy as np
import pytest
import torch

import free_block_sparse_predict_b200 as fb

from gpu_common import dev
from serving_common import AttnCase, check_attn

pytestmark = pytest.mark.gpu

SHAPES = [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128)]


def check(case, **kw):
    got = case.run(**kw)
    torch.cuda.synchronize()
    assert fb.sparge_device_status(case.ws) == 0
    check_attn(case, got, case.exact(kw.get("causal", True), kw.get("scale")))
    return got


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("d,group", SHAPES)
@pytest.mark.parametrize("Hq,Hkv", [(4, 4), (8, 2), (16, 2), (6, 1), (24, 2)])
def test_single_tokens(Hq, Hkv, d, group, dtype):
    check(AttnCase(fb, dev(), [1, 15, 16, 17, 63, 64, 65, 300, 1000], [1] * 9, Hq, Hkv, d, group, 16,
                   dtype, seed=Hq + d))


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,news,page", [
    ([5, 40, 129, 700], [5, 3, 1, 7], 16), ([33, 2048, 90], [33, 20, 64], 48),
    ([1, 2, 3], [1, 2, 3], 128), ([257], [257], 64), ([4097, 17], [9, 2], 256)])
def test_several_tokens(lens, news, page, causal):
    for d, group, Hq, Hkv in ((64, 64, 6, 2), (128, 32, 8, 2), (128, 128, 5, 5)):
        check(AttnCase(fb, dev(), lens, news, Hq, Hkv, d, group, page, torch.float16, seed=page, pad=3),
              causal=causal)


def test_long_context():
    """128K tokens: many chunks, joined."""
    check(AttnCase(fb, dev(), [131072, 100001], [1, 2], 8, 2, 128, 32, 64, torch.bfloat16))
    check(AttnCase(fb, dev(), [131073], [1], 4, 4, 64, 64, 16, torch.float16, q_scale=6.0))


def test_rows_that_see_nothing():
    """Requests without tokens in the cache, and more new tokens than the cache holds: the first
    of them stand before position 0."""
    case = AttnCase(fb, dev(), [0, 20, 3, 0], [2, 1, 5, 0], 4, 2, 64, 32, 16, torch.float16, pad=2)
    o, lse = check(case)
    assert bool((o[:2] == 0).all()) and bool((lse[:2] == -np.inf).all())
    assert bool((o[3:5] == 0).all()) and bool((lse[3:5] == -np.inf).all())
    check(case, causal=False)


def test_empty_calls():
    case = AttnCase(fb, dev(), [5, 9], [0, 0], 4, 2, 64, 32, 16, torch.float16, pad=3)
    check(case, max_q=4)
    fb.sparge_kv4_attn(case.c, case.q[:0], case.cache, case.table, case.lens_t, case.cu, 4,
                       torch.empty_like(case.q[:0]), case.ws)


@pytest.mark.parametrize("fill", ["stale", "nan"])
def test_unwritten_and_future_keys_do_not_reach_a_row(fill):
    """Memory behind the last token holds any bytes (scales that are NaN), and keys that a
    token may not see yet are NaN: no row that does not see them changes."""
    case = AttnCase(fb, dev(), [37, 130], [6, 9], 8, 2, 128, 64, 64, torch.float16, stale=fill == "stale")
    check(case)
    bad = torch.full((1, 2, 128), float("nan"), dtype=torch.float16, device=dev())
    fb.sparge_kv4_append(case.c, bad, bad, case.slots[0][-1:], case.cache)
    fb.sparge_kv4_append(case.c, bad, bad, case.slots[1][-2:-1], case.cache)
    want = case.exact()
    o, lse = case.run()
    nan_rows = [5, 6 + 7, 6 + 8]
    rest = [i for i in range(15) if i not in nan_rows]
    assert bool(o[nan_rows].isnan().all())
    case.T, case.pad = 15, 0
    keep = lambda x: x[rest]
    case.T = len(rest)
    check_attn(case, (keep(o), keep(lse)), tuple(keep(x) for x in want))


def test_extreme_sizes():
    """Large and small queries (one power of two a row), large values (p s near fp16's end), tiny
    values, and rows that are all zero."""
    for dtype, q_scale, kscale, vscale in ((torch.bfloat16, 3e5, 1e-6, 1.0), (torch.bfloat16, 1e-6, 1e3, 1.0),
                                           (torch.float16, 2.0, 1.0, 2e4), (torch.bfloat16, 2.0, 1.0, 2e4),
                                           (torch.float16, 2.0, 1.0, 0.02), (torch.float16, 0.0, 1.0, 1.0),
                                           (torch.float16, 60.0, 4.0, 1.0)):
        check(AttnCase(fb, dev(), [333, 50], [2, 1], 8, 2, 128, 32, 16, dtype, q_scale=q_scale,
                       kscale=kscale, vscale=vscale))


def test_one_key_gives_its_value():
    """A single key: weight 1, so the output is the value itself, rounded once."""
    case = AttnCase(fb, dev(), [1, 1, 1], [1, 1, 1], 4, 2, 128, 32, 16, torch.float16)
    o, lse = check(case)
    assert torch.equal(o, case.v.repeat_interleave(2, 1).half())


def test_scale_and_infinite_scores():
    case = AttnCase(fb, dev(), [200, 31], [1, 3], 4, 2, 64, 64, 16, torch.float16)
    check(case, scale=1.7)
    check(case, scale=1e-3)
    case.q[0, 0, 3] = float("inf")
    o, lse = case.run()
    assert bool(o[0, 0].isnan().all()) and bool(o[0, 1:].isfinite().all())


def test_bounds_larger_than_needed_and_max_len():
    case = AttnCase(fb, dev(), [70, 300, 9], [2, 1, 1], 8, 2, 64, 32, 16, torch.bfloat16)
    check(case, max_q=50)
    check(case, max_len=300)
    wide = torch.full((3, 5000), -1, dtype=torch.int32, device=dev())
    wide[:, :case.table.shape[1]] = case.table
    case.table = wide
    check(case)
    check(case, max_len=320)


def test_same_bits_every_time_and_on_any_stream():
    case = AttnCase(fb, dev(), [3000, 50, 1111], [1, 4, 2], 16, 4, 128, 64, 32, torch.bfloat16)
    o, lse = check(case)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = [case.run(stream=s) for s in (s1, s2, s1)]
    with torch.cuda.stream(s2):
        outs.append(case.run())
    torch.cuda.synchronize()
    for a, b in outs:
        assert torch.equal(a, o) and torch.equal(b, lse)


def test_inconsistent_device_data_stays_in_bounds():
    """Bad pages, lengths and offsets: reported, their keys left out, nothing else touched."""
    def fresh():
        return AttnCase(fb, dev(), [64, 40], [1, 2], 4, 2, 64, 64, 16, torch.float16)
    case = fresh()
    good, _ = case.run()
    case.table[0, 1] = 10 ** 6
    o, _ = case.run()
    assert fb.sparge_device_status(case.ws) == 1 and fb.sparge_device_status(case.ws) == 0
    assert torch.equal(o[1:], good[1:])
    keep = torch.cat([torch.arange(16), torch.arange(32, 64)]).to(dev())     # without the bad page
    case.k = torch.cat([case.k[:64][keep], case.k[64:]])
    case.v = torch.cat([case.v[:64][keep], case.v[64:]])
    case.lens = [48, 40]
    check_attn(case, (o, None), case.exact())
    case = fresh()
    case.lens_t[1] = 5000                       # longer than its table row
    o, _ = case.run()
    assert fb.sparge_device_status(case.ws) == 1 and torch.equal(o[0], good[0])
    case = fresh()
    case.lens_t[0] = -3
    o, lse = case.run()
    assert fb.sparge_device_status(case.ws) == 1 and bool((o[0] == 0).all())
    for cu in ([0, 9, 3], [-1, 1, 3], [0, 1, 4], [2, 1, 3]):
        case = fresh()
        case.cu = torch.tensor(cu, dtype=torch.int32, device=dev())
        case.run()
        assert fb.sparge_device_status(case.ws) == 1, cu


def test_captured_call_follows_its_buffers():
    """One graph over append and attention: lengths, tables and tokens change between replays."""
    case = AttnCase(fb, dev(), [100, 47], [1, 1], 8, 2, 128, 32, 16, torch.bfloat16)
    want = case.exact()
    o = torch.zeros(case.q.shape, dtype=case.q.dtype, device=dev())
    ws = fb.kv4_workspace(case.c, 8, 2, 2, 1, case.table.shape[1] * 16)
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    lens, table = case.lens_t.clone(), case.table.clone()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side, capture_error_mode="relaxed"):
        fb.sparge_kv4_attn(case.c, case.q, case.cache, table, lens, case.cu, 1, o, ws)
    g.replay()
    torch.cuda.synchronize()
    check_attn(case, (o, None), want)
    lens.copy_(torch.tensor([47, 100]))
    table.copy_(case.table.flip(0))
    g.replay()
    torch.cuda.synchronize()
    case.lens = [47, 100]
    case.k, case.v = (torch.cat([x[100:], x[:100]]) for x in (case.k, case.v))
    check_attn(case, (o, None), case.exact())
    assert fb.sparge_device_status(ws) == 0


def test_calls_of_different_shapes_share_a_workspace():
    """Large and small, one row tile and many: each leaves the workspace fit for the next."""
    cases = [AttnCase(fb, dev(), lens, news, 8, 2, 128, 32, 32, torch.bfloat16, seed=i) for i, (lens, news) in
             enumerate([([9000, 70], [1, 1]), ([70, 33, 40], [70, 33, 40]), ([5], [1]), ([2000] * 30, [1] * 30)])]
    need = [case.run() and case.ws.numel() for case in cases]
    ws = torch.zeros(max(need), dtype=torch.uint8, device=dev())
    for i in (0, 1, 2, 1, 0, 3, 2, 1, 3, 0):
        check(cases[i], ws=ws)


def test_cache_past_32_bits():
    """Pages that lie beyond 2^32 bytes."""
    c = fb.make_kv4(1, 128, 32, 1024, 1 << 15)
    case = AttnCase(fb, dev(), [1500], [1], 4, 1, 128, 32, 1024, torch.float16)
    big = fb.kv4_cache(c, dev())
    ids = torch.tensor([[c.num_pages - 1, c.num_pages - 70]], dtype=torch.int32, device=dev())
    for j in range(2):
        big[ids[0, j]] = case.cache[case.table[0, j]]
    want = case.exact()
    case.c, case.cache, case.table = c, big, ids
    check_attn(case, case.run(), want)


def test_binding_refusals():
    case = AttnCase(fb, dev(), [20, 30], [1, 1], 4, 2, 64, 32, 16, torch.float16)
    case.run()
    o = torch.empty(case.q.shape, dtype=torch.float16, device=dev())
    good = dict(c=case.c, q=case.q, cache=case.cache, block_table=case.table, seq_len=case.lens_t,
                cu_q=case.cu, max_q=1, o=o, ws=case.ws)
    fb.sparge_kv4_attn(**good)
    bad = [dict(q=case.q.float()), dict(q=case.q[:, :, :32]), dict(q=case.q.cpu()), dict(q=case.q[:, ::2]),
           dict(o=o[:1]), dict(o=o.bfloat16()), dict(o=o.cpu()), dict(block_table=case.table[0]),
           dict(block_table=case.table.long()), dict(block_table=case.table.t()), dict(seq_len=case.lens_t[:1]),
           dict(cu_q=case.cu[:2]), dict(cu_q=case.cu.long()), dict(ws=case.ws[:64]), dict(cache=case.cache[:1]),
           dict(scale=0.0), dict(scale=float("nan")), dict(scale=1e31), dict(max_q=-1), dict(lse=o), dict(ws=case.ws.cpu()),
           dict(q=case.q[:, :3], o=o[:, :3].contiguous()), dict(o=case.q.contiguous(), q=case.q.contiguous().view(2, 4, 64)[:, :4], seq_len=case.cu[:1])]
    for kw in bad:
        with pytest.raises(fb.SpargeError):
            fb.sparge_kv4_attn(**{**good, **kw})


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("d,group", SHAPES)
@pytest.mark.parametrize("lens,news,Hq,Hkv", [
    ([33], [33], 1, 1), ([64], [64], 1, 1), ([65], [65], 1, 1), ([1100], [1100], 1, 1),
    ([129, 64, 300], [129, 17, 257], 4, 2), ([2000, 63, 700, 5], [40, 1, 300, 5], 8, 1), ([9000], [70], 6, 2), ([1500, 1400], [513, 64], 5, 5)])
def test_pieces_of_prompts(lens, news, Hq, Hkv, d, group, dtype):
    """Many rows per request: one and two tiles of 128 rows, part tiles, units cut over CTAs, and
    requests with few rows in the same call."""
    for causal in (True, False):
        check(AttnCase(fb, dev(), lens, news, Hq, Hkv, d, group, 48, dtype, seed=sum(lens), pad=2), causal=causal)


def test_pieces_leave_unseen_keys_out():
    """As for few rows: NaN behind the last token, keys of the future that are NaN, a bad page."""
    case = AttnCase(fb, dev(), [200, 300], [70, 64], 4, 2, 64, 32, 16, torch.float16, stale=False)
    check(case)
    want = case.exact()
    bad = torch.full((1, 2, 64), float("nan"), dtype=torch.float16, device=dev())
    one = torch.ones_like(bad)
    fb.sparge_kv4_append(case.c, bad, one, case.slots[0][-1:], case.cache)      # K alone
    fb.sparge_kv4_append(case.c, one, bad, case.slots[1][-2:-1], case.cache)    # V alone
    o, lse = case.run()
    nan_rows = [69, 70 + 62, 70 + 63]
    rest = [i for i in range(134) if i not in nan_rows]
    assert bool(o[nan_rows].isnan().all())
    keep = lambda x: x[rest]
    case.T, case.pad = len(rest), 0
    check_attn(case, (keep(o), keep(lse)), tuple(keep(x) for x in want))


def test_pieces_with_extreme_values():
    for dtype, kscale, vscale in ((torch.bfloat16, 1.0, 1e5), (torch.bfloat16, 1e5, 1.0),
                                  (torch.float16, 1.0, 2e4), (torch.float16, 1.0, 0.02)):
        check(AttnCase(fb, dev(), [150], [100], 4, 2, 128, 64, 16, dtype, q_scale=2.0 / max(kscale, 1.0),
                       kscale=kscale, vscale=vscale))


def test_pieces_same_bits_and_counters():
    case = AttnCase(fb, dev(), [5000, 900], [90, 200], 8, 2, 128, 32, 64, torch.bfloat16)
    o, lse = check(case)
    for _ in range(3):
        a, b = case.run(ws=case.ws)
        torch.cuda.synchronize()
        assert torch.equal(a, o) and torch.equal(b, lse)
