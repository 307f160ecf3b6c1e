"""The entry points around the prompt pass reject bad arguments on the host
before touching the GPU, and their host-side helpers give what they say.  No
GPU needed: no call here reaches a CUDA runtime function."""
import ctypes
import math

import pytest
import torch


@pytest.fixture(scope="module")
def native():
    from free_block_sparse_predict_b200 import build
    build.build()
    from free_block_sparse_predict_b200 import _native
    return _native


P = lambda x: ctypes.c_void_p(x)
FAR = [P(0x10000000 * (i + 1)) for i in range(16)]


# ----------------------------------------------------------------------------
# rotary positions
# ----------------------------------------------------------------------------

def _rope(native, **kw):
    a = dict(B=2, H=4, N=100, d=64, rot=64, axes=3, interleaved=0, dtype=1,
             x_stride=(25600, 6400, 64), y_stride=(25600, 6400, 64), pos_stride=0)
    a.update(kw)
    return native.SpargeRope(*a.values())


def _call(native, p, x=FAR[0], y=FAR[1], pos=FAR[2], f=FAR[3], ax=FAR[4], perm=None, inverse=False):
    L = native.lib()
    ref = ctypes.byref(p) if p is not None else None
    if inverse:
        return L.sparge_rope_inverse(ref, y, x, pos, f, ax, perm, None)
    return L.sparge_rope_apply(ref, x, y, pos, f, ax, perm, None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), 1), (dict(H=-1), 1), (dict(N=-2), 1), (dict(d=0), 1), (dict(axes=0), 1),
    (dict(rot=0), 1), (dict(rot=66), 1), (dict(rot=31), 1), (dict(interleaved=2), 1),
    (dict(dtype=3), 1), (dict(pos_stride=-1), 1),
    (dict(d=68, rot=64), 2),                                  # 136-byte rows
    (dict(rot=24), 2),                                        # 48 bytes turn: not two equal vectors
    (dict(x_stride=(25600, 6400, 68)), 2),                    # 136-byte steps
    (dict(x_stride=(25600, -6400, 64)), 1),
    (dict(y_stride=(25600, 0, 64)), 1),                       # heads written on top of one another
    (dict(y_stride=(25600, 6400, 32)), 1),                    # half rows shared
    (dict(y_stride=(6400, 6400, 64)), 1),                     # batch 1 on head 1
    (dict(x_stride=(1 << 57, 1 << 57, 1 << 57), N=1 << 20), 1),
])
def test_rope_refusals(native, kw, code):
    assert _call(native, _rope(native, **kw)) == code


def test_rope_inverse_checks_what_it_writes(native):
    shared = (25600, 0, 64)
    assert _call(native, _rope(native, x_stride=shared), inverse=True) == 1
    assert _call(native, _rope(native, y_stride=shared)) == 1


def test_rope_pointers_and_overlap(native):
    p = _rope(native)
    assert _call(native, None) == 1
    for name in ("x", "y", "pos", "f", "ax"):
        assert _call(native, p, **{name: None}) == 1
    assert _call(native, p, x=P(0x10000008)) == 1
    assert _call(native, p, f=P(0x10000004)) == 1
    assert _call(native, p, perm=P(0x10000002)) == 1
    n = 2 * 4 * 100 * 64 * 2
    assert _call(native, p, y=P(FAR[0].value + n - 16)) == 1            # the last row's end
    assert _call(native, p, x=FAR[0], y=FAR[0], perm=FAR[5]) == 1       # in place needs no table
    q = _rope(native, y_stride=(6400, 12800, 64))
    assert _call(native, q, x=FAR[0], y=FAR[0]) == 1                    # in place, other strides


@pytest.mark.parametrize("kw", [dict(B=0), dict(H=0), dict(N=0)])
def test_rope_of_nothing(native, kw):
    assert _call(native, _rope(native, **kw), x=None, y=None, pos=None) == 0


def test_rope_frequencies():
    from free_block_sparse_predict_b200 import rope_frequencies
    f, a = rope_frequencies((2, 3, 0, 1), theta=100.0, device="cpu")
    assert f.dtype == torch.float64 and a.dtype == torch.int32
    want = [1.0, 0.1, 1.0, 100 ** (-1 / 3), 100 ** (-2 / 3), 1.0]
    assert all(math.isclose(x, y, rel_tol=1e-14) for x, y in zip(f.tolist(), want))
    assert a.tolist() == [0, 0, 1, 1, 1, 3]
    f, _ = rope_frequencies((1, 3), theta=16.0, joint=True, device="cpu")
    assert all(math.isclose(x, y, rel_tol=1e-14) for x, y in zip(f.tolist(), [1, .5, .25, .125]))


def test_grid_positions():
    from free_block_sparse_predict_b200 import SpargeError, grid_positions
    p = grid_positions(2 + 2 * 3 * 4 + 3, 2, 2, 3, 4, device="cpu")
    assert p.shape == (3, 29) and p.dtype == torch.int32
    assert p[:, :2].tolist() == [[0, 1]] * 3
    assert p[:, 2].tolist() == [2, 2, 2] and p[:, 2 + 13].tolist() == [3, 2, 3]
    assert p[:, 25].tolist() == [3, 4, 5]
    assert p[:, 26:].tolist() == [[6, 7, 8]] * 3
    with pytest.raises(SpargeError):
        grid_positions(10, 3, 2, 2, 2, device="cpu")


# ----------------------------------------------------------------------------
# pages
# ----------------------------------------------------------------------------

def _plan(native, R=4, P=16, width=8, pages=100, tokens=50, ptrs=None, **swap):
    names = ["new", "len", "table", "free", "count", "len_out", "count_out", "cu", "slots", "adm"]
    a = dict(zip(names, ptrs or FAR))
    a.update(swap)
    return native.lib().sparge_kv_plan(R, P, width, pages, tokens, *[a[n] for n in names], None)


def test_plan_refusals(native):
    for kw in (dict(R=-1), dict(P=0), dict(width=-1), dict(pages=-1), dict(tokens=-1)):
        assert _plan(native, **kw) == 1
    assert _plan(native, R=4097) == 2
    assert _plan(native, pages=1 << 27) == 2 and _plan(native, width=1 << 27) == 2
    for name in ("new", "len", "table", "free", "count", "len_out", "count_out", "cu", "slots",
                 "adm"):
        assert _plan(native, **{name: None}) == 1, name
        assert _plan(native, **{name: P(0x90000002)}) == 1, name
    assert _plan(native, len_out=FAR[0]) == 1                     # over new_len
    assert _plan(native, adm=P(FAR[8].value + 4 * 49)) == 1       # over the last slot
    assert _plan(native, len_out=P(FAR[1].value + 4)) == 1        # beside itself


def test_plan_oracle_by_hand():
    """The reference the GPU tests use, on a step small enough to follow."""
    import numpy as np
    from serving_common import plan_oracle
    table = np.array([[5, -1], [6, 7], [-1, -1]])
    got = plan_oracle([1, -1, 3], [4, 8, 0], table, np.array([9, 8, 0, 0]), 1, 4, 6)
    # 6, 7 come back on top of 9; request 0 takes 7, request 2 takes 6
    assert got["free"].tolist() == [9, 6, 7, 0] and got["count"] == 1
    assert got["table"].tolist() == [[5, 7], [6, 7], [6, -1]]
    assert got["slots"].tolist() == [28, 24, 25, 26, -1, -1]
    assert got["cu"].tolist() == [0, 1, 1, 4] and got["length"].tolist() == [5, 0, 3]


# ----------------------------------------------------------------------------
# the 4-bit cache
# ----------------------------------------------------------------------------

def _kv4(native, **kw):
    a = dict(Hkv=2, d=64, group=32, page_size=16, num_pages=10)
    a.update(kw)
    return native.SpargeKv4(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(Hkv=0), 1), (dict(d=96), 2), (dict(group=16), 2), (dict(group=128), 1),
    (dict(page_size=0), 1), (dict(page_size=24), 1), (dict(num_pages=-1), 1),
    (dict(num_pages=1 << 28), 2), (dict(d=0), 1), (dict(Hkv=70000), 2)])
def test_cache_shapes_refused(native, kw, code):
    c = _kv4(native, **kw)
    L, two = native.lib(), (ctypes.c_int64 * 2)(128, 64)
    assert L.sparge_kv4_bytes(ctypes.byref(c)) == 0
    assert L.sparge_kv4_append(ctypes.byref(c), 3, FAR[0], two, FAR[1], two, 1, FAR[2], FAR[3], None,
                               None) == code
    assert L.sparge_kv4_read(ctypes.byref(c), 3, FAR[3], FAR[2], FAR[0], two, FAR[1], two, 1,
                             None) == code


def test_cache_bytes(native):
    L = native.lib()
    assert L.sparge_kv4_bytes(ctypes.byref(_kv4(native))) == 10 * 2 * 16 * (64 + 4 * 2)
    c = _kv4(native, d=128, group=128, page_size=64, Hkv=8)
    assert L.sparge_kv4_bytes(ctypes.byref(c)) == 10 * 8 * 64 * (128 + 4)
    assert L.sparge_kv4_bytes(None) == 0


def test_cache_pointers_and_strides(native):
    L, c = native.lib(), _kv4(native)
    S = lambda a, b: (ctypes.c_int64 * 2)(a, b)

    def append(T=3, k=FAR[0], ks=S(128, 64), v=FAR[1], vs=S(128, 64), dt=1, slots=FAR[2],
               cache=FAR[3], status=None):
        return L.sparge_kv4_append(ctypes.byref(c), T, k, ks, v, vs, dt, slots, cache, status, None)

    def read(T=3, k=FAR[0], ks=S(128, 64), v=FAR[1], vs=S(128, 64), dt=1, slots=FAR[2],
             cache=FAR[3]):
        return L.sparge_kv4_read(ctypes.byref(c), T, cache, slots, k, ks, v, vs, dt, None)

    assert append(T=-1) == 1 and append(T=0, k=None) == 0
    for f in (append, read):
        assert f(slots=None) == 1 and f(cache=None) == 1 and f(dt=5) == 1
        assert f(cache=P(0x10000008)) == 1 and f(slots=P(0x10000002)) == 1
        assert f(k=P(0x10000008)) == 1 and f(ks=S(-128, 64)) == 1 and f(ks=None) == 1
        assert f(ks=S(132, 64)) == 2
        assert f(k=FAR[3]) == 1                                   # inside the cache
    assert append(k=None) == 1 and append(dt=2) == 2
    assert append(status=P(0x50000002)) == 1
    assert append(slots=P(FAR[3].value + 64)) == 1
    assert read(k=None, v=None) == 0
    assert read(ks=S(0, 64)) == 1 and read(ks=S(128, 32)) == 1    # rows that overlap
    assert read(k=P(FAR[2].value - 128)) == 1                     # over the slots


# ----------------------------------------------------------------------------
# attention over the cache
# ----------------------------------------------------------------------------

def _attn(native, **kw):
    a = dict(R=3, T=6, Hq=4, max_q=2, max_pages=9, max_len=0, causal=1, scale=0.125, dtype=1, q_stride=256)
    a.update(kw)
    return native.SpargeKv4Attn(*a.values())


def _attn_call(native, c, a, ws_bytes=1 << 30, **swap):
    p = dict(zip(("q", "cache", "table", "lens", "cu", "o", "lse", "ws"), FAR))
    p.update(swap)
    return native.lib().sparge_kv4_attn(ctypes.byref(c), ctypes.byref(a) if a else None, p["q"], p["cache"],
                                        p["table"], p["lens"], p["cu"], p["o"], p["lse"], p["ws"], ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(R=-1), 1), (dict(T=-1), 1), (dict(Hq=0), 1), (dict(Hq=5), 1), (dict(max_q=-1), 1),
    (dict(max_pages=-1), 1), (dict(max_len=-1), 1), (dict(causal=2), 1), (dict(scale=0.0), 1),
    (dict(scale=float("inf")), 1), (dict(scale=1e31), 1), (dict(dtype=2), 1),
    (dict(q_stride=128), 1), (dict(q_stride=260), 2),
    (dict(R=70000), 2), (dict(max_pages=1 << 27), 2), (dict(T=1 << 30), 2),
    (dict(max_q=1 << 30), 2)])
def test_attention_parameters_refused(native, kw, code):
    c, a = _kv4(native), _attn(native, **kw)
    assert native.lib().sparge_kv4_workspace_bytes(ctypes.byref(c), ctypes.byref(a)) == 0
    assert _attn_call(native, c, a) == code


def test_attention_pointers_and_workspace(native):
    c, a = _kv4(native), _attn(native)
    need = native.lib().sparge_kv4_workspace_bytes(ctypes.byref(c), ctypes.byref(a))
    assert need >= 256
    assert _attn_call(native, c, None) == 1
    assert _attn_call(native, c, a, ws_bytes=need - 1) == 5
    for n in ("q", "cache", "table", "lens", "cu", "o", "ws"):
        assert _attn_call(native, c, a, **{n: None}) == 1, n
        assert _attn_call(native, c, a, **{n: P(0x90000002)}) == 1, n
    assert _attn_call(native, c, a, lse=P(0x90000002)) == 1
    assert _attn_call(native, c, a, o=FAR[0]) == 1                # over q
    assert _attn_call(native, c, a, lse=FAR[5]) == 1              # over o
    assert _attn_call(native, c, a, ws=FAR[1]) == 1               # inside the cache
    for kw in (dict(R=0), dict(T=0), dict(max_q=0)):
        assert _attn_call(native, c, _attn(native, **kw), q=None, o=None) == 0


def test_binding_refuses_before_the_library_is_called():
    """Host tensors, things that are no tensors, a cache without a shape: SpargeError each."""
    import free_block_sparse_predict_b200 as fb
    i, f = torch.zeros(4, dtype=torch.int32), torch.zeros(2, dtype=torch.float64)
    x = torch.zeros(1, 2, 4, 64)
    c, rows = fb.make_kv4(2, 64, 32, 16, 1), torch.zeros(4, 2, 64)
    memory, table = torch.zeros(4096, dtype=torch.uint8), torch.zeros(4, 1, dtype=torch.int32)
    calls = [lambda t: fb.sparge_rope_apply(t, x, i[None], f, i[:2]),
             lambda t: fb.sparge_rope_inverse(x, t, i[None], f, i[:2]),
             lambda t: fb.sparge_kv_plan(i, i, table, i, i, 16, i, i, t, i, i),
             lambda t: fb.sparge_kv4_append(c, rows, rows, i, t),
             lambda t: fb.sparge_kv4_read(c, t, i, rows, rows),
             lambda t: fb.sparge_kv4_attn(c, t, memory, table, i, i, 1, rows, memory)]
    for call in calls:
        for t in (x, None, 3):
            with pytest.raises(fb.SpargeError) as e:
                call(t)
            assert e.value.code == 1
