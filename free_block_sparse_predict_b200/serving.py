"""Binding of the entry points around the prompt pass (include/sparge.h): rotary
positions with several axes, the bookkeeping of a paged cache, the cache in 4 bits and the
attention over it.

As in the package's main module, every ``sparge_*`` function has the name of the
C entry point it wraps and only checks and marshals arguments; a call runs on the
device that owns its tensors, on that device's current stream unless one is given.
"""
from __future__ import annotations

import ctypes
import struct
from typing import NamedTuple, Optional

import torch

from ._native import (SPARGE_BF16, SPARGE_F16, SPARGE_F32, SpargeError, SpargeKv4, SpargeKv4Attn,
                      SpargeRope, lib)

__all__ = ["Rope", "rope_frequencies", "grid_positions", "sparge_rope_apply",
           "sparge_rope_inverse", "sparge_kv_plan", "SpargeKv4", "make_kv4", "kv4_cache",
           "sparge_kv4_bytes", "sparge_kv4_append", "sparge_kv4_read",
           "sparge_kv4_workspace_bytes", "kv4_workspace", "sparge_kv4_attn"]

_DT = {torch.float16: SPARGE_F16, torch.bfloat16: SPARGE_BF16, torch.float32: SPARGE_F32}
_I32, _F32, _F64, _U8 = torch.int32, torch.float32, torch.float64, torch.uint8

# A single token's kernels run for microseconds, so these functions stay short: parameter
# structs are packed in one step (the C layout of SpargeRope and SpargeKv4Attn), tensors are
# checked by the cheapest accessors.
_ROPE = struct.Struct("@8i7q")
_ATTN = struct.Struct("@7ifiq")
assert _ROPE.size == ctypes.sizeof(SpargeRope) and _ATTN.size == ctypes.sizeof(SpargeKv4Attn)


def _bad(msg: str) -> SpargeError:
    return SpargeError(1, msg)


def _raise(code: int) -> None:
    raise SpargeError(code, lib().sparge_status_string(code).decode())


def _stream(stream, device: int) -> int:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _device(t: torch.Tensor, name: str) -> int:
    """Number of the CUDA device that owns t."""
    dev = t.get_device()
    if dev < 0 or not t.is_cuda:
        raise _bad(f"{name}: expected a CUDA tensor")
    return dev


def _flat(t, name: str, numel: int, dtype, device: int) -> int:
    """Address of a contiguous tensor of at least numel elements of dtype on the device."""
    if (t.dtype is dtype and t.get_device() == device and t.is_contiguous()
            and t.numel() >= numel):
        return t.data_ptr()
    if t.get_device() != device:
        raise _bad(f"{name}: expected a tensor on cuda:{device}, got {t.device}")
    if t.dtype is not dtype:
        raise _bad(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise _bad(f"{name}: expected a contiguous tensor")
    raise _bad(f"{name}: needs {numel} elements, has {t.numel()}")


# ----------------------------------------------------------------------------
# rotary positions
# ----------------------------------------------------------------------------

class Rope(NamedTuple):
    """Rotary positions of one token sequence, as sparge_forward and SpargeGraph take them."""
    pos: torch.Tensor        # int32 [axes, N] or [B, axes, N]
    inv_freq: torch.Tensor   # float64 [pairs], radians per position
    axis: torch.Tensor       # int32 [pairs], the axis that turns each pair
    interleaved: bool = False


def rope_frequencies(pairs, theta: float = 1e4, joint: bool = False, device="cuda"):
    """(inv_freq, axis) for ``pairs[a]`` channel pairs turned by axis a, in that order.

    Each axis has the whole spectrum theta^(-i / pairs[a]); with ``joint`` one spectrum
    theta^(-i / sum(pairs)) runs through all axes' pairs."""
    total = sum(pairs)
    if joint:
        f = -torch.arange(total, dtype=torch.float64) / total
    else:
        f = torch.cat([-torch.arange(n, dtype=torch.float64) / max(n, 1) for n in pairs])
    axis = torch.cat([torch.full((n,), a, dtype=torch.int32) for a, n in enumerate(pairs)])
    return (theta ** f).to(device), axis.to(device)


def grid_positions(N: int, prefix_len: int, T: int, Hg: int, Wg: int, device="cuda"):
    """Positions [3, N] (time, height, width) of a sequence with a T x Hg x Wg token grid
    behind prefix_len text tokens: text counts up on all axes at once, the grid's axes start
    where the text ends, and what follows goes on from the grid's largest coordinate."""
    L = T * Hg * Wg
    if min(N, prefix_len) < 0 or min(T, Hg, Wg) < 1 or prefix_len + L > N:
        raise _bad("the grid does not fit the sequence")
    pos = torch.empty((3, N), dtype=torch.int32)
    pos[:, :prefix_len] = torch.arange(prefix_len, dtype=torch.int32)
    g = torch.stack(torch.meshgrid(*(torch.arange(n, dtype=torch.int32) for n in (T, Hg, Wg)),
                                   indexing="ij"))
    pos[:, prefix_len:prefix_len + L] = prefix_len + g.reshape(3, L)
    rest = N - prefix_len - L
    pos[:, N - rest:] = prefix_len + max(T, Hg, Wg) + torch.arange(rest, dtype=torch.int32)
    return pos.to(device)


def _rope(inverse, x, y, pos, inv_freq, axis, perm, interleaved, stream):
    dev = _device(x, "x")
    shape, dtype = x.shape, x.dtype
    code = _DT.get(dtype)
    if len(shape) != 4 or shape != y.shape or y.dtype is not dtype or code is None:
        raise _bad("expected two [B, H, N, d] tensors of one shape and floating dtype")
    if y.get_device() != dev:
        raise _bad(f"y: expected a tensor on cuda:{dev}, got {y.device}")
    B, H, N, d = shape
    xb, xh, xn, xd = x.stride()
    yb, yh, yn, yd = y.stride()
    if d > 1 and (xd != 1 or yd != 1):
        raise _bad("the channels have to be contiguous")
    ps, pst = pos.shape, pos.stride()
    if len(ps) not in (2, 3) or ps[-1] != N or (len(ps) == 3 and ps[0] != B):
        raise _bad("pos: expected [axes, N] or [B, axes, N]")
    if pos.dtype is not _I32 or pos.get_device() != dev:
        raise _bad(f"pos: expected torch.int32 on cuda:{dev}")
    axes = ps[-2]
    if (N > 1 and pst[-1] != 1) or (axes > 1 and pst[-2] != N):
        raise _bad("pos: expected contiguous [axes, N] rows")
    pairs = inv_freq.numel()
    p = _ROPE.pack(B, H, N, d, 2 * pairs, axes, 1 if interleaved else 0, code, xb, xh, xn,
                   yb, yh, yn, pst[0] if len(ps) == 3 else 0)
    f = _flat(inv_freq, "inv_freq", pairs, _F64, dev)
    ax = _flat(axis, "axis", pairs, _I32, dev)
    table = None if perm is None else _flat(perm, "perm", N, _I32, dev)
    if inverse:
        rc = lib().sparge_rope_inverse(p, y.data_ptr(), x.data_ptr(), pos.data_ptr(), f, ax, table,
                                       _stream(stream, dev))
    else:
        rc = lib().sparge_rope_apply(p, x.data_ptr(), y.data_ptr(), pos.data_ptr(), f, ax, table,
                                     _stream(stream, dev))
    if rc:
        _raise(rc)


def sparge_rope_apply(x, y, pos, inv_freq, axis, perm: Optional[torch.Tensor] = None,
                      interleaved: bool = False, stream=None) -> None:
    """y[b, h, p] = x[b, h, s] turned by the angles pos[b, axis, s] * inv_freq, s = perm[p].

    x, y: [B, H, N, d] of any strides (a transposed [B, N, H, d], some heads of a packed
    projection); y may be x.  Pairs behind len(inv_freq) stay as they are."""
    _rope(False, x, y, pos, inv_freq, axis, perm, interleaved, stream)


def sparge_rope_inverse(y, x, pos, inv_freq, axis, perm: Optional[torch.Tensor] = None,
                        interleaved: bool = False, stream=None) -> None:
    """x[b, h, s] = y[b, h, p] turned back: the inverse of sparge_rope_apply and its gradient."""
    _rope(True, x, y, pos, inv_freq, axis, perm, interleaved, stream)


# ----------------------------------------------------------------------------
# pages
# ----------------------------------------------------------------------------

def sparge_kv_plan(new_len, seq_len, block_table, free_pages, free_count, page_size: int,
                   seq_len_out, free_count_out, cu_new, slot_map, admitted, stream=None) -> None:
    """One step of a paged cache's bookkeeping; every tensor is int32.

    new_len, seq_len, seq_len_out, admitted [R]; block_table [R, max_pages]; free_pages
    [num_pages]; free_count, free_count_out [1]; cu_new [R + 1]; slot_map [max_tokens].
    seq_len_out may be seq_len and free_count_out may be free_count."""
    dev = _device(cu_new, "cu_new")
    if block_table.dim() != 2:
        raise _bad("block_table: expected [R, max_pages]")
    R, width = block_table.shape
    rc = lib().sparge_kv_plan(
        R, page_size, width, free_pages.numel(), slot_map.numel(),
        _flat(new_len, "new_len", R, _I32, dev), _flat(seq_len, "seq_len", R, _I32, dev),
        _flat(block_table, "block_table", 0, _I32, dev),
        _flat(free_pages, "free_pages", 0, _I32, dev), _flat(free_count, "free_count", 1, _I32, dev),
        _flat(seq_len_out, "seq_len_out", R, _I32, dev),
        _flat(free_count_out, "free_count_out", 1, _I32, dev),
        _flat(cu_new, "cu_new", R + 1, _I32, dev), _flat(slot_map, "slot_map", 0, _I32, dev),
        _flat(admitted, "admitted", R, _I32, dev), _stream(stream, dev))
    if rc:
        _raise(rc)


# ----------------------------------------------------------------------------
# the cache in 4 bits
# ----------------------------------------------------------------------------

def make_kv4(Hkv: int, d: int, group: int, page_size: int, num_pages: int) -> SpargeKv4:
    """Shape of a 4-bit cache: KV heads, channels, channels per scale, tokens per page, pages."""
    return SpargeKv4(Hkv, d, group, page_size, num_pages)


def sparge_kv4_bytes(c: SpargeKv4) -> int:
    return int(lib().sparge_kv4_bytes(ctypes.byref(c)))


def kv4_cache(c: SpargeKv4, device="cuda") -> torch.Tensor:
    """Memory for the cache: uint8 [num_pages, Hkv, page_size / 16, bytes of a 16-token tile]."""
    if sparge_kv4_bytes(c) == 0:
        raise _bad("invalid cache parameters")
    tile = 16 * (c.d + 4 * (c.d // c.group))
    return torch.empty((c.num_pages, c.Hkv, c.page_size // 16, tile), dtype=torch.uint8,
                       device=device)


_PAIR = struct.Struct("@2q").pack


def _rows(x, name, T, Hkv, d, dev):
    """Address and packed token / head strides of a [T, Hkv, d] tensor."""
    if x.get_device() != dev:
        raise _bad(f"{name}: expected a tensor on cuda:{dev}, got {x.device}")
    if x.shape != (T, Hkv, d):
        raise _bad(f"{name}: expected [{T}, {Hkv}, {d}], got {list(x.shape)}")
    st, sh, sd = x.stride()
    if sd != 1:
        raise _bad(f"{name}: the channels have to be contiguous")
    return x.data_ptr(), _PAIR(st, sh)


def _cache_ptr(c, cache, Hkv: int, d: int, dev: int) -> int:
    group = c.group
    if group <= 0:
        raise _bad("invalid cache parameters")
    need = c.num_pages * Hkv * c.page_size * (d + 4 * (d // group))
    if (cache.dtype is not _U8 or not cache.is_contiguous() or cache.numel() < need
            or cache.get_device() != dev):
        raise _bad(f"cache: expected {need} contiguous bytes on cuda:{dev}")
    return cache.data_ptr()


def sparge_kv4_append(c: SpargeKv4, k, v, slot_map, cache, status=None, stream=None) -> None:
    """Rows of k and v [T, Hkv, d] (any token and head strides) into the slots slot_map [T];
    slots outside the cache are skipped.  status: an int32 tensor, or a workspace, whose first
    word receives SPARGE_ERANGE (6) when a scale was saturated."""
    dev, T, Hkv, d = _device(cache, "cache"), slot_map.numel(), c.Hkv, c.d
    dtype = k.dtype
    if dtype not in _DT or v.dtype is not dtype:
        raise _bad(f"k, v: expected one floating dtype, got {dtype} and {v.dtype}")
    pk, sk = _rows(k, "k", T, Hkv, d, dev)
    pv, sv = _rows(v, "v", T, Hkv, d, dev)
    if status is not None:
        if status.get_device() != dev or status.numel() * status.element_size() < 4:
            raise _bad(f"status: expected 4 bytes on cuda:{dev}")
        status = status.data_ptr()
    rc = lib().sparge_kv4_append(ctypes.byref(c), T, pk, sk, pv, sv, _DT[dtype],
                                 _flat(slot_map, "slot_map", T, _I32, dev),
                                 _cache_ptr(c, cache, Hkv, d, dev), status, _stream(stream, dev))
    if rc:
        _raise(rc)


def sparge_kv4_read(c: SpargeKv4, cache, slot_map, k, v, stream=None) -> None:
    """The values that the slots slot_map [T] hold, into rows of k and v [T, Hkv, d] (16-bit or
    float32; either may be None); rows whose slot is outside the cache stay as they were."""
    dev, T, Hkv, d = _device(cache, "cache"), slot_map.numel(), c.Hkv, c.d
    pk = pv = sk = sv = None
    first = k if k is not None else v
    if first is None:
        return
    dtype = first.dtype
    if dtype not in _DT or (v is not None and v.dtype is not dtype):
        raise _bad("k, v: expected one floating dtype")
    if k is not None:
        pk, sk = _rows(k, "k", T, Hkv, d, dev)
    if v is not None:
        pv, sv = _rows(v, "v", T, Hkv, d, dev)
    rc = lib().sparge_kv4_read(ctypes.byref(c), T, _cache_ptr(c, cache, Hkv, d, dev),
                               _flat(slot_map, "slot_map", T, _I32, dev), pk, sk, pv, sv,
                               _DT[dtype], _stream(stream, dev))
    if rc:
        _raise(rc)


# ----------------------------------------------------------------------------
# attention over the cache
# ----------------------------------------------------------------------------

def sparge_kv4_workspace_bytes(c: SpargeKv4, a: SpargeKv4Attn) -> int:
    return int(lib().sparge_kv4_workspace_bytes(ctypes.byref(c), ctypes.byref(a)))


def kv4_workspace(c: SpargeKv4, Hq: int, T: int, R: int, max_q: int, max_len: int,
                  device="cuda") -> torch.Tensor:
    """Workspace of sparge_kv4_attn for R requests of up to max_len tokens, T rows of q in all
    and up to max_q each: for a block table of ceil(max_len / page_size) columns, or with that
    max_len given to the call."""
    pages = -(-max_len // c.page_size) if c.page_size > 0 else 0
    a = SpargeKv4Attn(R, T, Hq, max_q, pages, max_len, 1, 1.0, SPARGE_F16, Hq * c.d)
    n = sparge_kv4_workspace_bytes(c, a)
    if n == 0:
        raise _bad("invalid parameters")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def sparge_kv4_attn(c: SpargeKv4, q, cache, block_table, seq_len, cu_q, max_q: int, o, ws,
                    scale: Optional[float] = None, causal: bool = True, lse=None,
                    max_len: int = 0, stream=None) -> None:
    """Attention of new tokens over the cache that holds them already.

    q [T, Hq, d] (any token stride), o [T, Hq, d], lse float32 [T, Hq] or None; block_table
    [R, max_pages], seq_len [R] and cu_q [R + 1] as sparge_kv_plan leaves them; max_q: most new
    tokens of a request; max_len: longest request (0: what the table holds); scale: 1/sqrt(d)
    unless given."""
    dev, shape, dtype, d = _device(q, "q"), q.shape, q.dtype, c.d
    if len(shape) != 3 or shape[2] != d or dtype not in _DT or dtype is _F32:
        raise _bad(f"q: expected [T, Hq, {d}] in 16 bits")
    T, Hq, _ = shape
    st, sh, sd = q.stride()
    if sd != 1 or (Hq > 1 and sh != d):
        raise _bad("q: heads and channels have to be contiguous")
    if o.shape != shape:
        raise _bad(f"o: expected {list(shape)}")
    if block_table.dim() != 2:
        raise _bad("block_table: expected [R, max_pages]")
    R, width = block_table.shape
    if ws.get_device() != dev or not ws.is_contiguous():
        raise _bad(f"ws: expected a contiguous tensor on cuda:{dev}")
    a = _ATTN.pack(R, T, Hq, max_q, width, max_len, 1 if causal else 0,
                   d ** -0.5 if scale is None else scale, _DT[dtype], st)
    rc = lib().sparge_kv4_attn(
        ctypes.byref(c), a, q.data_ptr(), _cache_ptr(c, cache, c.Hkv, d, dev),
        _flat(block_table, "block_table", 0, _I32, dev), _flat(seq_len, "seq_len", R, _I32, dev),
        _flat(cu_q, "cu_q", R + 1, _I32, dev), _flat(o, "o", 0, dtype, dev),
        None if lse is None else _flat(lse, "lse", T * Hq, _F32, dev), ws.data_ptr(),
        ws.numel() * ws.element_size(), _stream(stream, dev))
    if rc:
        _raise(rc)
