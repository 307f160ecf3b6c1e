"""Binding of the entry points around the prompt pass (include/sparge.h): rotary
positions with several axes, the bookkeeping of a paged cache, the cache in 4 bits and the
attention over it.

As in the package's main module, every ``sparge_*`` function has the name of the
C entry point it wraps and only checks and marshals arguments; a call runs on the
device that owns its tensors, on that device's current stream unless one is given.
"""
from __future__ import annotations

import ctypes
import math
from typing import NamedTuple, Optional

import torch

from ._native import (SPARGE_BF16, SPARGE_F16, SPARGE_F32, SpargeError, SpargeKv4, SpargeKv4Attn,
                      SpargeRope, lib)

__all__ = ["Rope", "rope_frequencies", "grid_positions", "sparge_rope_apply",
           "sparge_rope_inverse", "sparge_kv_plan", "SpargeKv4", "make_kv4", "kv4_cache",
           "sparge_kv4_bytes", "sparge_kv4_append", "sparge_kv4_read",
           "sparge_kv4_workspace_bytes", "kv4_workspace", "sparge_kv4_attn"]

_DT = {torch.float16: SPARGE_F16, torch.bfloat16: SPARGE_BF16, torch.float32: SPARGE_F32}


def _bad(msg: str) -> SpargeError:
    return SpargeError(1, msg)


def _check(code: int) -> None:
    if code != 0:
        raise SpargeError(code, lib().sparge_status_string(code).decode())


def _stream(stream, device) -> int:
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _device(t: torch.Tensor, name: str):
    if not t.is_cuda:
        raise _bad(f"{name}: expected a CUDA tensor")
    return t.device


def _flat(t, name: str, numel: int, dtype, device) -> int:
    """Address of a contiguous tensor of at least numel elements of dtype on device."""
    if t.device != device:
        raise _bad(f"{name}: expected a tensor on {device}, got {t.device}")
    if t.dtype != dtype:
        raise _bad(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise _bad(f"{name}: expected a contiguous tensor")
    if t.numel() < numel:
        raise _bad(f"{name}: needs {numel} elements, has {t.numel()}")
    return t.data_ptr()


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
    if x.dim() != 4 or x.shape != y.shape or x.dtype != y.dtype or x.dtype not in _DT:
        raise _bad("expected two [B, H, N, d] tensors of one shape and floating dtype")
    if y.device != dev:
        raise _bad(f"y: expected a tensor on {dev}, got {y.device}")
    B, H, N, d = x.shape
    sx, sy = x.stride(), y.stride()
    if d > 1 and (sx[3] != 1 or sy[3] != 1):
        raise _bad("the channels have to be contiguous")
    if pos.dim() not in (2, 3) or pos.shape[-1] != N or (pos.dim() == 3 and pos.shape[0] != B):
        raise _bad("pos: expected [axes, N] or [B, axes, N]")
    if pos.dtype != torch.int32 or pos.device != dev:
        raise _bad(f"pos: expected {torch.int32} on {dev}")
    axes, sp = pos.shape[-2], pos.stride()
    if (N > 1 and sp[-1] != 1) or (axes > 1 and sp[-2] != N):
        raise _bad("pos: expected contiguous [axes, N] rows")
    pairs = inv_freq.numel()
    p = SpargeRope(B, H, N, d, 2 * pairs, axes, int(interleaved), _DT[x.dtype],
                   (sx[0], sx[1], sx[2]), (sy[0], sy[1], sy[2]), sp[0] if pos.dim() == 3 else 0)
    args = (pos.data_ptr(), _flat(inv_freq, "inv_freq", pairs, torch.float64, dev),
            _flat(axis, "axis", pairs, torch.int32, dev),
            None if perm is None else _flat(perm, "perm", N, torch.int32, dev),
            _stream(stream, dev))
    if inverse:
        _check(lib().sparge_rope_inverse(ctypes.byref(p), y.data_ptr(), x.data_ptr(), *args))
    else:
        _check(lib().sparge_rope_apply(ctypes.byref(p), x.data_ptr(), y.data_ptr(), *args))


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
    (R, width), i32 = block_table.shape, torch.int32
    pages, tokens = free_pages.numel(), slot_map.numel()
    _check(lib().sparge_kv_plan(
        R, page_size, width, pages, tokens, _flat(new_len, "new_len", R, i32, dev),
        _flat(seq_len, "seq_len", R, i32, dev), _flat(block_table, "block_table", 0, i32, dev),
        _flat(free_pages, "free_pages", 0, i32, dev), _flat(free_count, "free_count", 1, i32, dev),
        _flat(seq_len_out, "seq_len_out", R, i32, dev),
        _flat(free_count_out, "free_count_out", 1, i32, dev),
        _flat(cu_new, "cu_new", R + 1, i32, dev), _flat(slot_map, "slot_map", 0, i32, dev),
        _flat(admitted, "admitted", R, i32, dev), _stream(stream, dev)))


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


_I64x2 = ctypes.c_int64 * 2


def _rows(x, name, c, T, dev, dtypes):
    """Address and token / head strides of a [T, Hkv, d] tensor."""
    if x.device != dev:
        raise _bad(f"{name}: expected a tensor on {dev}, got {x.device}")
    if x.dim() != 3 or tuple(x.shape) != (T, c.Hkv, c.d):
        raise _bad(f"{name}: expected [{T}, {c.Hkv}, {c.d}], got {list(x.shape)}")
    if x.dtype not in dtypes:
        raise _bad(f"{name}: got {x.dtype}")
    s = x.stride()
    if s[2] != 1:
        raise _bad(f"{name}: the channels have to be contiguous")
    return x.data_ptr(), _I64x2(s[0], s[1])


def _cache_ptr(c, cache) -> int:
    need = sparge_kv4_bytes(c)
    if need == 0 and c.num_pages != 0:
        raise _bad("invalid cache parameters")
    if cache.dtype != torch.uint8 or not cache.is_contiguous() or cache.numel() < need:
        raise _bad(f"cache: expected {need} contiguous bytes")
    return cache.data_ptr()


def sparge_kv4_append(c: SpargeKv4, k, v, slot_map, cache, status=None, stream=None) -> None:
    """Rows of k and v [T, Hkv, d] (any token and head strides) into the slots slot_map [T];
    slots outside the cache are skipped.  status: an int32 tensor, or a workspace, whose first
    word receives SPARGE_ERANGE (6) when a scale was saturated."""
    dev, T = _device(cache, "cache"), slot_map.numel()
    pc = _cache_ptr(c, cache)
    pk, sk = _rows(k, "k", c, T, dev, (torch.float16, torch.bfloat16))
    pv, sv = _rows(v, "v", c, T, dev, (k.dtype,))
    if status is not None:
        if status.device != dev or status.numel() * status.element_size() < 4:
            raise _bad(f"status: expected 4 bytes on {dev}")
        status = status.data_ptr()
    _check(lib().sparge_kv4_append(ctypes.byref(c), T, pk, sk, pv, sv, _DT[k.dtype],
                                   _flat(slot_map, "slot_map", T, torch.int32, dev), pc, status,
                                   _stream(stream, dev)))


def sparge_kv4_read(c: SpargeKv4, cache, slot_map, k, v, stream=None) -> None:
    """The values that the slots slot_map [T] hold, into rows of k and v [T, Hkv, d] (16-bit or
    float32; either may be None); rows whose slot is outside the cache stay as they were."""
    dev, T = _device(cache, "cache"), slot_map.numel()
    pc = _cache_ptr(c, cache)
    pk = pv = sk = sv = None
    first = k if k is not None else v
    if first is None:
        return
    if k is not None:
        pk, sk = _rows(k, "k", c, T, dev, _DT)
    if v is not None:
        pv, sv = _rows(v, "v", c, T, dev, (first.dtype,) if first.dtype in _DT else ())
    _check(lib().sparge_kv4_read(ctypes.byref(c), T, pc,
                                 _flat(slot_map, "slot_map", T, torch.int32, dev), pk, sk, pv, sv,
                                 _DT[first.dtype], _stream(stream, dev)))


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
    dev = _device(q, "q")
    if q.dim() != 3 or q.dtype not in (torch.float16, torch.bfloat16) or q.shape[2] != c.d:
        raise _bad(f"q: expected [T, Hq, {c.d}] in 16 bits")
    T, Hq, d = q.shape
    sq = q.stride()
    if sq[2] != 1 or (Hq > 1 and sq[1] != d):
        raise _bad("q: heads and channels have to be contiguous")
    if o.shape != q.shape:
        raise _bad(f"o: expected {list(q.shape)}")
    if block_table.dim() != 2:
        raise _bad("block_table: expected [R, max_pages]")
    (R, width), i32 = block_table.shape, torch.int32
    if cache.device != dev or ws.device != dev or not ws.is_contiguous():
        raise _bad(f"cache, ws: expected contiguous tensors on {dev}")
    a = SpargeKv4Attn(R, T, Hq, max_q, width, max_len, int(causal),
                      1.0 / math.sqrt(d) if scale is None else scale, _DT[q.dtype], sq[0])
    _check(lib().sparge_kv4_attn(
        ctypes.byref(c), ctypes.byref(a), q.data_ptr(), _cache_ptr(c, cache),
        _flat(block_table, "block_table", 0, i32, dev), _flat(seq_len, "seq_len", R, i32, dev),
        _flat(cu_q, "cu_q", R + 1, i32, dev), _flat(o, "o", 0, q.dtype, dev),
        None if lse is None else _flat(lse, "lse", T * Hq, torch.float32, dev), ws.data_ptr(),
        ws.numel() * ws.element_size(), _stream(stream, dev)))
