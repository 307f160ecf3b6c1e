"""Binding of the entry points around the prompt pass (include/sparge.h): rotary
positions with several axes, the bookkeeping of a paged cache, the cache in 4 bits and the
attention over it.

As in the package's main module, every ``sparge_*`` function has the name of the
C entry point it wraps and only checks and marshals arguments (in C++, the extension module
``_serving``, since a single token's kernels run for microseconds); a call runs on the device
that owns its tensors, on that device's current stream unless one is given.
"""
from __future__ import annotations

import ctypes
import importlib
from typing import NamedTuple, Optional

import torch

from ._native import SPARGE_F16, SpargeError, SpargeKv4, SpargeKv4Attn, lib

__all__ = ["Rope", "rope_frequencies", "grid_positions", "sparge_rope_apply",
           "sparge_rope_inverse", "sparge_kv_plan", "SpargeKv4", "make_kv4", "kv4_cache",
           "sparge_kv4_bytes", "sparge_kv4_append", "sparge_kv4_read",
           "sparge_kv4_workspace_bytes", "kv4_workspace", "sparge_kv4_attn"]


def _entries():
    """Addresses of the C entry points, in the order in which the extension module keeps them."""
    L = lib()
    return tuple(ctypes.cast(f, ctypes.c_void_p).value for f in (
        L.sparge_rope_apply, L.sparge_rope_inverse, L.sparge_kv_plan, L.sparge_kv4_append,
        L.sparge_kv4_read, L.sparge_kv4_attn, L.sparge_status_string))


_serving = None


def _load():
    """The extension module; raises if it has not been built (no fallback exists)."""
    global _serving
    try:
        module = importlib.import_module("._serving", __package__)
    except ImportError as e:
        raise ImportError(f"_serving cannot be loaded ({e}); build it with "
                          "`python -m free_block_sparse_predict_b200.build`") from e
    if module.torch_version != str(torch.__version__):
        # it reads torch's objects by their layout
        raise ImportError(f"_serving was built for torch {module.torch_version}, this is "
                          f"{torch.__version__}; build it again with "
                          "`python -m free_block_sparse_predict_b200.build`")
    module.setup(SpargeError, torch._C._cuda_getCurrentRawStream, _entries)
    _serving = module
    return module


def _bad(msg: str) -> SpargeError:
    return SpargeError(1, msg)


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


def sparge_rope_apply(x, y, pos, inv_freq, axis, perm: Optional[torch.Tensor] = None,
                      interleaved: bool = False, stream=None) -> None:
    """y[b, h, p] = x[b, h, s] turned by the angles pos[b, axis, s] * inv_freq, s = perm[p].

    x, y: [B, H, N, d] of any strides (a transposed [B, N, H, d], some heads of a packed
    projection); y may be x.  Pairs behind len(inv_freq) stay as they are."""
    (_serving or _load()).rope(x, y, pos, inv_freq, axis, perm, interleaved, False, stream)


def sparge_rope_inverse(y, x, pos, inv_freq, axis, perm: Optional[torch.Tensor] = None,
                        interleaved: bool = False, stream=None) -> None:
    """x[b, h, s] = y[b, h, p] turned back: the inverse of sparge_rope_apply, and its gradient
    where perm names no row twice."""
    (_serving or _load()).rope(x, y, pos, inv_freq, axis, perm, interleaved, True, stream)


# ----------------------------------------------------------------------------
# pages
# ----------------------------------------------------------------------------

def sparge_kv_plan(new_len, seq_len, block_table, free_pages, free_count, page_size: int,
                   seq_len_out, free_count_out, cu_new, slot_map, admitted, stream=None) -> None:
    """One step of a paged cache's bookkeeping; every tensor is int32.

    new_len, seq_len, seq_len_out, admitted [R]; block_table [R, max_pages]; free_pages
    [num_pages]; free_count, free_count_out [1]; cu_new [R + 1]; slot_map [max_tokens].
    seq_len_out may be seq_len and free_count_out may be free_count."""
    (_serving or _load()).kv_plan(
        new_len, seq_len, block_table, free_pages, free_count, page_size, seq_len_out,
        free_count_out, cu_new, slot_map, admitted, stream)


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


def sparge_kv4_append(c: SpargeKv4, k, v, slot_map, cache, status=None, stream=None) -> None:
    """Rows of k and v [T, Hkv, d] (any token and head strides) into the slots slot_map [T];
    slots outside the cache are skipped.  status: an int32 tensor, or a workspace, whose first
    word receives SPARGE_ERANGE (6) when a scale was saturated."""
    (_serving or _load()).kv4_append(c, k, v, slot_map, cache, status, stream)


def sparge_kv4_read(c: SpargeKv4, cache, slot_map, k, v, stream=None) -> None:
    """The values that the slots slot_map [T] hold, into rows of k and v [T, Hkv, d] (16-bit or
    float32; either may be None); rows whose slot is outside the cache stay as they were."""
    (_serving or _load()).kv4_read(c, cache, slot_map, k, v, stream)


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
    (_serving or _load()).kv4_attn(c, q, cache, block_table, seq_len, cu_q, max_q, o, ws, scale,
                                   causal, lse, max_len, stream)
