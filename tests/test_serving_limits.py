"""Sizes at the end of 32 bits: refused on the host where an index of a kernel or a sum of a check
would pass it.  No GPU needed: no call here reaches a CUDA runtime function."""
import ctypes

import pytest

from test_serving_abi import _attn, _attn_call, _kv4, _plan, native  # noqa: F401


@pytest.mark.parametrize("tokens", [2 ** 31 - 15, 2 ** 31 - 4, 2 ** 31 - 3, 2 ** 31 - 2, 2 ** 31 - 1])
def test_plan_refuses_slot_maps_whose_last_run_passes_32_bits(native, tokens):
    """The last four slots of the map start at up to tokens - 1, and their end is compared with it."""
    assert _plan(native, tokens=tokens) == 2


@pytest.mark.parametrize("T,stride", [(1 << 28, 1 << 40), (1 << 24, 1 << 36), (2, 1 << 60), (3, (1 << 63) - 8)])
def test_attention_refuses_strides_whose_extent_passes_62_bits(native, T, stride):
    c, a = _kv4(native), _attn(native, T=T, q_stride=stride)
    assert native.lib().sparge_kv4_workspace_bytes(ctypes.byref(c), ctypes.byref(a)) == 0
    assert _attn_call(native, c, a) == 1
