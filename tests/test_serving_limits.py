"""Sizes at the end of 32 bits: refused on the host where an index of a kernel or a sum of a check
would pass it.  No GPU needed: no call here reaches a CUDA runtime function."""
import pytest

from test_serving_abi import _plan, native  # noqa: F401


@pytest.mark.parametrize("tokens", [2 ** 31 - 15, 2 ** 31 - 4, 2 ** 31 - 3, 2 ** 31 - 2, 2 ** 31 - 1])
def test_plan_refuses_slot_maps_whose_last_run_passes_32_bits(native, tokens):
    """The last four slots of the map start at up to tokens - 1, and their end is compared with it."""
    assert _plan(native, tokens=tokens) == 2
