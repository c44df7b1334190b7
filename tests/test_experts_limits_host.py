"""The experts' moves at the limit of tokens x choices < 2^31: checked before anything is launched."""
import ctypes

import pytest

from device_wide_prefix_tile_amd import experts, sequence as seq

OK, INVALID = 0, 1
MB = 1 << 20  # fake device addresses: without rows nothing touches them


@pytest.mark.parametrize("choices", [1, 2, 3, 7, 200, 255, 256])
def test_tokens_times_choices(choices):
    def call(tokens):
        a = experts._DispatchArgs(dtype=2, tokens=tokens, rows=0, choices=choices, channels=64, places=MB, x=MB, x_stride=64)
        return seq._lib().expert_dispatch(ctypes.byref(a), None)
    most = (2 ** 31 - 1) // choices
    assert call(most) == OK and call(most + 1) == INVALID
    assert call(2 ** 31) == INVALID and call(min(2 ** 64 // choices + 1, 2 ** 64 - 1)) == INVALID
