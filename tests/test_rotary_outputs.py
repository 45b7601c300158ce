"""Host side of the rotary calls' choice for tokens without a position, without a GPU."""
import ctypes

import pytest

from test_chunks import ROT, P, api, turn  # noqa: F401


@pytest.mark.parametrize("zeros", [-1, 4])
def test_zeros_out_of_range_are_refused(api, zeros):  # noqa: F811
    rc, msg = turn(api, zeros=zeros)
    assert rc == 1 and "zeros" in msg


def test_zeros_in_an_inputs_place_are_refused(api):  # noqa: F811
    g, h = P(1 << 21), P(1 << 22)
    for ptrs, zeros in (([g, g, None, g, g, h], 1), ([g, g, None, g, h, g], 2), ([g, g, None, g, g, g], 3)):
        rc, msg = turn(api, ptrs=ptrs, zeros=zeros)
        assert rc == 1 and "in its input's place" in msg
    assert ctypes.sizeof(api.RotaryShape(**ROT).c()) == 80
