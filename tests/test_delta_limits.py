"""Calls of the gated delta rule that are refused for what their arguments share (CPU: before
anything is launched)."""
import ctypes

import pytest

from test_delta_ops_errors import D, INVALID, bwd, delta, fwd, lib  # noqa: F401 - lib: a fixture

STATES = 2 * 4 * 8 * 16 * 4  # bytes of the shape's states


@pytest.mark.parametrize("seqlen", [16, 1 << 20])
@pytest.mark.parametrize("first,last", [(4096, 4096), (4096, 4096 + STATES - 4), (4096 + STATES - 16, 4096)])
def test_states_must_not_overlap(lib, seqlen, first, last):  # noqa: F811
    """The segments of a long sequence run at once: its last state is written while the first
    one may still be read."""
    s, x, y = delta(seqlen=seqlen), ctypes.c_void_p(first), ctypes.c_void_p(last)
    assert fwd(lib, s, [D, D, D, D, None, D, D, x, None, D, y]) == INVALID
    assert bwd(lib, s, [D, D, D, D, None, D, D, D, None, D, x, D, D, D, D, D, None, None, y]) == INVALID


def test_states_side_by_side_are_no_overlap(lib):  # noqa: F811
    """(What is refused is the workspace.)"""
    s = delta()
    for first, last in ((4096, 4096 + STATES), (4096 + STATES, 4096)):
        x, y = ctypes.c_void_p(first), ctypes.c_void_p(last)
        assert fwd(lib, s, [D, D, D, D, None, D, D, x, None, D, y], ws=None) == 3
        assert bwd(lib, s, [D, D, D, D, None, D, D, D, None, D, x, D, D, D, D, D, None, None, y], ws=None) == 3
