"""The state-space entry points on the CPU: operands a launch would read although no token does."""

import pytest

from scan_primitives_amd import _binding as B
from tests.test_state_space_boundary import FAKE, _i64, lib  # noqa: F401


def _at(i):
    return FAKE + (i << 40)  # far enough apart for the operands of the largest shapes


@pytest.mark.parametrize("weight,last,code", [(None, _at(4), B.SX_E_DIM_003), (None, None, B.SX_OK)])
def test_causal_conv_of_no_tokens(lib, weight, last, code):  # noqa: F811
    got = lib.sx_causal_conv(B.SX_F32, _i64((2, 0, 64)), None, None, 4, weight, None, None, None, 0, None, last, None)
    assert got == code, lib.sx_last_error()


@pytest.mark.parametrize("a,last,code", [(None, _at(4), B.SX_E_DIM_003), (None, None, B.SX_OK)])
def test_selective_scan_of_no_tokens(lib, a, last, code):  # noqa: F811
    got = lib.sx_selective_scan(B.SX_F32, _i64((2, 0, 64)), None, None, None, None, a, _i64((2, 0, 1, 16)), None, None,
                                None, None, None, None, None, None, 1, None, None, None, last, None, 0, None)
    assert got == code, lib.sx_last_error()


def test_gradients_of_no_tokens(lib):  # noqa: F811
    got = lib.sx_causal_conv_backward(B.SX_F32, _i64((2, 0, 64)), None, None, 4, None, None, None, None, 0, None, None,
                                      None, None, _at(1), None, None, _at(2), 1 << 30, None)
    assert got == B.SX_E_DIM_003
    got = lib.sx_selective_scan_backward(B.SX_F32, _i64((2, 0, 64)), None, None, None, None, None, _i64((2, 0, 1, 16)),
                                         None, None, None, None, None, None, None, None, 1, None, None, None, None, None,
                                         None, None, _at(1), None, None, None, None, None, None, _at(2), 1 << 40, None)
    assert got == B.SX_E_DIM_003
