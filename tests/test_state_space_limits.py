"""The state-space entry points on the CPU: operands a launch would read although no token does, and sizes that no launch
takes."""

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


# A launch takes fewer than 2^32 threads along its grid. These shapes need as many or more.

CONV = [((1 << 16, 1, 1 << 16), (1 << 17, 1 << 17, 2), 1), ((1 << 19, 1, 1 << 16), None, 8)]


@pytest.mark.parametrize("x,strides,channels", CONV)
def test_causal_conv_of_more_than_a_launch(lib, x, strides, channels):  # noqa: F811
    def call(x):
        return lib.sx_causal_conv(B.SX_BF16, _i64(x), _i64(strides), _at(0), 4, _at(8), None, None, None, 0, _at(16),
                                  None, None)

    assert call(x) == B.SX_E_UNSUPPORTED and b"launch" in lib.sx_last_error()
    # a thread takes `channels` channels
    assert x[0] * x[2] // channels == 1 << 32


def test_causal_conv_gradient_of_more_than_a_launch(lib):  # noqa: F811
    got = lib.sx_causal_conv_backward(B.SX_F32, _i64((1 << 18, 1, 1 << 16)), None, _at(0), 4, _at(30), None, None, None, 0,
                                      None, _at(8), None, _at(16), _at(32), None, None, _at(64), 1 << 50, None)
    assert got == B.SX_E_UNSUPPORTED and b"launch" in lib.sx_last_error()


@pytest.mark.parametrize("x,strides", [((1 << 16, 1 << 16), (1 << 17, 2)), ((1 << 19, 1 << 16), None)])
def test_causal_conv_step_of_more_than_a_launch(lib, x, strides):  # noqa: F811
    got = lib.sx_causal_conv_step(B.SX_BF16, _i64(x), _i64(strides), _at(0), 2, _at(30), None, 0, x[0], x[1], _at(8), None,
                                  _at(16), None)
    assert got == B.SX_E_UNSUPPORTED and b"launch" in lib.sx_last_error()


def test_selective_scan_of_more_than_a_launch(lib):  # noqa: F811
    x, b = (1 << 14, 1, 1 << 16), (1 << 14, 1, 1, 16)  # 2^30 channels of four waves' lanes
    got = lib.sx_selective_scan(B.SX_BF16, _i64(x), None, _at(0), None, _at(4), _at(40), _i64(b), None, _at(8), None,
                                _at(12), None, None, None, None, 1, None, None, _at(16), None, _at(64), 1 << 50, None)
    assert got == B.SX_E_UNSUPPORTED and b"launch" in lib.sx_last_error()


@pytest.mark.parametrize("x,b", [((1, 1 << 23, 16), (1, 1 << 23, 16, 16)),      # 2^27 rows of b of 32 values
                                 ((1, 1, 1 << 24), (1, 1, 1, 16))])             # 2^28 rates, 16 threads each
def test_selective_scan_gradient_of_more_than_a_launch(lib, x, b):  # noqa: F811
    at = [_at(i) for i in range(0, 64, 2)]
    got = lib.sx_selective_scan_backward(B.SX_BF16, _i64(x), None, at[0], None, at[1], at[2], _i64(b), None, at[3], None,
                                         at[4], None, None, None, None, 1, None, None, None, at[5], None, at[6], at[7],
                                         at[8], at[9], at[10], None, None, None, None, at[11], 1 << 50, None)
    assert got == B.SX_E_UNSUPPORTED and b"launch" in lib.sx_last_error()


@pytest.mark.parametrize("n,lanes", [(16, 2), (32, 4)])
def test_selective_scan_step_of_more_than_a_launch(lib, n, lanes):  # noqa: F811
    rows = (1 << 16) // lanes
    x, b = (rows, 1 << 16), (rows, 1, n)
    got = lib.sx_selective_scan_step(B.SX_BF16, _i64(x), None, _at(0), None, _at(4), _at(90), _i64(b), None, _at(8), None,
                                     _at(12), None, None, None, None, 1, rows, n << 16, _at(16), None, _at(80), None)
    assert got == B.SX_E_UNSUPPORTED and b"launch" in lib.sx_last_error()


@pytest.mark.parametrize("x,groups", [((1 << 24, 2, 16), 2),            # a workgroup a sample
                                      ((2, 1 << 24), 1 << 24)])         # groups of one channel: too many columns of a grid
def test_group_norm_of_more_than_a_launch(lib, x, groups):  # noqa: F811
    shape = (x[0], 1, x[1]) if len(x) == 2 else x
    for gradient in (False, True):
        if gradient:
            got = lib.sx_group_norm_backward(B.SX_F32, _i64(shape), None, _at(0), groups, None, None, 1e-5, 0, None, _at(1),
                                             _at(2), None, None, _at(4), 1 << 50, None)
        else:
            got = lib.sx_group_norm(B.SX_F32, _i64(shape), None, _at(0), groups, None, None, 1e-5, 0, _at(2), _at(4),
                                    1 << 50, None)
        assert got == B.SX_E_UNSUPPORTED and b"launch" in lib.sx_last_error()
