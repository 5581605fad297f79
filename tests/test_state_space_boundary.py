"""The state-space entry points on the CPU: what the C ABI and the binding refuse before any device work."""

import pytest
import torch

import scan_primitives_amd as sx
from scan_primitives_amd import _binding as B

FAKE = 1 << 40
MB = 1 << 20


@pytest.fixture(scope="module")
def lib():
    return B.load_library()


def _i64(x):
    return None if x is None else B.i64_array(x)


def _at(i):
    return FAKE + i * 256 * MB


# ---------------------------------------------------------------- causal convolution

def _conv(lib, dtype=B.SX_BF16, x=(2, 130, 64), strides=None, taps=4, x_at=_at(0), w=_at(1), bias=_at(2), initial=None,
          lengths=None, act=1, out=_at(3), last=_at(4)):
    return lib.sx_causal_conv(dtype, _i64(x), _i64(strides), x_at, taps, w, bias, initial, lengths, act, out, last, None)


@pytest.mark.parametrize("kwargs,code", [
    (dict(dtype=7), B.SX_E_DIM_002),
    (dict(x=None), B.SX_E_DIM_001),
    (dict(x=(2, -1, 64)), B.SX_E_DIM_001),
    (dict(x=(2, 130, 0)), B.SX_E_DIM_001),
    (dict(x=(2, 130, 1 << 25)), B.SX_E_UNSUPPORTED),
    (dict(x=(1 << 30, 1 << 20, 64)), B.SX_E_UNSUPPORTED),
    (dict(taps=0), B.SX_E_DIM_001),
    (dict(taps=9), B.SX_E_UNSUPPORTED),
    (dict(act=2), B.SX_E_UNSUPPORTED),
    (dict(act=-1), B.SX_E_UNSUPPORTED),
    (dict(x_at=None), B.SX_E_DIM_003),
    (dict(w=None), B.SX_E_DIM_003),
    (dict(out=None), B.SX_E_DIM_003),
    (dict(out=_at(0) + 64), B.SX_E_ALIAS),
    (dict(out=_at(1)), B.SX_E_ALIAS),
    (dict(last=_at(3)), B.SX_E_ALIAS),
    (dict(last=_at(5), initial=_at(5)), B.SX_E_ALIAS),
    (dict(out=_at(3) + 8), B.SX_E_UNSUPPORTED),
    (dict(last=_at(4) + 2), B.SX_E_UNSUPPORTED),
])
def test_causal_conv_refuses(lib, kwargs, code):
    assert _conv(lib, **kwargs) == code, lib.sx_last_error()
    assert lib.sx_last_error()


def test_calls_of_nothing_are_no_ops(lib):
    assert _conv(lib, x=(0, 130, 64), x_at=None, out=None, last=None) == B.SX_OK
    assert _conv(lib, x=(2, 0, 64), x_at=None, out=None, last=None) == B.SX_OK
    assert _scan(lib, x=(0, 130, 64), b=(0, 130, 2, 16), x_at=None, out=None, last=None) == B.SX_OK
    assert _scan(lib, x=(2, 0, 64), b=(2, 0, 2, 16), x_at=None, out=None, last=None) == B.SX_OK
    assert _norm(lib, x=(0, 5, 64), x_at=None, out=None) == B.SX_OK
    assert _norm(lib, x=(5, 0, 64), x_at=None, out=None) == B.SX_OK
    assert _conv_step(lib, x=(0, 64), x_at=None, out=None) == B.SX_OK
    assert _scan_step(lib, x=(0, 64), b=(0, 2, 16), x_at=None, out=None) == B.SX_OK


def _conv_backward(lib, dtype=B.SX_F32, x=(2, 30, 64), taps=4, w=_at(1), go=_at(2), gs=None, initial=None, gx=_at(3),
                   gw=_at(4), gb=_at(5), gi=_at(6), ws=_at(7), ws_bytes=1 << 40, act=0):
    return lib.sx_causal_conv_backward(dtype, _i64(x), None, _at(0), taps, w, None, initial, None, act, None, go, gs, gx,
                                       gw, gb, gi, ws, ws_bytes, None)


@pytest.mark.parametrize("kwargs,code", [
    (dict(dtype=5), B.SX_E_DIM_002),
    (dict(taps=-1), B.SX_E_DIM_001),
    (dict(act=7), B.SX_E_UNSUPPORTED),
    (dict(w=None), B.SX_E_DIM_003),
    (dict(go=None), B.SX_E_DIM_003),
    (dict(gx=None), B.SX_E_DIM_003),
    (dict(gw=None), B.SX_E_DIM_003),
    (dict(gx=_at(2)), B.SX_E_ALIAS),
    (dict(gw=_at(3)), B.SX_E_ALIAS),
    (dict(gi=_at(8), gs=_at(8)), B.SX_E_ALIAS),
    (dict(gi=_at(8), initial=_at(8)), B.SX_E_ALIAS),
    (dict(gb=_at(5) + 4), B.SX_E_UNSUPPORTED),
    (dict(ws=None), B.SX_E_WORKSPACE),
    (dict(ws_bytes=64), B.SX_E_WORKSPACE),
    (dict(ws=_at(7) + 16), B.SX_E_WORKSPACE),
])
def test_causal_conv_backward_refuses(lib, kwargs, code):
    assert _conv_backward(lib, **kwargs) == code, lib.sx_last_error()


def _conv_step(lib, dtype=B.SX_BF16, x=(3, 64), taps=4, x_at=_at(0), w=_at(1), pool=8, stride=3 * 64, state=_at(2),
               slots=_at(3), out=_at(4), act=1):
    return lib.sx_causal_conv_step(dtype, _i64(x), None, x_at, taps, w, None, act, pool, stride, state, slots, out, None)


@pytest.mark.parametrize("kwargs,code", [
    (dict(dtype=3), B.SX_E_DIM_002),
    (dict(x=(3, 0)), B.SX_E_DIM_001),
    (dict(taps=12), B.SX_E_UNSUPPORTED),
    (dict(pool=-1), B.SX_E_DIM_001),
    (dict(pool=2, slots=None), B.SX_E_DIM_001),
    (dict(stride=3 * 64 - 1), B.SX_E_UNSUPPORTED),
    (dict(stride=0), B.SX_E_UNSUPPORTED),
    (dict(x_at=None), B.SX_E_DIM_003),
    (dict(w=None), B.SX_E_DIM_003),
    (dict(state=None), B.SX_E_DIM_003),
    (dict(out=None), B.SX_E_DIM_003),
    (dict(state=_at(0)), B.SX_E_ALIAS),
    (dict(state=_at(3)), B.SX_E_ALIAS),
    (dict(out=_at(2)), B.SX_E_ALIAS),
    (dict(out=_at(4) + 2), B.SX_E_UNSUPPORTED),
    (dict(state=_at(2) + 1), B.SX_E_UNSUPPORTED),
])
def test_causal_conv_step_refuses(lib, kwargs, code):
    assert _conv_step(lib, **kwargs) == code, lib.sx_last_error()


# ---------------------------------------------------------------- selective scan

def _scan(lib, dtype=B.SX_BF16, x=(2, 130, 64), b=(2, 130, 2, 16), x_at=_at(0), delta=_at(1), a=_at(2), b_at=_at(3),
          c=_at(4), skip=_at(5), z=_at(6), bias=_at(7), initial=None, lengths=None, out=_at(8), last=_at(9), ws=_at(10),
          ws_bytes=1 << 40):
    return lib.sx_selective_scan(dtype, _i64(x), None, x_at, None, delta, a, _i64(b), None, b_at, None, c, skip, None, z,
                                 bias, 1, initial, lengths, out, last, ws, ws_bytes, None)


SCAN = [
    (dict(dtype=7), B.SX_E_DIM_002),
    (dict(x=None), B.SX_E_DIM_001),
    (dict(b=None), B.SX_E_DIM_001),
    (dict(x=(2, 130, 0)), B.SX_E_DIM_001),
    (dict(x=(2, -1, 64)), B.SX_E_DIM_001),
    (dict(b=(2, 131, 2, 16)), B.SX_E_DIM_001),
    (dict(b=(3, 130, 2, 16)), B.SX_E_DIM_001),
    (dict(b=(2, 130, 3, 16)), B.SX_E_DIM_001),                # 3 groups do not divide 64 channels
    (dict(b=(2, 130, 0, 16)), B.SX_E_DIM_001),
    (dict(b=(2, 130, 2, 0)), B.SX_E_DIM_001),
    (dict(b=(2, 130, 2, 33)), B.SX_E_UNSUPPORTED),
    (dict(x=(2, 130, 1 << 25)), B.SX_E_UNSUPPORTED),
    (dict(x=(1 << 30, 1 << 20, 64), b=(1 << 30, 1 << 20, 1, 16)), B.SX_E_UNSUPPORTED),
    (dict(x=(1 << 31, 1, 64), b=(1 << 31, 1, 1, 16)), B.SX_E_UNSUPPORTED),
    (dict(x_at=None), B.SX_E_DIM_003),
    (dict(delta=None), B.SX_E_DIM_003),
    (dict(a=None), B.SX_E_DIM_003),
    (dict(b_at=None), B.SX_E_DIM_003),
    (dict(c=None), B.SX_E_DIM_003),
    (dict(out=None), B.SX_E_DIM_003),
    (dict(out=_at(0)), B.SX_E_ALIAS),
    (dict(out=_at(6) + 128), B.SX_E_ALIAS),
    (dict(out=_at(2)), B.SX_E_ALIAS),
    (dict(last=_at(8)), B.SX_E_ALIAS),
    (dict(last=_at(11), initial=_at(11)), B.SX_E_ALIAS),
    (dict(out=_at(8) + 2), B.SX_E_UNSUPPORTED),
    (dict(last=_at(9) + 4), B.SX_E_UNSUPPORTED),
]


@pytest.mark.parametrize("kwargs,code", SCAN)
def test_selective_scan_refuses(lib, kwargs, code):
    assert _scan(lib, **kwargs) == code, lib.sx_last_error()
    assert lib.sx_last_error()


def test_selective_scan_workspace(lib):
    # a long sequence of few channels is split, so it needs a workspace
    x, b = (1, 8192, 64), (1, 8192, 1, 16)
    need = lib.sx_selective_scan_workspace_bytes(B.SX_BF16, _i64(x), _i64(b))
    assert need > 0 and need % 256 == 0
    assert _scan(lib, x=x, b=b, ws=None) == B.SX_E_WORKSPACE
    assert _scan(lib, x=x, b=b, ws_bytes=need - 1) == B.SX_E_WORKSPACE
    assert _scan(lib, x=x, b=b, ws=_at(10) + 16) == B.SX_E_WORKSPACE
    assert lib.sx_selective_scan_workspace_bytes(B.SX_BF16, _i64(x), _i64((1, 8192, 1, 99))) == 0
    assert lib.sx_selective_scan_workspace_bytes(9, _i64(x), _i64(b)) == 0
    assert lib.sx_selective_scan_workspace_bytes(B.SX_BF16, _i64((1, 5, 64)), _i64((1, 5, 1, 16))) == 0


def _scan_backward(lib, dtype=B.SX_F32, x=(2, 30, 64), b=(2, 30, 2, 16), z=_at(6), go=_at(8), gs=None, initial=None,
                   gx=_at(9), gdelta=_at(10), ga=_at(11), gb=_at(12), gc=_at(13), gskip=_at(14), gz=_at(15), gbias=_at(16),
                   gi=_at(17), ws=_at(18), ws_bytes=1 << 40, a=_at(2)):
    return lib.sx_selective_scan_backward(dtype, _i64(x), None, _at(0), None, _at(1), a, _i64(b), None, _at(3), None,
                                          _at(4), _at(5), None, z, _at(7), 1, initial, None, None, go, gs, gx, gdelta, ga,
                                          gb, gc, gskip, gz, gbias, gi, ws, ws_bytes, None)


@pytest.mark.parametrize("kwargs,code", [
    (dict(dtype=5), B.SX_E_DIM_002),
    (dict(b=(2, 31, 2, 16)), B.SX_E_DIM_001),
    (dict(b=(2, 30, 2, 40)), B.SX_E_UNSUPPORTED),
    (dict(a=None), B.SX_E_DIM_003),
    (dict(go=None), B.SX_E_DIM_003),
    (dict(gx=None), B.SX_E_DIM_003),
    (dict(gdelta=None), B.SX_E_DIM_003),
    (dict(ga=None), B.SX_E_DIM_003),
    (dict(gb=None), B.SX_E_DIM_003),
    (dict(gc=None), B.SX_E_DIM_003),
    (dict(gz=None), B.SX_E_DIM_003),
    (dict(gx=_at(8)), B.SX_E_ALIAS),
    (dict(gx=_at(10)), B.SX_E_ALIAS),
    (dict(gi=_at(19), gs=_at(19)), B.SX_E_ALIAS),
    (dict(gi=_at(19), initial=_at(19)), B.SX_E_ALIAS),
    (dict(ga=_at(2)), B.SX_E_ALIAS),
    (dict(gskip=_at(14) + 4), B.SX_E_UNSUPPORTED),
    (dict(ws=None), B.SX_E_WORKSPACE),
    (dict(ws_bytes=256), B.SX_E_WORKSPACE),
])
def test_selective_scan_backward_refuses(lib, kwargs, code):
    assert _scan_backward(lib, **kwargs) == code, lib.sx_last_error()


def _scan_step(lib, dtype=B.SX_BF16, x=(3, 64), b=(3, 2, 16), x_at=_at(0), pool=8, stride=64 * 16, state=_at(8),
               slots=_at(9), out=_at(10)):
    return lib.sx_selective_scan_step(dtype, _i64(x), None, x_at, None, _at(1), _at(2), _i64(b), None, _at(3), None,
                                      _at(4), None, None, None, None, 1, pool, stride, state, slots, out, None)


@pytest.mark.parametrize("kwargs,code", [
    (dict(dtype=3), B.SX_E_DIM_002),
    (dict(b=(4, 2, 16)), B.SX_E_DIM_001),
    (dict(b=(3, 5, 16)), B.SX_E_DIM_001),
    (dict(b=(3, 2, 64)), B.SX_E_UNSUPPORTED),
    (dict(pool=-1), B.SX_E_DIM_001),
    (dict(pool=2, slots=None), B.SX_E_DIM_001),
    (dict(stride=64 * 16 - 4), B.SX_E_UNSUPPORTED),
    (dict(stride=0), B.SX_E_UNSUPPORTED),
    (dict(x_at=None), B.SX_E_DIM_003),
    (dict(state=None), B.SX_E_DIM_003),
    (dict(out=None), B.SX_E_DIM_003),
    (dict(state=_at(0)), B.SX_E_ALIAS),
    (dict(out=_at(8) + 256), B.SX_E_ALIAS),
    (dict(out=_at(10) + 4), B.SX_E_UNSUPPORTED),
    (dict(state=_at(8) + 2), B.SX_E_UNSUPPORTED),
])
def test_selective_scan_step_refuses(lib, kwargs, code):
    assert _scan_step(lib, **kwargs) == code, lib.sx_last_error()


# ---------------------------------------------------------------- group norm

def _norm(lib, dtype=B.SX_BF16, x=(3, 50, 64), strides=None, groups=8, x_at=_at(0), w=_at(1), bias=_at(2), eps=1e-5,
          act=0, out=_at(3), ws=_at(4), ws_bytes=1 << 40):
    return lib.sx_group_norm(dtype, _i64(x), _i64(strides), x_at, groups, w, bias, eps, act, out, ws, ws_bytes, None)


NORM = [
    (dict(dtype=7), B.SX_E_DIM_002),
    (dict(x=None), B.SX_E_DIM_001),
    (dict(x=(3, 50, 0)), B.SX_E_DIM_001),
    (dict(x=(3, -50, 64)), B.SX_E_DIM_001),
    (dict(x=(1 << 40, 1 << 10, 64)), B.SX_E_UNSUPPORTED),
    (dict(groups=0), B.SX_E_DIM_001),
    (dict(groups=-8), B.SX_E_DIM_001),
    (dict(groups=7), B.SX_E_DIM_001),
    (dict(eps=-1.0), B.SX_E_DIM_001),
    (dict(eps=float("nan")), B.SX_E_DIM_001),
    (dict(act=3), B.SX_E_UNSUPPORTED),
    (dict(strides=(50 * 64, 1, 50)), B.SX_E_UNSUPPORTED),     # channels first
    (dict(x_at=None), B.SX_E_DIM_003),
    (dict(out=None), B.SX_E_DIM_003),
    (dict(out=_at(0)), B.SX_E_ALIAS),
    (dict(out=_at(1)), B.SX_E_ALIAS),
    (dict(out=_at(3) + 2), B.SX_E_UNSUPPORTED),
    (dict(ws=None), B.SX_E_WORKSPACE),
    (dict(ws_bytes=8), B.SX_E_WORKSPACE),
    (dict(ws=_at(4) + 128), B.SX_E_WORKSPACE),
]


@pytest.mark.parametrize("kwargs,code", NORM)
def test_group_norm_refuses(lib, kwargs, code):
    assert _norm(lib, **kwargs) == code, lib.sx_last_error()


def test_group_norm_backward_refuses(lib):
    def call(x=(3, 50, 64), groups=8, gs=None, go=_at(3), gx=_at(4), gw=_at(5), ws=_at(6), ws_bytes=1 << 40):
        return lib.sx_group_norm_backward(B.SX_F32, _i64(x), None, _at(0), groups, _at(1), _at(2), 1e-5, 1, _i64(gs), go,
                                          gx, gw, None, ws, ws_bytes, None)

    assert call(groups=9) == B.SX_E_DIM_001
    assert call(gs=(3200, 1, 50)) == B.SX_E_UNSUPPORTED
    assert call(go=None) == B.SX_E_DIM_003
    assert call(gx=None) == B.SX_E_DIM_003
    assert call(gx=_at(3)) == B.SX_E_ALIAS
    assert call(gw=_at(4)) == B.SX_E_ALIAS
    assert call(gw=_at(1)) == B.SX_E_ALIAS
    assert call(ws=None) == B.SX_E_WORKSPACE
    assert call(ws_bytes=16) == B.SX_E_WORKSPACE
    assert call(ws=_at(6) + 8) == B.SX_E_WORKSPACE


def test_workspaces_of_shapes_that_are_refused(lib):
    assert lib.sx_causal_conv_backward_workspace_bytes(B.SX_F32, _i64((2, 30, 64)), 9) == 0
    assert lib.sx_causal_conv_backward_workspace_bytes(B.SX_F32, _i64((2, 30, 64)), 4) > 0
    assert lib.sx_selective_scan_backward_workspace_bytes(B.SX_F32, _i64((2, 30, 64)), _i64((2, 30, 5, 16))) == 0
    assert lib.sx_group_norm_workspace_bytes(B.SX_F32, _i64((2, 30, 64)), 7) == 0
    assert lib.sx_group_norm_backward_workspace_bytes(4, _i64((2, 30, 64)), 8) == 0


# ---------------------------------------------------------------- the binding

def test_binding_refuses_host_tensors():
    x, d, w = torch.zeros(1, 2, 4), torch.zeros(4), torch.zeros(4, 3)
    a, b = torch.zeros(4, 2), torch.zeros(1, 2, 1, 2)
    for call in (lambda: sx.causal_conv(x, w), lambda: sx.causal_conv_backward(x, w, x),
                 lambda: sx.causal_conv_step(x[:, 0], w, torch.zeros(1, 2, 4)),
                 lambda: sx.selective_scan(x, x, a, b, b), lambda: sx.selective_scan_backward(x, x, a, b, b, x),
                 lambda: sx.selective_scan_step(x[:, 0], x[:, 0], a, b[:, 0], b[:, 0], torch.zeros(1, 4, 2)),
                 lambda: sx.group_norm(x, 2, weight=d), lambda: sx.group_norm_backward(x, 2, x)):
        with pytest.raises(sx.SxError) as e:
            call()
        assert e.value.code == B.SX_E_UNSUPPORTED
    for call in (lambda: sx.causal_conv(None, w), lambda: sx.selective_scan(x, x, None, b, b),
                 lambda: sx.group_norm([1.0], 1)):
        with pytest.raises(sx.SxError) as e:
            call()
        assert e.value.code in (B.SX_E_DIM_003, B.SX_E_UNSUPPORTED)


def test_the_binding_without_its_extension(monkeypatch):
    monkeypatch.setattr(B, "_marshal", B._LongWay())
    test_binding_refuses_host_tensors()
