"""The linear-attention entry points on the CPU: what the C ABI and the binding refuse before any device work."""

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


def _forward(lib, dtype=B.SX_BF16, q=(2, 130, 4, 32), k=None, v=(2, 130, 4, 32), g=(2, 130, 4), q_at=_at(0),
             k_at=_at(1), v_at=_at(2), g_at=_at(3), out=_at(4), last=_at(5), ws=_at(6), ws_bytes=0, initial=None, lengths=None,
             qs=None):
    k = q if k is None else k
    return lib.sx_decay_attention(dtype, _i64(q), _i64(qs), q_at, _i64(k), None, k_at, _i64(v), None, v_at, len(g),
                                  _i64(g), None, g_at, initial, lengths, 1.0, out, last, ws, ws_bytes, None)


FORWARD = [
    (dict(dtype=7), B.SX_E_DIM_002),
    (dict(q=(2, 130, 4, 0)), B.SX_E_DIM_001),
    (dict(q=(2, -1, 4, 32)), B.SX_E_DIM_001),
    (dict(k=(2, 131, 4, 32)), B.SX_E_DIM_001),
    (dict(k=(2, 130, 4, 31)), B.SX_E_DIM_001),
    (dict(v=(3, 130, 4, 32)), B.SX_E_DIM_001),
    (dict(g=(2, 131, 4)), B.SX_E_DIM_001),
    (dict(g=(130, 4)), B.SX_E_DIM_001),                       # neither [H] nor [B, T, H]
    (dict(g=(0,)), B.SX_E_DIM_001),
    (dict(g=(6,)), B.SX_E_DIM_001),                           # 4 heads do not divide 6
    (dict(v=(2, 130, 3, 32)), B.SX_E_DIM_001),
    (dict(q=(2, 130, 0, 32)), B.SX_E_DIM_001),
    (dict(q=(2, 130, 4, 257)), B.SX_E_UNSUPPORTED),
    (dict(v=(2, 130, 4, 300)), B.SX_E_UNSUPPORTED),
    (dict(q_at=None), B.SX_E_DIM_003),
    (dict(k_at=None), B.SX_E_DIM_003),
    (dict(v_at=None), B.SX_E_DIM_003),
    (dict(g_at=None), B.SX_E_DIM_003),
    (dict(out=None), B.SX_E_DIM_003),
    (dict(out=_at(0) + 64), B.SX_E_ALIAS),
    (dict(out=_at(3)), B.SX_E_ALIAS),
    (dict(last=_at(4)), B.SX_E_ALIAS),
    (dict(last=_at(7), initial=_at(7)), B.SX_E_ALIAS),
    (dict(out=_at(4) + 8), B.SX_E_UNSUPPORTED),               # alignment
    (dict(last=_at(5) + 4), B.SX_E_UNSUPPORTED),
]


@pytest.mark.parametrize("kwargs,code", FORWARD)
def test_decay_attention_refuses(lib, kwargs, code):
    assert _forward(lib, **kwargs) == code, lib.sx_last_error()
    assert lib.sx_last_error()


def test_decay_attention_workspace(lib):
    # a long sequence of one head is split, so it needs a workspace; many rows need none
    q, v = _i64((1, 8192, 1, 64)), _i64((1, 8192, 1, 64))
    need = lib.sx_decay_attention_workspace_bytes(B.SX_BF16, q, v, 1)
    assert need > 0 and need % 256 == 0
    long = dict(q=(1, 8192, 1, 64), v=(1, 8192, 1, 64), g=(1,))
    assert _forward(lib, **long, ws=None) == B.SX_E_WORKSPACE
    assert _forward(lib, **long, ws_bytes=need - 1) == B.SX_E_WORKSPACE
    assert _forward(lib, **long, ws=_at(6) + 16, ws_bytes=need) == B.SX_E_WORKSPACE
    assert lib.sx_decay_attention_workspace_bytes(B.SX_BF16, _i64((1, 8, 1, 999)), v, 1) == 0
    assert lib.sx_decay_attention_workspace_bytes(9, q, v, 1) == 0


def test_decay_attention_of_nothing_is_a_no_op(lib):
    assert _forward(lib, q=(0, 130, 4, 32), v=(0, 130, 4, 32), g=(4,), q_at=None, out=None) == B.SX_OK
    assert _forward(lib, q=(2, 0, 4, 32), v=(2, 0, 4, 32), g=(4,), q_at=None, out=None, last=None) == B.SX_OK


def _backward(lib, dtype=B.SX_F32, q=(2, 30, 4, 32), v=(2, 30, 4, 32), g=(2, 30, 4), go=_at(4), initial=None, gi=None,
              gq=_at(8), gk=_at(9), gv=_at(10), gg=_at(11), gs=None, ws=_at(12), ws_bytes=1 << 40):
    return lib.sx_decay_attention_backward(dtype, _i64(q), None, _at(0), _i64(q), None, _at(1), _i64(v), None, _at(2),
                                           len(g), _i64(g), None, _at(3), None, go, gs, initial, None, 1.0, gq, gk, gv,
                                           gg, gi, ws, ws_bytes, None)


@pytest.mark.parametrize("kwargs,code", [
    (dict(dtype=5), B.SX_E_DIM_002),
    (dict(v=(2, 31, 4, 32)), B.SX_E_DIM_001),
    (dict(q=(2, 30, 4, 257)), B.SX_E_UNSUPPORTED),
    (dict(go=None), B.SX_E_DIM_003),
    (dict(gq=None), B.SX_E_DIM_003),
    (dict(gk=None), B.SX_E_DIM_003),
    (dict(gv=None), B.SX_E_DIM_003),
    (dict(gg=None), B.SX_E_DIM_003),
    (dict(initial=_at(5)), B.SX_E_DIM_003),                   # its gradient is missing
    (dict(initial=_at(5), gi=_at(5)), B.SX_E_ALIAS),
    (dict(gq=_at(4)), B.SX_E_ALIAS),
    (dict(gq=_at(9)), B.SX_E_ALIAS),
    (dict(gs=_at(11)), B.SX_E_ALIAS),
    (dict(gv=_at(10) + 4), B.SX_E_UNSUPPORTED),
    (dict(ws=None), B.SX_E_WORKSPACE),
    (dict(ws_bytes=256), B.SX_E_WORKSPACE),
])
def test_decay_attention_backward_refuses(lib, kwargs, code):
    assert _backward(lib, **kwargs) == code, lib.sx_last_error()


def _step(lib, dtype=B.SX_BF16, q=(3, 4, 32), k=None, v=(3, 4, 16), g=(3, 4), q_at=_at(0), state=_at(4), slots=_at(5),
          pool=8, strides=None, out=_at(6)):
    k = q if k is None else k
    return lib.sx_decay_attention_step(dtype, _i64(q), None, q_at, _i64(k), None, _at(1), _i64(v), None, _at(2), len(g),
                                       _i64(g), None, _at(3), pool, _i64(strides), state, slots, 1.0, out, None)


@pytest.mark.parametrize("kwargs,code", [
    (dict(dtype=3), B.SX_E_DIM_002),
    (dict(k=(3, 4, 31)), B.SX_E_DIM_001),
    (dict(v=(4, 4, 16)), B.SX_E_DIM_001),
    (dict(g=(2, 4)), B.SX_E_DIM_001),
    (dict(g=(3, 1, 4)), B.SX_E_DIM_001),
    (dict(g=(6,)), B.SX_E_DIM_001),
    (dict(pool=-1), B.SX_E_DIM_001),
    (dict(pool=2, slots=None), B.SX_E_DIM_001),               # three rows, two states
    (dict(q=(3, 4, 300)), B.SX_E_UNSUPPORTED),
    (dict(strides=(2048, 512, 1, 32)), B.SX_E_UNSUPPORTED),   # a head's state transposed
    (dict(strides=(2048, 256, 16, 1)), B.SX_E_UNSUPPORTED),   # heads overlap
    (dict(strides=(0, 512, 16, 1)), B.SX_E_UNSUPPORTED),      # one state for all slots
    (dict(q_at=None), B.SX_E_DIM_003),
    (dict(state=None), B.SX_E_DIM_003),
    (dict(out=None), B.SX_E_DIM_003),
    (dict(state=_at(0)), B.SX_E_ALIAS),
    (dict(out=_at(4)), B.SX_E_ALIAS),
    (dict(out=_at(6) + 2), B.SX_E_UNSUPPORTED),
])
def test_decay_attention_step_refuses(lib, kwargs, code):
    assert _step(lib, **kwargs) == code, lib.sx_last_error()


def test_decay_attention_step_of_nothing_is_a_no_op(lib):
    assert _step(lib, q=(0, 4, 32), v=(0, 4, 16), g=(4,), q_at=None, out=None) == B.SX_OK


def _rotate(lib, dtype=B.SX_BF16, q=(2, 5, 4, 64), k=(2, 5, 2, 64), q_at=_at(0), positions=_at(2), rotated=64,
            turns=_at(3), eps=1e-6, out_q=_at(4), out_k=_at(5)):
    return lib.sx_head_norm_rotate(dtype, _i64(q), None, q_at, _i64(k), None, _at(1), 1, None, positions, rotated,
                                   turns, None, None, eps, 0, out_q, out_k, None)


ROTATE = [
    (dict(dtype=4), B.SX_E_DIM_002),
    (dict(k=(2, 6, 2, 64)), B.SX_E_DIM_001),
    (dict(k=(2, 5, 2, 63)), B.SX_E_DIM_001),
    (dict(q=(2, 5, 4, 0), k=(2, 5, 2, 0)), B.SX_E_DIM_001),
    (dict(q=(2, 5, 4, 258), k=(2, 5, 2, 258)), B.SX_E_UNSUPPORTED),
    (dict(rotated=63), B.SX_E_DIM_001),
    (dict(rotated=66), B.SX_E_DIM_001),
    (dict(rotated=-2), B.SX_E_DIM_001),
    (dict(eps=-1.0), B.SX_E_DIM_001),
    (dict(eps=float("nan")), B.SX_E_DIM_001),
    (dict(q_at=None), B.SX_E_DIM_003),
    (dict(positions=None), B.SX_E_DIM_003),
    (dict(turns=None), B.SX_E_DIM_003),
    (dict(out_q=None), B.SX_E_DIM_003),
    (dict(out_k=None), B.SX_E_DIM_003),
    (dict(out_q=_at(0)), B.SX_E_ALIAS),
    (dict(out_k=_at(4)), B.SX_E_ALIAS),
    (dict(out_q=_at(2)), B.SX_E_ALIAS),
    (dict(out_q=_at(4) + 2), B.SX_E_UNSUPPORTED),
]


@pytest.mark.parametrize("kwargs,code", ROTATE)
def test_head_norm_rotate_refuses(lib, kwargs, code):
    assert _rotate(lib, **kwargs) == code, lib.sx_last_error()


def test_head_norm_rotate_backward_refuses(lib):
    q, k = (2, 5, 4, 64), (2, 5, 2, 64)

    def call(rotated=64, gq=_at(4), out_q=_at(6), gqw=_at(8), ws=_at(9), ws_bytes=1 << 30):
        return lib.sx_head_norm_rotate_backward(B.SX_F32, _i64(q), None, _at(0), _i64(k), None, _at(1), 1, None, _at(2),
                                                rotated, _at(3), None, gq, None, _at(5), None, None, 1e-6, 0, out_q,
                                                _at(7), gqw, None, ws, ws_bytes, None)

    assert call(rotated=65) == B.SX_E_DIM_001
    assert call(gq=None) == B.SX_E_DIM_003
    assert call(out_q=None) == B.SX_E_DIM_003
    assert call(out_q=_at(4)) == B.SX_E_ALIAS
    assert call(gqw=_at(6)) == B.SX_E_ALIAS
    assert call(ws=None) == B.SX_E_WORKSPACE
    assert call(ws_bytes=16) == B.SX_E_WORKSPACE
    assert call(ws=_at(9) + 8) == B.SX_E_WORKSPACE


def test_binding_refuses_host_tensors():
    x, g = torch.zeros(1, 2, 1, 4), torch.zeros(1)
    pos, turns = torch.zeros(1, 2, dtype=torch.int64), sx.rotation_turns(4)
    for call in (lambda: sx.decay_attention(x, x, x, g), lambda: sx.decay_attention_backward(x, x, x, g, x),
                 lambda: sx.decay_attention_step(x[:, 0], x[:, 0], x[:, 0], g, torch.zeros(1, 1, 4, 4)),
                 lambda: sx.head_norm_rotate(x, x, pos, turns),
                 lambda: sx.head_norm_rotate_backward(x, x, pos, turns, x, x)):
        with pytest.raises(sx.SxError) as e:
            call()
        assert e.value.code == B.SX_E_UNSUPPORTED
    with pytest.raises(sx.SxError) as e:
        sx.decay_attention(None, x, x, g)
    assert e.value.code == B.SX_E_DIM_003


def test_rotation_turns():
    t = sx.rotation_turns(4, base=100.0)
    assert t.dtype == torch.float64
    torch.testing.assert_close(t * 2 * torch.pi, torch.tensor([1.0, 0.1], dtype=torch.float64))
    assert sx.rotation_turns(0).numel() == 0
    with pytest.raises(sx.SxError):
        sx.rotation_turns(3)


def test_decay_attention_step_state_alignment(lib):
    assert _step(lib, state=_at(4) + 2) == B.SX_E_UNSUPPORTED  # inside an f32
    assert b"4-byte aligned" in lib.sx_last_error()


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are no memory: the call must not reach a GPU")
@pytest.mark.parametrize("at", [4, 8, 12])
def test_decay_attention_step_takes_a_state_off_16_byte_borders(lib, at):
    # what is left to refuse it is that there is no device
    assert _step(lib, state=_at(4) + at) == _step(lib) == B.SX_E_DEVICE, lib.sx_last_error()


def test_the_binding_without_its_extension(monkeypatch, tmp_path):
    monkeypatch.setattr(B, "_marshal", None)
    monkeypatch.setattr(B, "MARSHAL_PATH", str(tmp_path / "_sx_marshal.so"))
    with pytest.warns(RuntimeWarning, match="not built or does not load"):
        test_binding_refuses_host_tensors()
    (tmp_path / "_sx_marshal.so").write_bytes(b"another machine's")
    monkeypatch.setattr(B, "_marshal", None)
    with pytest.warns(RuntimeWarning, match="not built or does not load"):
        test_binding_refuses_host_tensors()


def test_the_library_is_built_where_the_extension_does_not_compile(monkeypatch, tmp_path):
    from scan_primitives_amd import build_lib

    old, tmp = tmp_path / "_sx_marshal.so", tmp_path / "_sx_marshal.so.tmp"
    old.write_bytes(b"of other sources")
    monkeypatch.setattr(build_lib, "MARSHAL_PATH", str(old))
    rc, msgs = build_lib._run([str(tmp_path / "no compiler"), "-c"])
    assert rc != 0 and msgs
    assert build_lib._put_marshal(str(tmp), rc, msgs) is False and not old.exists()
    tmp.write_bytes(b"of these")
    assert build_lib._put_marshal(str(tmp), 0, []) is True and old.read_bytes() == b"of these" and not tmp.exists()
