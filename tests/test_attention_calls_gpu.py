"""How decay attention and head norm + rotation are called: optional values of any truth, states that are
written in place, tensors that carry more than their numbers, states at any alignment, long
segments, states that are not finite."""

import numpy as np
import pytest
import torch
import torch.autograd.forward_ad as forward_ad

import scan_primitives_amd as sx
from scan_primitives_amd import _binding as B
from tests import test_head_rotate_gpu as rotate
from tests.test_decay_attention_gpu import (_backward, _close, _forward, _np, _oracle_vjp, _roundings, make,
                                            make_step)

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("true,false", [(1, 0), (np.bool_(True), np.bool_(False)), ("yes", "")])
def test_whether_the_state_is_wanted_goes_by_truth(true, false):
    s = make(t=70, initial=True)
    args = dict(initial=s["initial"], scale=s["scale"])
    out, state = sx.decay_attention(s["q"], s["k"], s["v"], s["g"], return_state=True, **args)
    got = sx.decay_attention(s["q"], s["k"], s["v"], s["g"], return_state=true, **args)
    assert torch.equal(got[0], out) and torch.equal(got[1], state)
    assert torch.equal(sx.decay_attention(s["q"], s["k"], s["v"], s["g"], return_state=false, **args), out)


def test_every_call_without_the_bindings_extension(monkeypatch):
    s, r, one, other = make(t=70, initial=True, lengths=[70, 9]), rotate.make(), make_step(), make_step()
    want = (*_forward(s), *_backward(s), *rotate._forward(r), *rotate._backward(r), _step(one), one["state"])
    monkeypatch.setattr(B, "_marshal", B._LongWay())
    got = (*_forward(s), *_backward(s), *rotate._forward(r), *rotate._backward(r), _step(other), other["state"])
    for a, b in zip(want, got):
        assert torch.equal(a, b)


def _step(s, scale=1.0):
    return sx.decay_attention_step(s["q"], s["k"], s["v"], s["g"], s["state"], slots=s["slots"], scale=scale)


@pytest.mark.parametrize("scale", [1.0, 1])  # the binding's short way and its long one
def test_a_step_on_a_saved_state_is_noticed(scale):
    p, s = make(t=20, type=F32, initial=True), make_step(b=2, pool=2, type=F32)
    q = p["q"].clone().requires_grad_()
    s["state"], s["slots"] = p["initial"], None
    before = s["state"]._version
    loss = sx.decay_attention(q, p["k"], p["v"], p["g"], initial=s["state"]).sum()
    _step(s, scale)
    assert s["state"]._version > before
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


@pytest.mark.parametrize("scale", [1.0, 1])
def test_a_step_does_not_overwrite_a_state_that_autograd_records(scale):
    s = make_step(type=F32)
    kept = s["state"].clone()
    s["state"] = s["state"].requires_grad_()
    with pytest.raises(sx.SxError) as e:
        _step(s, scale)
    assert e.value.code == B.SX_E_UNSUPPORTED and torch.equal(s["state"], kept)
    with torch.no_grad():  # as torch's own operations in place
        _step(s, scale)
    assert not torch.equal(s["state"], kept)


@pytest.mark.parametrize("scale", [1.0, 1])
def test_a_step_on_a_state_made_in_inference_mode(scale):
    s, e = make_step(), make_step()
    with torch.inference_mode():
        s["state"] = s["state"].clone()
    got, want = _step(s, scale), _step(e, scale)
    assert torch.equal(got, want) and torch.equal(s["state"], e["state"])


def _scan_calls(x):
    """Every scan and its gradient on tensors made from x [4, 16]."""
    init = torch.zeros(16, device="cuda")
    a = x.reshape(4, 4, 4)
    return [lambda: sx.element_scan("tanh_affine", init, [x, torch.ones_like(init).expand(4, 16)]),
            lambda: sx.element_scan_backward("tanh_affine", init, [x, x], torch.zeros_like(init).expand(4, 16), x),
            lambda: sx.matrix_scan(a, a), lambda: sx.linear_scan(0.5, x), lambda: sx.cumsum(x),
            lambda: sx.matrix_scan_backward(a, a.shape, a, a)]


def test_tangents_are_refused():
    s, r, one = make(t=20, type=F32), rotate.make(type=F32), make_step(type=F32)
    with forward_ad.dual_level():
        dual = lambda x: forward_ad.make_dual(x, torch.ones_like(x))  # noqa: E731
        calls = [lambda: sx.decay_attention(dual(s["q"]), s["k"], s["v"], s["g"]),
                 lambda: sx.decay_attention(s["q"], s["k"], s["v"], dual(s["g"]), scale=1),
                 lambda: sx.decay_attention(s["q"], s["k"], s["v"], s["g"], initial=dual(s["gs"])),
                 lambda: sx.decay_attention_backward(s["q"], s["k"], s["v"], s["g"], dual(s["go"])),
                 lambda: sx.decay_attention_step(one["q"], dual(one["k"]), one["v"], one["g"], one["state"]),
                 lambda: sx.decay_attention_step(one["q"], one["k"], one["v"], one["g"], dual(one["state"])),
                 lambda: sx.head_norm_rotate(r["q"], dual(r["k"]), r["positions"], r["turns"]),
                 lambda: sx.head_norm_rotate(r["q"], r["k"], r["positions"], r["turns"], k_weight=dual(r["kw"])),
                 lambda: sx.head_norm_rotate_backward(r["q"], r["k"], r["positions"], r["turns"], dual(r["gq"]),
                                                      r["gk"])]
        for i, call in enumerate(calls + _scan_calls(dual(torch.rand(4, 16, device="cuda")))):
            with pytest.raises(sx.SxError) as e:
                call()
            assert e.value.code == B.SX_E_UNSUPPORTED, i
        # tensors without a tangent are as ever
        assert torch.equal(sx.decay_attention(s["q"], s["k"], s["v"], s["g"], scale=s["scale"]), _forward(s)[0])


def _negated(x):
    """A lazily negated view with the values of x."""
    view = torch.complex(torch.zeros_like(x), -x).conj().imag
    assert view.is_neg() and torch.equal(view, x)
    return view


def test_lazily_negated_views_are_read_with_their_sign():
    s, r, one = make(t=40, type=F32, initial=True), rotate.make(type=F32), make_step(type=F32)
    want = (*_forward(s), *_backward(s))
    for n in ("q", "k", "v", "g", "initial", "go", "gs"):
        kept, s[n] = s[n], _negated(s[n])
        for a, b in zip((*_forward(s), *_backward(s)), want):
            torch.testing.assert_close(a, b, rtol=1e-4, atol=1e-4, msg=n)  # other strides, another order of the sums
        s[n] = kept
    want = (*rotate._forward(r), *rotate._backward(r))
    for n in ("q", "k", "turns", "qw", "kw", "gq", "gk"):
        kept, r[n] = r[n], _negated(r[n])
        for a, b in zip((*rotate._forward(r), *rotate._backward(r)), want):
            torch.testing.assert_close(a, b, rtol=1e-4, atol=1e-4, msg=n)
        r[n] = kept
    x = torch.rand(4, 16, device="cuda")
    for i, (a, b) in enumerate(zip(_scan_calls(_negated(x)), _scan_calls(x))):
        torch.testing.assert_close(a(), b(), msg=str(i))
    state, one["k"] = one["state"].clone(), _negated(one["k"])
    got = sx.decay_attention_step(one["q"], one["k"], one["v"], one["g"], one["state"], slots=one["slots"])
    want = sx.decay_attention_step(one["q"], one["k"].clone(), one["v"], one["g"], state, slots=one["slots"])
    assert torch.equal(got, want) and torch.equal(one["state"], state)
    with pytest.raises(sx.SxError) as e:  # a state is written: its numbers have to be what is in memory
        sx.decay_attention_step(one["q"], one["k"], one["v"], one["g"], _negated(state))
    assert e.value.code == B.SX_E_UNSUPPORTED


@pytest.mark.parametrize("name,at", [("q", 0), ("k", 1), ("v", 2)])
def test_autograd_of_a_lazily_negated_view(name, at):
    s = make(t=40, type=F32)
    x = torch.complex(torch.zeros_like(s[name]), -s[name]).requires_grad_()
    out = sx.decay_attention(*(x.conj().imag if n == name else s[n] for n in ("q", "k", "v", "g")), scale=s["scale"])
    torch.testing.assert_close(out, _forward(s)[0], rtol=1e-4, atol=1e-4)
    out.backward(s["go"])
    torch.testing.assert_close(-x.grad.imag, _backward(s, grad_state=False)[at], rtol=1e-4, atol=1e-4)


@pytest.mark.parametrize("name,room,view,dk,dv", [
    ("slots from the second on", (5, 1, 33, 33), lambda x: x[1:], 33, 33),
    ("heads from the second on", (4, 3, 33, 47), lambda x: x[:, 1:], 33, 47),
    ("states a word past a 16-byte border", (4, 2, 32 * 32 + 4), lambda x: x[..., 1:-3].unflatten(-1, (32, 32)), 32,
     32),
])
def test_a_step_on_a_view_of_a_pool(name, room, view, dk, dv):
    room = torch.randn(room, device="cuda")
    state = view(room)
    s = make_step(b=3, pool=4, h=state.shape[1], dk=dk, dv=dv, slots=None)
    kept, alone = room.clone(), state.clone(memory_format=torch.contiguous_format)
    assert state.data_ptr() % 16 != 0 and alone.data_ptr() % 16 == 0
    got = sx.decay_attention_step(s["q"], s["k"], s["v"], s["g"], state, scale=s["scale"])
    assert torch.equal(got, sx.decay_attention_step(s["q"], s["k"], s["v"], s["g"], alone, scale=s["scale"]))
    assert torch.equal(state, alone)
    view(kept).copy_(state)
    assert torch.equal(room, kept)  # nothing else of the buffer has changed


def _whole_numbers(b=1, t=200, h=4, dk=16, dv=16, type=F32, cuts=False, lengths=None, hq=None, seed=0):
    """Operands of -1, 0 and 1 and decays of one or nothing: every product and sum is a whole number."""
    s = make(b=b, t=t, h=h, hq=hq, dk=dk, dv=dv, type=type, initial=True, lengths=lengths, seed=seed,
             decay="cuts" if cuts else "none")
    if cuts:
        s["g"] = torch.where(torch.isinf(s["g"]), s["g"], torch.zeros_like(s["g"]))
    for n in ("q", "k", "v", "go", "initial", "gs"):
        s[n] = s[n].float().round().clamp(-1, 1).to(s[n].dtype)
    s["scale"] = 1.0
    return s


@pytest.mark.parametrize("type", [BF, F32])
@pytest.mark.parametrize("name,kwargs", [
    ("one chunk", dict(t=20)), ("chunks", dict(t=200)), ("segments", dict(t=1000, h=2)),
    ("cuts", dict(t=300, cuts=True)),
    ("segments, cuts", dict(t=1000, h=2, cuts=True)), ("two column blocks", dict(t=150, dk=130, dv=8)),
    ("shared", dict(t=150, h=6, hq=2)), ("ragged", dict(b=3, t=300, lengths=[300, 0, 77], cuts=True)),
    # segments of several spans (256 tokens in f32, 512 in bf16 at most), rows that end in and between them
    ("spans", dict(t=1500, h=260, dk=5, dv=3, cuts=True)),
    ("spans, ragged", dict(b=4, t=1500, h=90, lengths=[1500, 0, 700, 1024], dk=5, dv=6)),
    ("spans, two column blocks", dict(t=1100, h=260, dk=130, dv=9)),
    ("spans and segments", dict(b=2, t=6000, h=50, lengths=[6000, 1111], dk=4, dv=7, cuts=True)),
])
def test_the_decays_gradient_of_whole_numbers_is_exact(type, name, kwargs):
    s = _whole_numbers(type=type, **kwargs)
    # no sum of absolute values that enters a result reaches 2^24: in 32 bits nothing is rounded
    ref = _oracle_vjp(s)
    assert np.abs(ref[3]).max() < 2.0 ** 22
    assert np.array_equal(_np(_backward(s)[3]), ref[3])


@pytest.mark.parametrize("type,t", [(F32, 1000), (BF, 1500), (F32, 8300), (BF, 16500)])
def test_what_large_tokens_leave_is_taken_off_at_a_segments_end(type, t):
    # Heads enough that each is one segment (the last two lengths: of more than 256 chunks). The first quarter's
    # values and gradients are 2^10 times the others', and a decay of exp(-0.05) a token leaves nothing of them 512
    # tokens on: but the roundings of the sums that are carried, which only the sum that is known at the end takes off.
    # Without it they are about 2^-24 (2^10)^2 times a chunk's sums of the other tokens.
    s = make(b=1, t=t, h=260, dk=2, dv=2, type=type)
    s["g"] = torch.full_like(s["g"], -0.05)
    s["v"][:, :t // 4] *= 1024
    s["go"][:, :t // 4] *= 1024
    tail = t // 4 + 512
    got = _backward(s, grad_state=False)[3]
    ref, size = _oracle_vjp(s, grad_state=False), _oracle_vjp(s, grad_state=False, size=True)
    # a chunk of 64 tokens' sums of q . grad_q and k . grad_k, as everywhere
    mass = (np.abs(_np(s["q"])) * size[0]).sum(-1) + (np.abs(_np(s["k"])) * size[1]).sum(-1)
    floor = 64.0 * mass[:, tail:].max()
    _close("grad_log_decay", got[:, tail:], ref[3][:, tail:], size[3][:, tail:], _roundings(s), False, floor=floor)


@pytest.mark.parametrize("type", [BF, F32])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("t,at", [(1, 0), (40, 0), (150, 70), (150, 64), (1000, 0), (1000, 700)])
def test_a_cut_clears_a_state_that_is_not_finite(type, value, t, at):
    s = make(b=1, t=t, h=2, dk=40, dv=24, type=type, initial=True)
    s["g"][:, at] = -float("inf")
    clean, grads = _forward(s), _backward(s)
    s["initial"][0, 0, 3], s["initial"][0, 1, :, 5] = value, value
    out, last = _forward(s)
    assert torch.equal(out[:, at:], clean[0][:, at:]) and torch.equal(last, clean[1])
    assert at == 0 or not torch.isfinite(out[:, :at, 0]).any()
    gq, gk, gv, gg, gi = _backward(s)
    assert torch.equal(gq[:, at:], grads[0][:, at:])
    for a, b in ((gk, grads[1]), (gv, grads[2]), (gi, grads[4])):
        assert torch.equal(a, b)
    if at == 0:
        # what is carried over the borders is kept by differences: another start, other roundings of them
        torch.testing.assert_close(gg, grads[3], rtol=1e-4, atol=1e-3)
    assert torch.isfinite(gg[:, at:]).all() and not gg[:, at].any()


@pytest.mark.parametrize("type", [BF, F32])
def test_a_cut_clears_a_gradient_of_the_state_that_is_not_finite(type):
    s = make(b=1, t=150, h=2, dk=40, dv=24, type=type, initial=True)
    s["g"][:, 70] = -float("inf")
    clean = _backward(s)
    s["gs"][0, 0, 3, 4] = float("nan")
    got = _backward(s)
    assert torch.equal(got[0], clean[0]) and torch.equal(got[4], clean[4])
    assert torch.equal(got[1][:, :70], clean[1][:, :70]) and torch.equal(got[2][:, :70], clean[2][:, :70])


@pytest.mark.parametrize("dv", [24, 33, 128])
@pytest.mark.parametrize("g", [-float("inf"), -150.0])
def test_a_first_token_that_cuts_starts_on_an_uncleared_slot(dv, g):
    s, e = (make_step(b=5, pool=8, dk=40, dv=dv, slots="all used") for _ in range(2))
    s["g"][2] = e["g"][2] = g
    slot = s["slots"][2].long()
    s["state"][slot], e["state"][slot] = float("nan"), 0.0
    s["state"][slot, 1] = float("inf")
    got, want = (sx.decay_attention_step(x["q"], x["k"], x["v"], x["g"], x["state"], slots=x["slots"]) for x in (s, e))
    assert torch.equal(got, want) and torch.equal(s["state"], e["state"])


@pytest.mark.parametrize("type", [BF, F32])
def test_what_large_tokens_leave_does_not_pass_between_them(type):
    # The same with large tokens at both ends: what their roundings leave in a sum that is carried through the middle is
    # known at neither end alone. The middle's spans start from sums of their own. (Of the middle, the tokens 512 and a
    # span of 512 at most away from the large ones.)
    t = 8300
    s = make(b=1, t=t, h=260, dk=2, dv=2, type=type)
    s["g"] = torch.full_like(s["g"], -0.05)
    for part in (slice(0, t // 4), slice(3 * t // 4, t)):
        s["v"][:, part] *= 1024
        s["go"][:, part] *= 1024
    middle = slice(t // 4 + 1024, 3 * t // 4 - 1024)
    got = _backward(s, grad_state=False)[3]
    ref, size = _oracle_vjp(s, grad_state=False), _oracle_vjp(s, grad_state=False, size=True)
    mass = (np.abs(_np(s["q"])) * size[0]).sum(-1) + (np.abs(_np(s["k"])) * size[1]).sum(-1)
    floor = 64.0 * mass[:, middle].max()
    _close("grad_log_decay", got[:, middle], ref[3][:, middle], size[3][:, middle], _roundings(s), False, floor=floor)
