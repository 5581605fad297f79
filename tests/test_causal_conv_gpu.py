"""The causal convolution on the GPU against the 64-bit oracle.

Tolerances, from the arithmetic: a result is a sum of K + 1 terms in 32 bits,
off by at most (K + 1) 2^-24 of what they add up to before they cancel (the
oracle's `size`); SiLU's exponential, reciprocal and products add at most 8 more
such steps (its slope is at most 1.1), and a gradient's weights and biases, sums over n
tokens, eight standard deviations of as many independent roundings, 8 sqrt(n) 2^-24. bf16
results are rounded once: 2^-8 of themselves.
"""

import numpy as np
import pytest
import torch

import scan_primitives_amd as sx
from oracle import state_space as os_

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def _np(x):
    return None if x is None else x.detach().double().cpu().numpy()


def close(name, got, ref, size, steps, floor=0.0):
    bf16 = got.dtype == BF
    got = _np(got)
    assert got.shape == ref.shape, name
    assert np.isfinite(got).all(), f"{name}: not finite"
    tol = floor + steps * 2.0 ** -24 * size + (2.0 ** -8 * np.abs(ref) if bf16 else 0.0)
    over = np.abs(got - ref) - tol
    if over.size and over.max() > 1e-37:
        at = np.unravel_index(np.argmax(over), over.shape)
        raise AssertionError(f"{name} at {at}: got {got[at]!r}, ref {ref[at]!r}, tolerance {tol[at]!r}")


def make(b=2, t=100, d=72, k=4, type=BF, act="silu", bias=True, initial=False, lengths=None, layout="plain", seed=0):
    gen = torch.Generator().manual_seed(2000 + seed)
    r = lambda *shape: torch.randn(*shape, generator=gen)  # noqa: E731

    def laid():
        if layout == "half of a projection":
            return r(b, t, 2 * d).to(type).to(DEV)[..., d:]
        if layout == "channels first":
            return r(b, d, t).to(type).to(DEV).transpose(1, 2)
        if layout == "odd offset":
            return r(b, t, d + 3).to(type).to(DEV)[..., 1:d + 1]
        if layout == "one row for all":
            return r(1, t, d).to(type).to(DEV).expand(b, t, d)
        if layout == "every other token":
            return r(b, 2 * t, d).to(type).to(DEV)[:, ::2]
        return r(b, t, d).to(type).to(DEV)

    return dict(x=laid(), weight=r(d, k).to(DEV), bias=r(d).to(DEV) if bias else None,
                initial=r(b, k - 1, d).to(type).to(DEV) if initial else None,
                lengths=None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device=DEV),
                activation=act), dict(grad_out=laid(), grad_state=r(b, k - 1, d).to(type).to(DEV) if initial else None)


def host(s):
    s = {n: (_np(v) if isinstance(v, torch.Tensor) else v) for n, v in s.items()}
    if s.get("lengths") is not None:
        s["lengths"] = s["lengths"].astype(np.int64)
    return s


CASES = {
    "ordinary": dict(),
    "f32": dict(type=F32),
    "one token": dict(t=1, initial=True),
    "two tokens": dict(t=2, initial=True, lengths=[2, 1]),
    "one tap": dict(k=1, t=37, initial=True),
    "two taps, no activation": dict(k=2, act=None, type=F32),
    "three taps": dict(k=3, initial=True, type=F32),
    "five taps": dict(k=5, t=9, initial=True),
    "seven taps": dict(k=7, t=5, initial=True, lengths=[5, 3], type=F32),
    "eight taps": dict(k=8, t=300, initial=True, lengths=[300, 4]),
    "one channel": dict(d=1, type=F32, initial=True),
    "three channels": dict(d=3),
    "five channels": dict(d=5, type=F32),
    "odd channels": dict(d=333, t=65),
    "odd channels f32": dict(d=1050, t=33, type=F32, initial=True),
    "many channels": dict(b=1, d=4096, t=130),
    "long": dict(b=1, d=16, t=9000, initial=True),
    "long f32": dict(b=3, d=9, t=4001, type=F32, initial=True, lengths=[4001, 0, 2000]),
    "ragged": dict(b=5, t=130, lengths=[130, 0, 1, 2, 77], initial=True),
    "lengths out of range": dict(b=3, t=40, lengths=[-5, 99, 40]),
    "no bias": dict(bias=False),
    "half of a projection": dict(layout="half of a projection"),
    "channels first": dict(layout="channels first", initial=True),
    "channels first f32": dict(layout="channels first", type=F32),
    "odd offset": dict(layout="odd offset"),
    "one row for all": dict(layout="one row for all"),
    "every other token": dict(layout="every other token", type=F32),
}


@pytest.mark.parametrize("name", CASES)
def test_forward(name):
    s, _ = make(**CASES[name])
    out, last = sx.causal_conv(return_state=True, **s)
    ref, want = os_.causal_conv(**host(s))
    size, _ = os_.causal_conv(size=True, **host(s))
    close("out", out, ref, size, s["weight"].shape[1] + 9)
    assert np.array_equal(_np(last), want)
    assert torch.equal(out, sx.causal_conv(**s))


@pytest.mark.parametrize("name", CASES)
def test_backward(name):
    s, g = make(**CASES[name])
    got = sx.causal_conv_backward(**s, **g)
    ref, size = (os_.causal_conv_vjp(**host(s), **host(g), size=z) for z in (False, True))
    k, n = s["weight"].shape[1], s["x"].shape[0] * s["x"].shape[1]
    for i, what in enumerate(("grad_x", "grad_weight", "grad_bias", "grad_initial")):
        if got[i] is None:
            assert what == "grad_bias" and s["bias"] is None
            continue
        close(what, got[i], ref[i], size[i], 2 * k + 20 + (8 * np.sqrt(n) if i in (1, 2) else 0))


def make_step(b=3, pool=5, d=72, k=4, type=BF, act="silu", slots="some", seed=0):
    gen = torch.Generator().manual_seed(2100 + seed)
    r = lambda *shape: torch.randn(*shape, generator=gen)  # noqa: E731
    s = dict(x=r(b, d).to(type).to(DEV), weight=r(d, k).to(DEV), state=r(pool, k - 1, d).to(type).to(DEV),
             bias=r(d).to(DEV), activation=act, slots=None)
    if slots == "some":
        at = torch.randperm(pool, generator=gen)[:b].to(torch.int32)
        at[b // 2] = -1 if b > 1 else at[0]
        s["slots"] = at.to(DEV)
    elif slots == "outside":
        s["slots"] = torch.tensor([pool, -2, 1 << 30][:b], dtype=torch.int32, device=DEV)
    return s


@pytest.mark.parametrize("name,kwargs", [
    ("ordinary", dict()), ("f32", dict(type=F32)), ("one request", dict(b=1, pool=1, slots=None)),
    ("no slots", dict(slots=None)), ("all idle", dict(slots="outside")), ("one tap", dict(k=1)),
    ("two taps f32", dict(k=2, type=F32, act=None)), ("eight taps", dict(k=8, d=40)), ("odd", dict(d=333)),
    ("odd f32", dict(d=51, type=F32)), ("one channel", dict(d=1)), ("many", dict(b=128, pool=144, d=4096)),
])
def test_step(name, kwargs):
    s = make_step(**kwargs)
    h = host(s)
    if h["slots"] is not None:
        h["slots"] = h["slots"].astype(np.int64)
    ref, want = os_.causal_conv_step(**h)
    size, _ = os_.causal_conv_step(**{**{n: np.abs(v) if isinstance(v, np.ndarray) and n != "slots" else v
                                         for n, v in h.items()}, "activation": None})
    out = sx.causal_conv_step(**s)
    close("out", out, ref, size, s["weight"].shape[1] + 9)
    assert np.array_equal(_np(s["state"]), want)


def test_steps_follow_the_prompt():
    s, _ = make(b=2, t=40, d=96, type=F32, initial=True)
    whole = sx.causal_conv(**s)
    head = dict(s, x=s["x"][:, :30])
    out, state = sx.causal_conv(return_state=True, **head)
    assert torch.equal(out, whole[:, :30])
    for t in range(30, 40):
        one = sx.causal_conv_step(s["x"][:, t], s["weight"], state, bias=s["bias"], activation=s["activation"])
        assert torch.equal(one, whole[:, t])


def test_a_pool_of_views_and_what_lies_between():
    room = torch.randn(4, 5, 40, device=DEV)
    kept, state = room.clone(), room[:, 1:4]
    s = make_step(b=4, pool=4, d=40, type=F32, slots=None)
    alone = state.clone()
    got = sx.causal_conv_step(s["x"], s["weight"], state, bias=s["bias"])
    assert torch.equal(got, sx.causal_conv_step(s["x"], s["weight"], alone, bias=s["bias"])) and torch.equal(state, alone)
    kept[:, 1:4] = state
    assert torch.equal(room, kept)


@pytest.mark.parametrize("type", [BF, F32])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_what_does_not_exist_is_not_read(type, value):
    s, g = make(b=3, t=70, lengths=[70, 0, 33], type=type, initial=True)
    want = (*sx.causal_conv(return_state=True, **s), *sx.causal_conv_backward(**s, **g))
    for x in (s["x"], g["grad_out"]):
        x[1], x[2, 33:] = value, value
    got = (*sx.causal_conv(return_state=True, **s), *sx.causal_conv_backward(**s, **g))
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert not want[0][1].any() and not want[0][2, 33:].any() and not want[2][1].any() and not want[2][2, 33:].any()


@pytest.mark.parametrize("type", [BF, F32])
def test_a_nan_stays_in_its_channel_and_window(type):
    s, _ = make(b=1, t=50, d=24, type=type)
    clean = sx.causal_conv(**s)
    s["x"][0, 20, 7] = float("nan")
    out = sx.causal_conv(**s)
    bad = torch.zeros_like(out, dtype=torch.bool)
    bad[0, 20:24, 7] = True
    assert torch.equal(torch.isnan(out), bad) and torch.equal(out[~bad], clean[~bad])


def test_no_tokens_and_no_rows():
    s, g = make(b=2, t=0, initial=True, type=F32)
    out, last = sx.causal_conv(return_state=True, **s)
    assert out.shape == (2, 0, 72) and torch.equal(last, s["initial"])
    gx, gw, gb, gi = sx.causal_conv_backward(**s, **g)
    assert gx.shape == (2, 0, 72) and not gw.any() and not gb.any() and torch.equal(gi, g["grad_state"])
    s, g = make(b=0, t=5, type=F32)
    assert sx.causal_conv(**s).shape == (0, 5, 72)
    gx, gw, gb, gi = sx.causal_conv_backward(**s, **g)
    assert not gw.any() and not gb.any()


def test_autograd_gives_the_backward_call():
    s, g = make(t=40, type=F32, initial=True, lengths=[40, 11])
    leaves = {n: s[n].clone().requires_grad_() for n in ("x", "weight", "bias", "initial")}
    out, last = sx.causal_conv(return_state=True, **{**s, **leaves})
    torch.autograd.backward([out, last], [g["grad_out"], g["grad_state"]])
    for a, n in zip(sx.causal_conv_backward(**s, **g), leaves):
        assert torch.equal(leaves[n].grad, a)
    out, last = sx.causal_conv(return_state=True, **{**s, "x": leaves["x"]})
    leaves["x"].grad = None
    last.backward(g["grad_state"])  # the state alone
    want = sx.causal_conv_backward(**s, grad_out=torch.zeros_like(g["grad_out"]), grad_state=g["grad_state"])
    assert torch.equal(leaves["x"].grad, want[0])


@pytest.mark.parametrize("act", [None, "silu"])
def test_gradient_matches_differences_of_the_forward_call(act):
    s, g = make(b=2, t=30, d=20, k=3, type=F32, initial=True, act=act, lengths=[30, 17])
    grads = sx.causal_conv_backward(**s, **g)
    gen = torch.Generator().manual_seed(5)
    loss = lambda q: sum((a.double() * b.double()).sum().item()  # noqa: E731
                         for a, b in zip(sx.causal_conv(return_state=True, **q), (g["grad_out"], g["grad_state"])))
    for n, grad in zip(("x", "weight", "bias", "initial"), grads):
        step = torch.randn(s[n].shape, generator=gen).to(DEV)
        e = 1e-2
        d = (loss({**s, n: s[n] + e * step}) - loss({**s, n: s[n] - e * step})) / (2 * e)
        want = (grad.double() * step.double()).sum().item()
        # the third derivative's share e^2, and f32 roundings of 2 x 30 x 20 values over 2 e
        assert abs(d - want) <= 2e-3 * abs(want) + 5e-3 * grad.double().norm().item(), n


def test_far_apart_rows():
    # rows whose offsets pass 2^31 elements
    t, d, far = 20, 16, (1 << 31) + 24
    room = torch.empty(far + 4 * t * d, dtype=BF, device=DEV)
    x = room.as_strided((2, t, d), (far, d, 1))
    s, g = make(b=2, t=t, d=d, initial=True)
    x.copy_(s["x"])
    go = room.as_strided((2, t, d), (far, d, 1), t * d)
    go.copy_(g["grad_out"])
    want = (*sx.causal_conv(return_state=True, **s), *sx.causal_conv_backward(**s, **g))
    s["x"], g["grad_out"] = x, go
    for a, b in zip((*sx.causal_conv(return_state=True, **s), *sx.causal_conv_backward(**s, **g)), want):
        assert torch.equal(a, b)
