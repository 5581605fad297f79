"""The selective scan on the GPU against the 64-bit oracle.

Tolerances, from the arithmetic. A state's term is multiplied by a decay a
token, whose exponential is off by at most one step of 2^-23, always to the same side
perhaps: 2 T 2^-24 of what the terms add up to (the oracle's `size`). The other
roundings (the sums and products of T tokens, N states, as many channels as share a
row, and B T tokens for what all add to: n of them) are independent: eight
standard deviations are 8 sqrt(n) 2^-24. Steps, gates and their slopes (softplus
and SiLU by a series and hardware's exponential and reciprocal) are off by at most 16
steps each; a rate's rounding enters as |sum of dt a| exp(sum of dt a), at most one more.
A decay below 2^-126 is zero in 32 bits: what it would have carried from the largest
state to the largest adjoint, of every token and state, is the gradients' floor.
bf16 results are rounded once: 2^-8 of themselves.
"""

import numpy as np
import pytest
import torch

import scan_primitives_amd as sx
from oracle import state_space as os_
from tests.test_causal_conv_gpu import BF, DEV, F32, _np, close, host

pytestmark = pytest.mark.gpu


def make(b=2, t=100, d=72, n=16, g=1, type=BF, gate=True, skip=True, bias=True, softplus=True, initial=False,
         lengths=None, layout="plain", steps="ordinary", seed=0):
    gen = torch.Generator().manual_seed(3000 + seed)
    r = lambda *shape: torch.randn(*shape, generator=gen)  # noqa: E731

    def laid(*shape):
        if layout == "slices":
            return r(*shape[:-1], 2 * shape[-1] + 1).to(type).to(DEV)[..., 1:shape[-1] + 1]
        if layout == "channels first":
            return r(shape[0], *shape[2:], shape[1]).to(type).to(DEV).movedim(-1, 1)
        if layout == "one row for all":
            return r(1, *shape[1:]).to(type).to(DEV).expand(*shape)
        if layout == "every other":
            return r(*shape[:-1], 2 * shape[-1]).to(type).to(DEV)[..., ::2]
        return r(*shape).to(type).to(DEV)

    delta = laid(b, t, d)
    if steps == "none":            # no step at all: softplus of -200 is zero in 32 bits
        delta = torch.full_like(delta, -200.0)
    elif steps == "large":         # a state forgets at once
        delta = delta * 4 + 30
    elif steps == "small":
        delta = delta * 0.1 - 9
    s = dict(x=laid(b, t, d), delta=delta, a=-torch.rand(d, n, generator=gen).mul(4).exp().to(DEV), b=laid(b, t, g, n),
             c=laid(b, t, g, n), skip=r(d).to(DEV) if skip else None, z=laid(b, t, d) if gate else None,
             delta_bias=(r(d) - 3).to(DEV) if bias else None, softplus=softplus,
             initial=r(b, d, n).to(DEV) if initial else None,
             lengths=None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device=DEV))
    if not softplus:
        s["delta"] = (s["delta"].abs() * 0.1).to(type)
        s["delta_bias"] = s["delta_bias"].abs() * 0.01 if bias else None
    return s, dict(grad_out=laid(b, t, d), grad_state=r(b, d, n).to(DEV) if initial else None)


CASES = {
    "ordinary": dict(),
    "f32": dict(type=F32, initial=True),
    "one token": dict(t=1, initial=True),
    "one token f32": dict(t=1, type=F32, d=3, n=1),
    "two tokens": dict(t=2, initial=True, lengths=[2, 1]),
    "eight tokens": dict(t=8, type=F32),
    "nine tokens": dict(t=9, initial=True),
    "fifteen tokens": dict(t=15),
    "sixteen tokens": dict(t=16, type=F32),
    "seventeen tokens": dict(t=17, initial=True, lengths=[17, 16]),
    "one state": dict(n=1, type=F32),
    "three states": dict(n=3, initial=True),
    "four states": dict(n=4, type=F32),
    "five states": dict(n=5),
    "eight states": dict(n=8, initial=True),
    "twelve states": dict(n=12, type=F32, initial=True),
    "seventeen states": dict(n=17, initial=True),
    "thirty-two states": dict(n=32, type=F32, initial=True),
    "thirty-two states bf16": dict(n=32, t=260, lengths=[260, 13]),
    "one channel": dict(d=1, type=F32),
    "odd channels": dict(d=77, initial=True),
    "a channel more than a block": dict(d=65, type=F32),
    "a channel more than two blocks": dict(d=129),
    "whole blocks": dict(d=256, type=F32),
    "four channels more than a block": dict(d=68, t=40),
    "five channels more than a block": dict(d=69, t=40, type=F32, initial=True),
    "three channels more than two blocks": dict(d=131, t=40, initial=True),
    "five channels more than two blocks": dict(d=133, t=300, type=F32),
    "seventy channels a group": dict(d=210, g=3, t=50, initial=True),
    "five channels": dict(d=5, t=33),
    "eleven states": dict(n=11, t=60, d=70, initial=True),
    "ten states, many segments": dict(b=1, n=10, t=700, d=66, initial=True),
    "groups": dict(d=96, g=3, initial=True),
    "groups of odd sizes": dict(d=99, g=3, type=F32, initial=True),
    "a group a channel": dict(d=12, g=12, type=F32, n=6),
    "groups over blocks": dict(d=400, g=2, n=8),
    "ragged": dict(b=5, t=130, lengths=[130, 0, 1, 77, 64], initial=True),
    "ragged f32": dict(b=3, t=300, lengths=[300, 0, 155], type=F32, initial=True, gate=False),
    "lengths out of range": dict(b=3, t=40, lengths=[-5, 99, 40]),
    "segments": dict(b=1, t=1500, initial=True),
    "segments f32": dict(b=1, t=1111, d=33, type=F32, initial=True),
    "segments, ragged": dict(b=3, t=1300, d=40, lengths=[1300, 5, 700], initial=True, n=8),
    "segments, no gate": dict(b=1, t=700, d=130, gate=False, type=F32, n=4),
    "segments of many states": dict(b=1, t=600, d=24, n=29, g=2, initial=True),
    "no gate": dict(gate=False),
    "nothing optional": dict(gate=False, skip=False, bias=False, type=F32),
    "no softplus": dict(softplus=False, type=F32, initial=True),
    "no softplus, no bias": dict(softplus=False, bias=False),
    "no steps": dict(steps="none", initial=True, type=F32),
    "large steps": dict(steps="large", initial=True, type=F32),
    "small steps": dict(steps="small", initial=True, t=300, type=F32),
    "slices": dict(layout="slices", initial=True),
    "slices f32": dict(layout="slices", type=F32, d=64),
    "channels first": dict(layout="channels first", initial=True),
    "channels first f32": dict(layout="channels first", type=F32, g=2),
    "one row for all": dict(layout="one row for all", type=F32),
    "every other": dict(layout="every other"),
}


def _floor(s, g):
    most = lambda x: 0.0 if x is None or x.numel() == 0 else x.double().abs().max().item()  # noqa: E731
    b, t, _ = s["x"].shape
    v = most(s["delta"]) + most(s["delta_bias"])
    dt = v + 1.0  # softplus(v) <= |v| + 1
    h = most(s["initial"]) + t * dt * most(s["x"]) * most(s["b"])
    lam = most(g["grad_state"]) + t * most(g["grad_out"]) * (most(s["z"]) + 1.0) * most(s["c"])
    return 2.0 ** -126 * b * t * s["a"].shape[1] * dt * max(1.0, most(s["a"])) * h * lam


def _steps(s, tokens=False, rows=False):
    b, t, d = s["x"].shape
    n = 6 * t + s["a"].shape[1] + 64 + (b * t if tokens else 0) + (d // s["b"].shape[2] if rows else 0)
    return 2 * t + 8 * np.sqrt(n) + 50


@pytest.mark.parametrize("name", CASES)
def test_forward(name):
    s, _ = make(**CASES[name])
    out, last = sx.selective_scan(return_state=True, **s)
    (ref, want), (size, sstate) = (os_.selective_scan(size=z, **host(s)) for z in (False, True))
    close("out", out, ref, size, _steps(s))
    close("last state", last, want, sstate, _steps(s))
    assert torch.equal(out, sx.selective_scan(**s))


NAMES = ("grad_x", "grad_delta", "grad_a", "grad_b", "grad_c", "grad_skip", "grad_z", "grad_delta_bias", "grad_initial")


@pytest.mark.parametrize("name", CASES)
def test_backward(name):
    s, g = make(**CASES[name])
    got = sx.selective_scan_backward(**s, **g)
    ref, size = (os_.selective_scan_vjp(size=z, **host(s), **host(g)) for z in (False, True))
    for i, what in enumerate(NAMES):
        if got[i] is None:
            assert s[{"grad_skip": "skip", "grad_z": "z", "grad_delta_bias": "delta_bias"}[what]] is None
            continue
        close(what, got[i], ref[i], size[i], 2 * _steps(s, tokens=what in ("grad_a", "grad_skip", "grad_delta_bias"),
                                                        rows=what in ("grad_b", "grad_c")),
              floor=_floor(s, g))


def make_step(b=3, pool=5, d=72, n=16, g=1, type=BF, gate=True, slots="some", softplus=True, seed=0):
    s, _ = make(b=b, t=1, d=d, n=n, g=g, type=type, gate=gate, softplus=softplus, seed=seed)
    gen = torch.Generator().manual_seed(3100 + seed)
    s = {k: (v[:, 0] if k in ("x", "delta", "b", "c", "z") and v is not None else v) for k, v in s.items()
         if k not in ("initial", "lengths")}
    s["state"] = torch.randn(pool, d, n, generator=gen).to(DEV)
    s["slots"] = None
    if slots == "some":
        at = torch.randperm(pool, generator=gen)[:b].to(torch.int32)
        at[b // 2] = -1 if b > 1 else at[0]
        s["slots"] = at.to(DEV)
    elif slots == "outside":
        s["slots"] = torch.tensor([pool, -2, 1 << 30][:b], dtype=torch.int32, device=DEV)
    return s


@pytest.mark.parametrize("name,kwargs", [
    ("ordinary", dict()), ("f32", dict(type=F32)), ("one request", dict(b=1, pool=1, slots=None)),
    ("no slots", dict(slots=None)), ("all idle", dict(slots="outside")), ("one state", dict(n=1, type=F32)),
    ("three states", dict(n=3)), ("four states", dict(n=4)), ("six states", dict(n=6, type=F32)), ("eight states", dict(n=8)),
    ("thirteen states", dict(n=13)), ("twenty states", dict(n=20, type=F32)), ("thirty-two states", dict(n=32)),
    ("groups", dict(d=96, g=3)), ("odd channels", dict(d=77, type=F32)), ("one channel", dict(d=1)),
    ("no gate", dict(gate=False)), ("no softplus", dict(softplus=False, type=F32)),
    ("many", dict(b=128, pool=144, d=1024)),
])
def test_step(name, kwargs):
    s = make_step(**kwargs)
    h = host(s)
    if h["slots"] is not None:
        h["slots"] = h["slots"].astype(np.int64)
    (ref, want), (size, sstate) = (os_.selective_scan_step(size=z, **h) for z in (False, True))
    out = sx.selective_scan_step(**s)
    close("out", out, ref, size, 150)
    close("state", s["state"], want, sstate, 100)


def test_steps_follow_the_prompt():
    s, _ = make(b=2, t=80, d=96, type=F32, initial=True)
    (whole, last), size = sx.selective_scan(return_state=True, **s), os_.selective_scan(size=True, **host(s))
    tokens = ("x", "delta", "b", "c", "z")
    _, state = sx.selective_scan(return_state=True, **{k: (v[:, :64] if k in tokens else v) for k, v in s.items()})
    for t in range(64, 80):
        one = {k: (v[:, t] if k in tokens else v) for k, v in s.items() if k not in ("initial", "lengths")}
        out = sx.selective_scan_step(state=state, **one)
        close(f"token {t}", out, _np(whole[:, t]), size[0][:, t], 2 * _steps(s))
    close("state", state, _np(last), size[1], 2 * _steps(s))


def test_a_pool_of_views_and_what_lies_between():
    for room in (torch.randn(4, 41, 16, device=DEV), torch.randn(4, 42, 16, device=DEV)):
        for off in (0, 1):
            state = room[:, off:40 + off]
            s = make_step(b=4, pool=4, d=40, type=F32, slots=None)
            kept, alone = room.clone(), state.clone()
            got = sx.selective_scan_step(**{**s, "state": state})
            assert torch.equal(got, sx.selective_scan_step(**{**s, "state": alone})) and torch.equal(state, alone)
            kept[:, off:40 + off] = state
            assert torch.equal(room, kept)
    flat = torch.randn(4 * 640 + 3, device=DEV)  # states off 16-byte borders
    state = flat[1:4 * 640 + 1].view(4, 40, 16)
    s = make_step(b=4, pool=4, d=40, type=F32, slots=None)
    alone = state.clone()
    assert state.data_ptr() % 16
    assert torch.equal(sx.selective_scan_step(**{**s, "state": state}), sx.selective_scan_step(**{**s, "state": alone}))
    assert torch.equal(state, alone)


@pytest.mark.parametrize("type", [BF, F32])
@pytest.mark.parametrize("t", [70, 900])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_what_does_not_exist_is_not_read(type, t, value):
    s, g = make(b=3, t=t, lengths=[t, 0, 33], type=type, initial=True, d=40)
    want = (*sx.selective_scan(return_state=True, **s), *sx.selective_scan_backward(**s, **g))
    for x in (s["x"], s["delta"], s["b"], s["c"], s["z"], g["grad_out"]):
        x[1], x[2, 33:] = value, value
    got = (*sx.selective_scan(return_state=True, **s), *sx.selective_scan_backward(**s, **g))
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert torch.equal(want[1][1], s["initial"][1]) and torch.equal(want[10][1], g["grad_state"][1])
    for i in (0, 2, 3, 5, 6, 8):
        assert not want[i][1].any() and not want[i][2, 33:].any()


@pytest.mark.parametrize("t,at", [(50, 20), (900, 500)])
@pytest.mark.parametrize("name", ["x", "delta", "z", "b", "c", "initial"])
def test_infinities_reach_no_earlier_token_and_no_other_channel(t, at, name):
    s, _ = make(b=2, t=t, d=80, g=2, type=F32, initial=True)
    clean, state = sx.selective_scan(return_state=True, **s)
    if name == "initial":
        at = 0
        s[name][0, 7, 3] = float("inf")
    elif name in ("b", "c"):
        s[name][0, at, 0, 3] = float("inf")
    else:
        s[name][0, at, 7] = float("nan")
    out, last = sx.selective_scan(return_state=True, **s)
    hit = slice(0, 40) if name in ("b", "c") else slice(7, 8)
    same = torch.ones_like(out, dtype=torch.bool)
    same[0, at:, hit] = False
    assert torch.equal(out[same], clean[same])
    if name in ("x", "delta", "z"):
        assert torch.isnan(out[0, at, 7])
    states = torch.ones_like(state, dtype=torch.bool)
    states[0, hit] = False
    assert torch.equal(last[states], state[states])
    if name in ("z", "c"):
        assert torch.equal(last, state) and torch.equal(out[0, at + 1:], clean[0, at + 1:])


def test_no_tokens_and_no_rows():
    s, g = make(b=2, t=0, initial=True, type=F32)
    out, last = sx.selective_scan(return_state=True, **s)
    assert out.shape == (2, 0, 72) and torch.equal(last, s["initial"])
    got = sx.selective_scan_backward(**s, **g)
    assert not got[2].any() and not got[5].any() and not got[7].any() and torch.equal(got[8], g["grad_state"])
    s, g = make(b=0, t=5, type=F32)
    assert sx.selective_scan(**s).shape == (0, 5, 72)
    got = sx.selective_scan_backward(**s, **g)
    assert not got[2].any() and not got[5].any() and not got[7].any()


def test_autograd_gives_the_backward_call():
    s, g = make(t=40, d=48, g=2, type=F32, initial=True, lengths=[40, 11])
    names = ("x", "delta", "a", "b", "c", "skip", "z", "delta_bias", "initial")
    leaves = {n: s[n].clone().requires_grad_() for n in names}
    out, last = sx.selective_scan(return_state=True, **{**s, **leaves})
    torch.autograd.backward([out, last], [g["grad_out"], g["grad_state"]])
    for a, n in zip(sx.selective_scan_backward(**s, **g), names):
        assert torch.equal(leaves[n].grad, a), n
    # the state alone, and of two operands
    two = {n: s[n].clone().requires_grad_() for n in ("a", "b")}
    _, last = sx.selective_scan(return_state=True, **{**s, **two})
    last.backward(g["grad_state"])
    want = sx.selective_scan_backward(**s, grad_out=torch.zeros_like(g["grad_out"]), grad_state=g["grad_state"])
    assert torch.equal(two["a"].grad, want[2]) and torch.equal(two["b"].grad, want[3])


@pytest.mark.parametrize("t,gate,softplus", [(30, True, True), (600, False, True), (20, True, False)])
def test_gradient_matches_differences_of_the_forward_call(t, gate, softplus):
    s, g = make(b=2, t=t, d=12, n=6, g=2, type=F32, initial=True, lengths=[t, 17], gate=gate, softplus=softplus)
    grads = sx.selective_scan_backward(**s, **g)
    gen = torch.Generator().manual_seed(5)
    loss = lambda q: sum((a.double() * b.double()).sum().item()  # noqa: E731
                         for a, b in zip(sx.selective_scan(return_state=True, **q), (g["grad_out"], g["grad_state"])))
    for n, grad in zip(("x", "delta", "a", "b", "c", "skip", "z", "delta_bias", "initial"), grads):
        if grad is None:
            continue
        step = torch.randn(s[n].shape, generator=gen).to(DEV)
        e = 3e-3
        d = (loss({**s, n: s[n] + e * step}) - loss({**s, n: s[n] - e * step})) / (2 * e)
        want = (grad.double() * step.double()).sum().item()
        # the third derivative's share e^2 times a few, and f32 roundings of 2 t 12 values over 2 e
        assert abs(d - want) <= 5e-3 * abs(want) + 1e-2 * grad.double().norm().item(), n


def test_far_apart_tokens():
    # tokens 2^24 elements apart: offsets within a tile pass what its 32-bit ones are used for
    t, d, far = 18, 16, 1 << 24
    s, g = make(b=1, t=t, d=d, initial=True)
    want = (*sx.selective_scan(return_state=True, **s), *sx.selective_scan_backward(**s, **g))
    room = torch.zeros(t * far + 64, dtype=BF, device=DEV)
    for i, (where, n) in enumerate(((s, "x"), (s, "delta"), (s, "z"), (g, "grad_out"), (s, "b"), (s, "c"))):
        view = room.as_strided(where[n].shape, (0, far, *where[n].stride()[2:]), i * 32)
        view.copy_(where[n])
        where[n] = view
    for a, b in zip((*sx.selective_scan(return_state=True, **s), *sx.selective_scan_backward(**s, **g)), want):
        assert torch.equal(a, b)


def test_far_apart_rows_and_a_pool_past_32_bits():
    t, d, far = 20, 16, (1 << 31) + 24
    s, g = make(b=2, t=t, d=d, initial=True)
    want = (*sx.selective_scan(return_state=True, **s), *sx.selective_scan_backward(**s, **g))
    room = torch.empty(far + 8 * t * d, dtype=BF, device=DEV)
    for i, (where, n) in enumerate(((s, "x"), (s, "delta"), (s, "z"), (g, "grad_out"), (s, "b"), (s, "c"))):
        v = where[n]
        view = room.as_strided(v.shape, (far, *v.stride()[1:]), i * t * d)
        view.copy_(v)
        where[n] = view
    for a, b in zip((*sx.selective_scan(return_state=True, **s), *sx.selective_scan_backward(**s, **g)), want):
        assert torch.equal(a, b)
    del room
    one = make_step(b=2, pool=2, d=64, type=F32, slots=None)
    small = one["state"].clone()
    want = sx.selective_scan_step(**{**one, "state": small})
    slots = (1 << 31) // (64 * 16) + 5  # states whose offsets pass 2^31 elements
    pool = torch.zeros(slots, 64, 16, device=DEV)
    at = torch.tensor([slots - 1, 3], dtype=torch.int32, device=DEV)
    pool[at.long()] = one["state"]
    got = sx.selective_scan_step(**{**one, "state": pool, "slots": at})
    assert torch.equal(got, want) and torch.equal(pool[at.long()], small)
