"""How the state-space operators are called: graphs and other streams, both ways into the library, values of any
truth, tensors that carry more than their numbers, states that are written in place."""

import numpy as np
import pytest
import torch
import torch.autograd.forward_ad as forward_ad

import scan_primitives_amd as sx
from scan_primitives_amd import _binding as B
from tests import test_causal_conv_gpu as conv
from tests import test_group_norm_gpu as norm
from tests import test_selective_scan_gpu as scan

pytestmark = pytest.mark.gpu
BF, F32, DEV = torch.bfloat16, torch.float32, "cuda:0"


def _calls(seed=0, type=F32):
    """Every prompt and gradient: functions without arguments, and the tensors they read."""
    c, cg = conv.make(t=90, initial=True, lengths=[90, 40], type=type, seed=seed)
    s, sg = scan.make(b=1, t=900, d=70, initial=True, type=type, seed=seed)
    r, rg = scan.make(b=3, t=50, d=64, g=2, lengths=[50, 0, 9], initial=True, type=type, seed=seed)
    n, ng = norm.make(shape=(500, 64), type=type, act="silu", seed=seed)
    m, mg = norm.make(shape=(2, 300, 48), type=type, act="silu", seed=seed)
    fs = [lambda: sx.causal_conv(return_state=True, **c), lambda: sx.causal_conv_backward(**c, **cg),
          lambda: sx.selective_scan(return_state=True, **s), lambda: sx.selective_scan_backward(**s, **sg),
          lambda: sx.selective_scan(return_state=True, **r), lambda: sx.selective_scan_backward(**r, **rg),
          lambda: (sx.group_norm(**n),), lambda: sx.group_norm_backward(grad_out=ng, **n),
          lambda: (sx.group_norm(**m),), lambda: sx.group_norm_backward(grad_out=mg, **m)]
    tensors = [v for d in (c, cg, s, sg, r, rg, n, m) for v in d.values() if isinstance(v, torch.Tensor)] + [ng, mg]
    return fs, tensors


def _all(fs):
    return [t for f in fs for t in f() if t is not None]


@pytest.mark.parametrize("type", [BF, F32])
def test_results_repeat(type):
    fs, _ = _calls(type=type)
    want = _all(fs)
    for _ in range(3):
        for a, b in zip(_all(fs), want):
            assert torch.equal(a, b)


def test_replays_of_a_graph_and_another_stream():
    fs, mine = _calls()
    gs, others = _calls(seed=7)
    eager, other = _all(fs), _all(gs)
    torch.cuda.synchronize()
    graph, second = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = _all(fs)
    with torch.cuda.graph(second):
        more = _all(gs)
    for i in range(4):
        _all(gs)
        torch.cuda.synchronize()
        for c in captured + more:
            c.zero_()
        if i == 2:  # the graph reads what its inputs hold when it is replayed
            for a, b in zip(mine, others):
                a.copy_(b)
        graph.replay()
        second.replay()
        torch.cuda.synchronize()
        for c, e in zip(captured, other if i >= 2 else eager):
            assert torch.equal(c, e)
        for c, e in zip(more, other):
            assert torch.equal(c, e)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = _all(gs)
        at_once = _all(gs)
    here = _all(gs)  # at the same time, on this stream
    side.synchronize()
    torch.cuda.synchronize()
    for a, b, c, d in zip(got, at_once, here, other):
        assert torch.equal(a, d) and torch.equal(b, d) and torch.equal(c, d)


def test_replays_of_captured_steps_advance_the_states():
    c, e = conv.make_step(), conv.make_step()
    s, f = scan.make_step(), scan.make_step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = sx.causal_conv_step(**c), sx.selective_scan_step(**s)
    for _ in range(4):
        want = sx.causal_conv_step(**e), sx.selective_scan_step(**f)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
        assert torch.equal(c["state"], e["state"]) and torch.equal(s["state"], f["state"])


def _steps():
    c, s = conv.make_step(), scan.make_step()
    return [sx.causal_conv_step(**c), c["state"], sx.selective_scan_step(**s), s["state"]]


def test_every_call_without_the_bindings_extension(monkeypatch):
    fs, _ = _calls()
    want = _all(fs) + _steps()
    monkeypatch.setattr(B, "_marshal", B._LongWay())
    for a, b in zip(_all(fs) + _steps(), want):
        assert torch.equal(a, b)


def test_operands_that_have_to_be_converted():
    fs, _ = _calls()
    want = _all(fs)
    turned = lambda x: x.t().contiguous().t() if x.dim() == 2 else torch.stack([x, x], -1)[..., 0]  # noqa: E731
    c, cg = conv.make(t=90, initial=True, lengths=[90, 40], type=F32)
    s, sg = scan.make(b=1, t=900, d=70, initial=True, type=F32)
    n, ng = norm.make(shape=(500, 64), type=F32, act="silu")
    for d, names in ((c, ("weight", "bias", "initial", "lengths")), (s, ("a", "skip", "delta_bias", "initial")),
                     (n, ("weight", "bias"))):
        for k in names:
            d[k] = turned(d[k])
            assert not d[k].is_contiguous() or d[k].numel() == 1
    cg["grad_state"], sg["grad_state"] = turned(cg["grad_state"]), turned(sg["grad_state"])
    got = _all([lambda: sx.causal_conv(return_state=True, **c), lambda: sx.causal_conv_backward(**c, **cg),
                lambda: sx.selective_scan(return_state=True, **s), lambda: sx.selective_scan_backward(**s, **sg)])
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert torch.equal(sx.group_norm(**n), fs[6]()[0])


@pytest.mark.parametrize("true,false", [(1, 0), (np.bool_(True), np.bool_(False)), ("yes", "")])
def test_truth_values(true, false):
    c, _ = conv.make(t=20, initial=True)
    s, _ = scan.make(t=20, initial=True)
    for f, d in ((sx.causal_conv, c), (sx.selective_scan, s)):
        out, state = f(return_state=True, **d)
        got = f(return_state=true, **d)
        assert torch.equal(got[0], out) and torch.equal(got[1], state)
        assert torch.equal(f(return_state=false, **d), out)
    # (negative steps grow without end, to values that are not finite)
    same = lambda a, b: torch.testing.assert_close(a, b, rtol=0, atol=0, equal_nan=True)  # noqa: E731
    same(sx.selective_scan(**{**s, "softplus": true}), sx.selective_scan(**s))
    same(sx.selective_scan(**{**s, "softplus": false}), sx.selective_scan(**{**s, "softplus": False}))


@pytest.mark.parametrize("name", ["conv", "scan"])
@pytest.mark.parametrize("short", [True, False])
def test_states_that_autograd_knows(name, short, monkeypatch):
    if not short:
        monkeypatch.setattr(B, "_marshal", B._LongWay())
    make, step = (conv.make_step, sx.causal_conv_step) if name == "conv" else (scan.make_step, sx.selective_scan_step)
    s = make(type=F32)
    kept = s["state"].clone()
    s["state"].requires_grad_()
    with pytest.raises(sx.SxError) as e:
        step(**s)
    assert e.value.code == B.SX_E_UNSUPPORTED and torch.equal(s["state"], kept)
    with torch.no_grad():
        step(**s)
    assert not torch.equal(s["state"], kept)
    s = make(type=F32)
    before = s["state"]._version
    x = torch.ones_like(s["state"]).requires_grad_()
    loss = (x * s["state"]).sum()
    step(**s)
    assert s["state"]._version > before
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    s, e = make(type=F32), make(type=F32)
    with torch.inference_mode():
        s["state"] = s["state"].clone()
    assert torch.equal(step(**s), step(**e)) and torch.equal(s["state"], e["state"])


def test_tangents_are_refused():
    c, cg = conv.make(t=20, type=F32)
    s, sg = scan.make(t=20, type=F32)
    n, ng = norm.make(shape=(9, 16), type=F32)
    one, two = conv.make_step(type=F32), scan.make_step(type=F32)
    with forward_ad.dual_level():
        dual = lambda x: forward_ad.make_dual(x, torch.ones_like(x))  # noqa: E731
        calls = [lambda k=k: sx.causal_conv(**{**c, k: dual(c[k])}) for k in ("x", "weight", "bias")]
        calls += [lambda: sx.causal_conv_backward(**c, grad_out=dual(cg["grad_out"]))]
        calls += [lambda k=k: sx.selective_scan(**{**s, k: dual(s[k])})
                  for k in ("x", "delta", "a", "b", "c", "skip", "z", "delta_bias")]
        calls += [lambda: sx.selective_scan_backward(**s, grad_out=dual(sg["grad_out"]))]
        calls += [lambda k=k: sx.group_norm(**{**n, k: dual(n[k])}) for k in ("x", "weight", "bias")]
        calls += [lambda: sx.group_norm_backward(grad_out=dual(ng), **n)]
        calls += [lambda: sx.causal_conv_step(**{**one, "state": dual(one["state"])}),
                  lambda: sx.selective_scan_step(**{**two, "b": dual(two["b"])})]
        for i, call in enumerate(calls):
            with pytest.raises(sx.SxError) as e:
                call()
            assert e.value.code == B.SX_E_UNSUPPORTED, i


def _negated(x):
    """A lazily negated view with the values of x."""
    view = torch.complex(torch.zeros_like(x), -x).conj().imag
    assert view.is_neg() and torch.equal(view, x)
    return view


def test_lazily_negated_views_are_read_with_their_sign():
    c, cg = conv.make(t=40, type=F32, initial=True)
    s, sg = scan.make(t=40, type=F32, initial=True, d=24)
    n, ng = norm.make(shape=(9, 16), type=F32)
    for f, d in ((lambda q: sx.causal_conv_backward(**q), {**c, **cg}), (lambda q: [sx.causal_conv(**q)], c),
                 (lambda q: sx.selective_scan_backward(**q), {**s, **sg}), (lambda q: [sx.selective_scan(**q)], s),
                 (lambda q: sx.group_norm_backward(**q), {**n, "grad_out": ng}), (lambda q: [sx.group_norm(**q)], n)):
        want = f(d)
        for k, v in d.items():
            if isinstance(v, torch.Tensor) and v.dtype == F32:
                for a, b in zip(f({**d, k: _negated(v)}), want):
                    torch.testing.assert_close(a, b, rtol=1e-4, atol=1e-4, msg=k)
    for make, step in ((conv.make_step, sx.causal_conv_step), (scan.make_step, sx.selective_scan_step)):
        one = make(type=F32)
        with pytest.raises(sx.SxError) as e:
            step(**{**one, "state": _negated(one["state"])})
        assert e.value.code == B.SX_E_UNSUPPORTED


@pytest.mark.parametrize("call,code", [
    (lambda c, s, n: sx.causal_conv(**{**c, "weight": c["weight"].double()}), B.SX_E_DIM_002),
    (lambda c, s, n: sx.causal_conv(**{**c, "x": c["x"].half()}), B.SX_E_DIM_002),
    (lambda c, s, n: sx.causal_conv(**{**c, "weight": c["weight"][1:]}), B.SX_E_DIM_001),
    (lambda c, s, n: sx.causal_conv(**{**c, "bias": c["bias"][1:]}), B.SX_E_DIM_001),
    (lambda c, s, n: sx.causal_conv(**{**c, "weight": c["weight"][:, :0]}), B.SX_E_DIM_001),
    (lambda c, s, n: sx.causal_conv(**{**c, "initial": torch.zeros(2, 4, 72, device=DEV)}), B.SX_E_DIM_001),
    (lambda c, s, n: sx.causal_conv(**{**c, "lengths": torch.zeros(2, device=DEV)}), B.SX_E_DIM_002),
    (lambda c, s, n: sx.causal_conv(**{**c, "activation": "tanh"}), B.SX_E_UNSUPPORTED),
    (lambda c, s, n: sx.causal_conv(**{**c, "activation": 1}), B.SX_E_UNSUPPORTED),
    (lambda c, s, n: sx.causal_conv(**{**c, "x": c["x"][0]}), B.SX_E_DIM_001),
    (lambda c, s, n: sx.causal_conv(**{**c, "bias": c["bias"].cpu()}), B.SX_E_UNSUPPORTED),
    (lambda c, s, n: sx.causal_conv_backward(**c, grad_out=c["x"][:, 1:]), B.SX_E_DIM_001),
    (lambda c, s, n: sx.selective_scan(**{**s, "delta": s["delta"][:, 1:]}), B.SX_E_DIM_001),
    (lambda c, s, n: sx.selective_scan(**{**s, "delta": s["delta"].bfloat16()}), B.SX_E_DIM_002),
    (lambda c, s, n: sx.selective_scan(**{**s, "a": s["a"][:, 1:]}), B.SX_E_DIM_001),
    (lambda c, s, n: sx.selective_scan(**{**s, "a": s["a"].bfloat16()}), B.SX_E_DIM_002),
    (lambda c, s, n: sx.selective_scan(**{**s, "b": s["b"][:, :, 0]}), B.SX_E_DIM_001),
    (lambda c, s, n: sx.selective_scan(**{**s, "c": s["c"][:, :, :, 1:]}), B.SX_E_DIM_001),
    (lambda c, s, n: sx.selective_scan(**{**s, "z": s["z"][..., 1:]}), B.SX_E_DIM_001),
    (lambda c, s, n: sx.selective_scan(**{**s, "skip": s["skip"][1:]}), B.SX_E_DIM_001),
    (lambda c, s, n: sx.selective_scan(**{**s, "initial": s["x"]}), B.SX_E_DIM_001),
    (lambda c, s, n: sx.selective_scan_backward(**s, grad_out=s["x"].bfloat16()), B.SX_E_DIM_002),
    (lambda c, s, n: sx.group_norm(**{**n, "groups": 5}), B.SX_E_DIM_001),
    (lambda c, s, n: sx.group_norm(**{**n, "x": n["x"][0]}), B.SX_E_DIM_001),
    (lambda c, s, n: sx.group_norm(**{**n, "x": n["x"].half()}), B.SX_E_DIM_002),
    (lambda c, s, n: sx.group_norm(**{**n, "weight": n["weight"][1:]}), B.SX_E_DIM_001),
    (lambda c, s, n: sx.group_norm(**{**n, "eps": -1.0}), B.SX_E_DIM_001),
    (lambda c, s, n: sx.group_norm(**{**n, "activation": "relu"}), B.SX_E_UNSUPPORTED),
    (lambda c, s, n: sx.group_norm_backward(**n, grad_out=n["x"][1:]), B.SX_E_DIM_001),
])
def test_the_binding_refuses(call, code):
    c, s, n = conv.make(type=F32)[0], scan.make(type=F32)[0], norm.make(type=F32)[0]
    with pytest.raises(sx.SxError) as e:
        call(c, s, n)
    assert e.value.code == code, str(e.value)


def test_steps_refuse_pools_that_do_not_fit():
    c, s = conv.make_step(type=F32), scan.make_step(type=F32)
    for step, d in ((sx.causal_conv_step, c), (sx.selective_scan_step, s)):
        for state, code in ((d["state"][:, 1:], B.SX_E_DIM_001), (d["state"].double(), B.SX_E_DIM_002),
                            (d["state"].transpose(1, 2).contiguous().transpose(1, 2), B.SX_E_UNSUPPORTED),
                            (d["state"][:1].expand(4, -1, -1), B.SX_E_UNSUPPORTED), (d["state"][0], B.SX_E_DIM_001)):
            with pytest.raises(sx.SxError) as e:
                step(**{**d, "state": state})
            assert e.value.code == code, str(e.value)
        with pytest.raises(sx.SxError) as e:
            step(**{**d, "slots": None, "state": d["state"][:2]})
        assert e.value.code == B.SX_E_DIM_001
