"""Decay attention on the GPU against the 64-bit oracle.

Tolerances, from the arithmetic: a result is a sum of at most T dk products in
32 bits, and a term meets at most n = T + dk + 64 roundings on its way (the
running sums of a chunk, the states' products with the decays). They are
independent, so eight of their standard deviations are 8 sqrt(n) 2^-24 of what
the terms add up to before they cancel (the oracle's `size`). With bf16
operands two products (scores with values, rows with the state) may take their
32-bit operand in parts that carry 14 bits at least: 2 x 2^-14 of the same
size; and the result is rounded to bf16 once: 2^-8 of itself. States and the
decay's gradient stay in f32 with all their bits. The decay's gradient may be
formed from differences of sums of q . grad_q and k . grad_k over a chunk of
64 tokens: its size is that of the largest such sum.
"""

import numpy as np
import pytest
import torch

import scan_primitives_amd as sx
from oracle import attention as oa

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def _np(x):
    return None if x is None else x.detach().double().cpu().numpy()


def _close(name, got, ref, size, n, bf16, floor=None):
    got = _np(got)
    assert got.shape == ref.shape, name
    assert np.isfinite(got).all(), f"{name}: not finite"
    tol = 8.0 * np.sqrt(n) * 2.0 ** -24 * size
    if floor is not None:
        tol = tol + 8.0 * np.sqrt(n) * 2.0 ** -24 * floor
    if bf16:
        tol = tol + 2.0 ** -13 * size + 2.0 ** -8 * np.abs(ref)
    over = np.abs(got - ref) - tol
    if over.size and over.max() > 1e-37:
        at = np.unravel_index(np.argmax(over), over.shape)
        raise AssertionError(f"{name} at {at}: got {got[at]!r}, ref {ref[at]!r}, tolerance {tol[at]!r}")


def _rand(gen, *shape):
    return torch.randn(*shape, generator=gen)


def make(b=2, t=100, h=4, hq=None, hk=None, hv=None, dk=32, dv=32, type=BF, decay="token", initial=False, lengths=None,
         layout="plain", seed=0):
    gen = torch.Generator().manual_seed(1000 + seed)
    hq, hk, hv = hq or h, hk or hq or h, hv or h

    def laid(heads, d):
        if layout == "heads first":       # [B, heads, T, d] seen as [B, T, heads, d]
            return _rand(gen, b, heads, t, d).to(type).to(DEV).transpose(1, 2)
        if layout == "every other":       # element stride 2
            return _rand(gen, b, t, heads, 2 * d).to(type).to(DEV)[..., ::2]
        if layout == "odd offset":        # rows that start off any 16-byte border
            return _rand(gen, b, t, heads, d + 3).to(type).to(DEV)[..., 1:d + 1]
        if layout == "broadcast":         # one batch row for all
            return _rand(gen, 1, t, heads, d).to(type).to(DEV).expand(b, t, heads, d)
        return _rand(gen, b, t, heads, d).to(type).to(DEV)

    s = dict(q=laid(hq, dk), k=laid(hk, dk), v=laid(hv, dv), scale=dk ** -0.5)
    base = torch.log1p(-torch.exp2(-1.0 - 7.0 * torch.rand(h, generator=gen)))
    g = base if decay == "head" else base * (0.25 + 1.5 * torch.rand(b, t, h, generator=gen))
    if decay == "none":
        g = torch.zeros(b, t, h)
    elif decay == "cuts":
        g = torch.where(torch.rand(b, t, 1, generator=gen) < 0.1, torch.full_like(g, -float("inf")), g)
    elif decay == "all cut":
        g = torch.full((b, t, h), -float("inf"))
    elif decay == "lowest":
        g = torch.where(torch.rand(b, t, h, generator=gen) < 0.1, torch.full_like(g, torch.finfo(F32).min), g)
    elif decay == "growing":
        g = torch.full((b, t, h), 0.01)
    elif decay == "strong":
        g = -40.0 * torch.rand(b, t, h, generator=gen)
    s["g"] = g.to(DEV)
    if layout == "heads first" and s["g"].dim() == 3:
        s["g"] = s["g"].transpose(1, 2).contiguous().transpose(1, 2)
    s["initial"] = _rand(gen, b, h, dk, dv).to(DEV) if initial else None
    s["lengths"] = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device=DEV)
    s["go"] = _rand(gen, b, t, h, dv).to(type).to(DEV)
    s["gs"] = _rand(gen, b, h, dk, dv).to(DEV)
    return s


def _lengths(s):
    return None if s["lengths"] is None else np.clip(_np(s["lengths"]), 0, s["q"].shape[1])


def _oracle(s, size=False):
    return oa.decay_attention(_np(s["q"]), _np(s["k"]), _np(s["v"]), _np(s["g"]), _np(s["initial"]), _lengths(s),
                              s["scale"], size=size)


def _oracle_vjp(s, grad_state=True, size=False):
    return oa.decay_attention_vjp(_np(s["q"]), _np(s["k"]), _np(s["v"]), _np(s["g"]), _np(s["go"]), _np(s["initial"]),
                                  _lengths(s), s["scale"], _np(s["gs"]) if grad_state else None, size=size)


def _forward(s):
    return sx.decay_attention(s["q"], s["k"], s["v"], s["g"], initial=s["initial"], lengths=s["lengths"],
                              scale=s["scale"], return_state=True)


def _backward(s, grad_state=True):
    return sx.decay_attention_backward(s["q"], s["k"], s["v"], s["g"], s["go"], initial=s["initial"],
                                       lengths=s["lengths"], scale=s["scale"],
                                       grad_state=s["gs"] if grad_state else None)


def _roundings(s):
    return s["q"].shape[1] + s["q"].shape[-1] + s["v"].shape[-1] + 64


def check_forward(s):
    out, last = _forward(s)
    ref, size = _oracle(s), _oracle(s, size=True)
    bf16 = s["q"].dtype == BF
    assert out.dtype == s["q"].dtype and last.dtype == F32
    _close("out", out, ref[0], size[0], _roundings(s), bf16)
    _close("last state", last, ref[1], size[1], _roundings(s), False)


def check_backward(s, grad_state=True):
    got = _backward(s, grad_state)
    ref, size = _oracle_vjp(s, grad_state), _oracle_vjp(s, grad_state, size=True)
    bf16, n = s["q"].dtype == BF, _roundings(s)
    for name, i in (("grad_q", 0), ("grad_k", 1), ("grad_v", 2)):
        assert got[i].dtype == s["q"].dtype
        _close(name, got[i], ref[i], size[i], n, bf16)
    h = s["g"].shape[-1]
    wide = lambda x: np.abs(np.repeat(_np(x), h // x.shape[2], axis=2))  # noqa: E731
    per = lambda x: np.repeat(x, h // x.shape[2], axis=2)  # noqa: E731
    mass = (wide(s["q"]) * per(size[0])).sum(-1) + (wide(s["k"]) * per(size[1])).sum(-1)
    mass = np.where(np.isfinite(mass), mass, 0.0)
    live = np.arange(mass.shape[1])[None, :, None] < (np.full(mass.shape[0], mass.shape[1]) if s["lengths"] is None else
                                                      _lengths(s))[:, None, None]
    mass = np.where(live, mass, 0.0)
    floor = 64.0 * mass.max(initial=0.0)
    if s["g"].dim() == 1:
        floor = floor * np.sqrt(max(mass.shape[0] * mass.shape[1], 1))
    _close("grad_log_decay", got[3], ref[3], size[3], n, False, floor=floor)
    _close("grad_initial", got[4], ref[4], size[4], n, False)


SHAPES = {
    "one token": dict(t=1),
    "one token f32": dict(t=1, type=F32, initial=True),
    "two tokens, one head, width one": dict(b=1, t=2, h=1, dk=1, dv=1, initial=True),
    "a chunk less one": dict(t=63, dk=64, dv=64),
    "a chunk": dict(t=64, dk=64, dv=64, initial=True),
    "a chunk and one": dict(t=65, dk=64, dv=64),
    "f32 a chunk and one": dict(t=33, dk=64, dv=64, type=F32),
    "segments": dict(b=1, t=1000, h=2, dk=64, dv=64, initial=True),
    "segments f32": dict(b=1, t=500, h=2, dk=64, dv=64, type=F32, initial=True),
    "segments, wide": dict(b=1, t=515, h=1, dk=128, dv=128),
    "odd widths": dict(dk=33, dv=47, initial=True),
    "odd widths f32": dict(dk=129, dv=17, type=F32, initial=True),
    "narrow keys, wide values": dict(dk=5, dv=130),
    "widest": dict(b=1, t=130, h=2, dk=256, dv=256, initial=True),
    "widest f32": dict(b=1, t=70, h=2, dk=256, dv=200, type=F32, initial=True),
    "128 f32": dict(b=1, t=150, h=2, dk=128, dv=128, type=F32, initial=True),
    "shared heads": dict(h=6, hq=2, hk=3, hv=1, dk=24, dv=40, initial=True),
    "shared heads f32": dict(h=6, hq=1, hk=6, hv=2, dk=24, dv=40, type=F32),
    "one decay a head": dict(decay="head", t=300, initial=True),
    "no decay": dict(decay="none", t=300),
    "cuts": dict(decay="cuts", t=200, initial=True),
    "cuts f32": dict(decay="cuts", t=200, type=F32, initial=True),
    "all cut": dict(decay="all cut", initial=True),
    "decays of the lowest value": dict(decay="lowest", initial=True),
    "strong decays": dict(decay="strong", t=200, initial=True),
    "growing": dict(decay="growing", t=200),
    "ragged": dict(b=4, t=200, lengths=[200, 0, 1, 129], initial=True),
    "ragged f32": dict(b=4, t=100, lengths=[31, 32, 33, 0], type=F32, initial=True),
    "lengths outside": dict(b=3, t=70, lengths=[-5, 1000, 64], initial=True),
    "ragged segments": dict(b=2, t=1000, h=2, lengths=[1000, 300], dk=64, dv=64, decay="cuts", initial=True),
    "heads first": dict(layout="heads first", initial=True),
    "every other": dict(layout="every other", dk=64, dv=48),
    "odd offset": dict(layout="odd offset", dk=64, dv=48),
    "odd offset f32": dict(layout="odd offset", dk=64, dv=48, type=F32),
    "broadcast rows": dict(layout="broadcast", b=3),
}


@pytest.mark.parametrize("name", SHAPES)
def test_forward(name):
    print(f"\n[case] decay attention: {name}", flush=True)
    check_forward(make(**SHAPES[name]))


@pytest.mark.parametrize("name", SHAPES)
def test_backward(name):
    print(f"\n[case] decay attention gradient: {name}", flush=True)
    check_backward(make(**SHAPES[name]), grad_state=SHAPES[name].get("initial", False))


# Rows whose last 16-byte piece holds fewer elements: one piece, one and an element, several column blocks, segments,
# shared heads (f32 results before their sum), rows off any 16-byte border.
CUT = {
    "one piece": dict(dk=8, dv=8, layout="odd offset"),
    "one piece and one": dict(dk=9, dv=9, initial=True),
    "one piece and one f32": dict(dk=5, dv=5, type=F32, initial=True),
    "keys cut": dict(dk=70, dv=64, t=140),
    "values cut": dict(dk=64, dv=70, t=140),
    "two column blocks": dict(dk=31, dv=133, t=80, layout="odd offset"),
    "segments": dict(b=1, t=700, h=2, dk=59, dv=101, initial=True),
    "ragged segments f32": dict(b=2, t=500, h=2, lengths=[500, 77], dk=43, dv=61, type=F32, layout="odd offset"),
    "shared heads": dict(h=6, hq=2, hk=3, hv=1, dk=27, dv=42, t=130, initial=True),
    "shared heads f32": dict(h=6, hq=1, hk=6, hv=2, dk=26, dv=41, type=F32),
}


@pytest.mark.parametrize("name", CUT)
def test_cut_rows(name):
    print(f"\n[case] decay attention, cut rows: {name}", flush=True)
    s = make(**CUT[name], seed=50)
    check_forward(s)
    check_backward(s, grad_state=CUT[name].get("initial", False))


def test_an_infinity_in_a_cut_row():
    s = make(b=1, t=150, h=2, dk=35, dv=37)
    clean = _forward(s)[0]
    s["v"][0, 77, 0, 36] = float("inf")
    out = _forward(s)[0]
    assert torch.equal(out[..., :36], clean[..., :36]) and torch.equal(out[:, :, 1], clean[:, :, 1])
    assert torch.equal(out[:, :77], clean[:, :77]) and not torch.isfinite(out[0, 77:, 0, 36]).any()


@pytest.mark.parametrize("type", [BF, F32])
def test_no_tokens(type):
    s = make(t=0, type=type, initial=True)
    out, last = _forward(s)
    assert out.shape == (2, 0, 4, 32) and torch.equal(last, s["initial"])
    got = _backward(s)
    assert torch.equal(got[4], s["gs"]) and got[3].shape == (2, 0, 4)
    s = make(t=0, type=type, decay="head")
    assert not _backward(s, grad_state=False)[3].any()


def test_no_rows():
    s = make(b=0, initial=True)
    out, last = _forward(s)
    assert out.shape == (0, 100, 4, 32) and last.shape == (0, 4, 32, 32)
    s = make(b=0, decay="head")
    assert not _backward(s)[3].any()


@pytest.mark.parametrize("type", [BF, F32])
def test_what_does_not_exist_is_not_read(type):
    s = make(b=2, t=90, lengths=[50, 0], type=type, initial=True)
    clean = [x.clone() for x in (*_forward(s), *_backward(s))]
    for name in ("q", "k", "v", "go", "g"):
        for i, n in enumerate((50, 0)):
            s[name][i, n:] = float("nan") if name != "g" else float("inf")
    for a, b in zip(clean, (*_forward(s), *_backward(s))):
        assert torch.equal(a, b)


@pytest.mark.parametrize("type", [BF, F32])
@pytest.mark.parametrize("name", ["q", "k", "v"])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_infinities_reach_no_earlier_token(type, name, value):
    s = make(b=1, t=150, h=2, type=type)
    clean = _forward(s)[0]
    s[name][0, 77, 0, 3] = value
    out = _forward(s)[0]
    assert torch.equal(out[:, :77], clean[:, :77]) and torch.equal(out[:, :, 1], clean[:, :, 1])
    assert not torch.isfinite(out[0, 77, 0]).all()
    if name == "q":
        assert torch.equal(out[:, 78:], clean[:, 78:])


def test_autograd_gives_the_backward_call():
    s = make(t=70, type=F32, initial=True, lengths=[70, 30])
    leaves = [s[n].clone().requires_grad_() for n in ("q", "k", "v", "g", "initial")]
    out, last = sx.decay_attention(*leaves[:4], initial=leaves[4], lengths=s["lengths"], scale=s["scale"],
                                   return_state=True)
    ((out * s["go"]).sum() + (last * s["gs"]).sum()).backward()
    for leaf, want in zip(leaves, _backward(s)):
        assert torch.equal(leaf.grad, want)
    # only some of the inputs, and no gradient of the state
    q = s["q"].clone().requires_grad_()
    sx.decay_attention(q, s["k"], s["v"], s["g"], scale=s["scale"]).backward(s["go"])
    s["initial"], s["lengths"] = None, None
    assert torch.equal(q.grad, _backward(s, grad_state=False)[0])


def test_gradient_matches_differences_of_the_forward_call():
    s = make(t=80, type=F32, initial=True, decay="token")
    gen = torch.Generator().manual_seed(5)
    grads = _backward(s)

    def loss():
        out, last = _forward(s)
        return (out.double() * s["go"]).sum() + (last.double() * s["gs"]).sum()

    for name, grad in zip(("q", "k", "v", "g", "initial"), grads):
        x, e = s[name], 1e-2
        d = torch.randn(x.shape, generator=gen).to(DEV)
        s[name] = x + e * d
        up = loss()
        s[name] = x - e * d
        down = loss()
        s[name] = x
        want, got = ((up - down) / (2 * e)).item(), (grad.double() * d).sum().item()
        # forward errors of 2^-24 a term over 2e, the third derivative's share e^2 (the decay's alone is not linear)
        size = (grad.double().abs() * d.abs()).sum().item()
        assert abs(got - want) <= 2e-3 * size / np.sqrt(grad.numel()) + 5e-3 * abs(want), name


@pytest.mark.parametrize("type", [BF, F32])
def test_results_repeat(type):
    s = make(b=1, t=1000, h=4, hq=2, hv=1, dk=64, dv=64, type=type, initial=True)
    first = (*_forward(s), *_backward(s))
    for _ in range(3):
        for a, b in zip(first, (*_forward(s), *_backward(s))):
            assert torch.equal(a, b)


def test_replays_of_a_graph_and_another_stream():
    s = make(b=1, t=1000, h=2, hq=1, dk=64, dv=64, initial=True)
    t = make(b=1, t=1000, h=2, hq=1, dk=64, dv=64, initial=True, seed=3)
    eager, other = (*_forward(s), *_backward(s)), (*_forward(t), *_backward(t))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = (*_forward(s), *_backward(s))
    for i in range(4):
        (*_forward(t), *_backward(t))
        torch.cuda.synchronize()
        for c in captured:
            c.zero_()
        if i == 2:  # the graph reads what its inputs hold when it is replayed
            for n in ("q", "k", "v", "g", "initial", "go", "gs"):
                s[n].copy_(t[n])
        graph.replay()
        torch.cuda.synchronize()
        for c, e in zip(captured, other if i >= 2 else eager):
            assert torch.equal(c, e)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = (*_forward(t), *_backward(t))
    side.synchronize()
    for a, b in zip(got, other):
        assert torch.equal(a, b)


def test_both_ways_into_the_library():
    # an operand that has to be converted, or a scale that is no float, takes the binding's long way
    s = make(t=90, h=4, initial=True, lengths=[90, 40])
    want = (*_forward(s), *_backward(s))
    s["initial"] = s["initial"].transpose(2, 3).contiguous().transpose(2, 3)
    s["gs"] = s["gs"].transpose(0, 1).contiguous().transpose(0, 1)
    for a, b in zip(want, (*_forward(s), *_backward(s))):
        assert torch.equal(a, b)
    s["scale"] = 1.0
    want = _forward(s)
    s["scale"] = 1
    assert torch.equal(want[0], _forward(s)[0])
    one = make_step()
    kept = one["state"].clone()
    want = sx.decay_attention_step(one["q"], one["k"], one["v"], one["g"], kept, slots=one["slots"], scale=1.0)
    got = sx.decay_attention_step(one["q"], one["k"], one["v"], one["g"], one["state"], slots=one["slots"], scale=1)
    assert torch.equal(want, got) and torch.equal(kept, one["state"])
    for bad in (dict(log_decay=s["g"].double()), dict(v=s["v"].float()), dict(lengths=s["lengths"].long()),
                dict(initial=s["initial"][:1]), dict(q=s["q"][0]), dict(k=s["k"][:, :, :, :3]), dict(q=None)):
        args = dict(q=s["q"], k=s["k"], v=s["v"], log_decay=s["g"], initial=s["initial"], lengths=s["lengths"])
        with pytest.raises(sx.SxError):
            sx.decay_attention(**{**args, **bad})


def test_far_apart_rows():
    # batch rows more than 2^31 elements apart in one buffer
    base = make(b=2, t=70, h=2, dk=32, dv=32)
    out = _forward(base)
    apart = (1 << 31) + 4096
    room = torch.empty(apart + 70 * 2 * 32, dtype=BF, device=DEV)
    far = dict(base)
    for name in ("q", "k", "v"):
        x = room.as_strided((2, 70, 2, 32), (apart, 64, 32, 1))
        x.copy_(base[name])
        far[name] = x
        if name != "v":
            far[name] = base[name] if name == "q" else x
        got = _forward(far)
        assert torch.equal(got[0], out[0]) and torch.equal(got[1], out[1])
        far[name] = base[name]


# ---------------------------------------------------------------- one token

def make_step(b=5, pool=8, h=4, hq=None, hv=None, dk=32, dv=32, type=BF, per_head=False, slots="some idle", seed=0,
              layout="plain"):
    gen = torch.Generator().manual_seed(2000 + seed)
    hq, hv = hq or h, hv or h
    kv = _rand(gen, b, hq * dk + hv * dv + 1).to(type).to(DEV)
    off = 1 if layout == "odd offset" else 0
    s = dict(q=_rand(gen, b, hq, dk).to(type).to(DEV), k=kv[:, off:off + hq * dk].view(b, hq, dk),
             v=kv[:, off + hq * dk:off + hq * dk + hv * dv].view(b, hv, dv), scale=dk ** -0.5)
    if layout == "every other":
        s["q"] = _rand(gen, b, hq, 2 * dk).to(type).to(DEV)[..., ::2]
    s["g"] = (-torch.rand(h, generator=gen) if per_head else -torch.rand(b, h, generator=gen)).to(DEV)
    s["state"] = _rand(gen, pool, h, dk, dv).to(DEV)
    if layout == "heads apart":
        s["state"] = _rand(gen, h, pool, dk, dv).to(DEV).transpose(0, 1)
    s["slots"] = None
    if slots is not None:
        idx = torch.randperm(pool, generator=gen)[:b]
        if slots == "some idle" and b > 2:
            idx[1], idx[b - 1] = -1, pool
        if slots == "all idle":
            idx[:] = -1
        s["slots"] = idx.to(torch.int32).to(DEV)
    return s


def check_step(s):
    args = [_np(s[n]) for n in ("q", "k", "v", "g", "state")]
    slots = None if s["slots"] is None else s["slots"].tolist()
    ref = oa.decay_attention_step(*args, slots=slots, scale=s["scale"])
    size = oa.decay_attention_step(*args, slots=slots, scale=s["scale"], size=True)
    out = sx.decay_attention_step(s["q"], s["k"], s["v"], s["g"], s["state"], slots=s["slots"], scale=s["scale"])
    n = s["q"].shape[-1] + 16
    _close("out", out, ref[0], size[0], n, s["q"].dtype == BF)
    _close("state", s["state"], ref[1], size[1], n, False)


STEPS = {
    "plain": dict(),
    "f32": dict(type=F32),
    "one request": dict(b=1, pool=1, slots=None),
    "a state a row": dict(slots=None),
    "all idle": dict(slots="all idle"),
    "one decay a head": dict(per_head=True),
    "shared heads": dict(h=6, hq=2, hv=3),
    "width one": dict(dk=1, dv=1),
    "odd widths": dict(dk=33, dv=47),
    "odd widths f32": dict(dk=129, dv=7, type=F32),
    "128": dict(dk=128, dv=128, b=9, pool=11),
    "72 columns": dict(dk=40, dv=72),
    "widest": dict(dk=256, dv=256),
    "heads apart": dict(layout="heads apart"),
    "odd offset": dict(layout="odd offset"),
    "every other": dict(layout="every other"),
}


@pytest.mark.parametrize("name", STEPS)
def test_step(name):
    print(f"\n[case] decay attention step: {name}", flush=True)
    check_step(make_step(**STEPS[name]))


def test_steps_follow_the_prompt():
    s = make(b=3, t=40, h=4, hq=2, dk=48, dv=32, initial=True)
    out, last = _forward(s)
    state = s["initial"].clone()
    for t in range(40):
        o = sx.decay_attention_step(s["q"][:, t], s["k"][:, t], s["v"][:, t], s["g"][:, t], state, scale=s["scale"])
        # both are the same value rounded to bf16: one step of it apart at most
        assert ((o - out[:, t]).float().abs() <= 2.0 ** -7 * out[:, t].float().abs() + 1e-3).all()
    torch.testing.assert_close(state, last, rtol=1e-5, atol=1e-5)


def test_step_on_a_pool_past_32_bits():
    h, dk, dv = 2, 128, 128
    pool = (1 << 31) // (h * dk * dv) + 9  # elements; byte offsets pass 2^33
    s = make_step(b=2, pool=2, h=h, dk=dk, dv=dv, slots=None)
    small = s["state"].clone()
    want = sx.decay_attention_step(s["q"], s["k"], s["v"], s["g"], small, scale=s["scale"])
    big = torch.empty(pool, h, dk, dv, device=DEV)
    slots = torch.tensor([pool - 1, 3], dtype=torch.int32, device=DEV)
    big[pool - 1], big[3] = s["state"][0], s["state"][1]
    got = sx.decay_attention_step(s["q"], s["k"], s["v"], s["g"], big, slots=slots, scale=s["scale"])
    assert torch.equal(got, want)
    assert torch.equal(big[pool - 1], small[0]) and torch.equal(big[3], small[1])


def test_replays_of_a_captured_step_advance_the_state():
    s, e = make_step(), make_step()
    call = lambda x: sx.decay_attention_step(x["q"], x["k"], x["v"], x["g"], x["state"], slots=x["slots"],  # noqa: E731
                                             scale=x["scale"])
    call(s), call(e)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(s)
    for _ in range(4):
        want = call(e)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(s["state"], e["state"])
