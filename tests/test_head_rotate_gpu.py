"""Head norm + rotation on the GPU against the 64-bit oracle.

Tolerances: a row's sum of squares adds eight squares in a lane and at most
five more steps between lanes; with the root, the three products, the cosine
and sine (an angle in turns kept to 2^-25 of a turn, then 2 units each) and
the two of the turn, fewer than 32 roundings of 2^-24 meet, on the size of the
two components that turn together; a bf16 result is rounded once more, 2^-8.
Weights' gradients are sums over n rows: 8 sqrt(n) deviations on top.
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


def make(b=2, t=9, hq=4, hk=2, d=64, rot=None, type=BF, near=False, weights=True, first=1000, positions="int64",
         layout="plain", seed=0):
    gen = torch.Generator().manual_seed(3000 + seed)
    rand = lambda *shape: torch.randn(*shape, generator=gen)  # noqa: E731
    rot = d - d % 2 if rot is None else rot
    qkv = rand(b, t, (hq + hk) * d + 1).to(type).to(DEV)
    off = 1 if layout == "odd offset" else 0
    s = dict(q=qkv[..., off:off + hq * d].view(b, t, hq, d),
             k=qkv[..., off + hq * d:off + (hq + hk) * d].view(b, t, hk, d))
    if layout == "aligned":
        whole = rand(b, t, (hq + hk) * d).to(type).to(DEV)
        s["q"], s["k"] = whole[..., :hq * d].view(b, t, hq, d), whole[..., hq * d:].view(b, t, hk, d)
    if layout == "heads first":
        s["q"], s["k"] = (rand(b, h, t, d).to(type).to(DEV).transpose(1, 2) for h in (hq, hk))
    if layout == "every other":
        s["q"], s["k"] = (rand(b, t, h, 2 * d).to(type).to(DEV)[..., ::2] for h in (hq, hk))
    if layout == "expanded":
        s["q"], s["k"] = (rand(b, t, 1, d).to(type).to(DEV).expand(b, t, h, d) for h in (hq, hk))
    s["gq"], s["gk"] = rand(b, t, hq, d).to(type).to(DEV), rand(b, t, hk, d).to(type).to(DEV)
    s["qw"], s["kw"] = (1 + 0.2 * rand(d)).to(DEV), (1 + 0.2 * rand(d)).to(DEV)
    if not weights:
        s["qw"] = s["kw"] = None
    kind = torch.int32 if positions == "int32" else torch.int64
    s["positions"] = (first + torch.randint(0, 5000, (b, t), generator=gen)).to(kind).to(DEV)
    if positions == "row":
        s["positions"] = s["positions"][0]
    if positions == "negative":
        s["positions"] = -s["positions"]
    s["turns"] = sx.rotation_turns(rot).to(DEV)
    s["near"] = near
    return s


CASES = {
    "plain": dict(),
    "one token": dict(b=1, t=1),
    "f32": dict(type=F32),
    "128": dict(d=128, hq=8, hk=2, layout="aligned"),
    "128 f32 neighbours": dict(d=128, type=F32, near=True, layout="aligned"),
    "64 aligned": dict(layout="aligned"),
    "80, half turned": dict(d=80, rot=40, near=True, type=F32, layout="aligned"),
    "80, half turned, halves": dict(d=80, rot=40, layout="aligned"),
    "ten turned": dict(d=64, rot=10),
    "ten turned, aligned": dict(d=64, rot=10, layout="aligned"),
    "two turned neighbours": dict(d=64, rot=2, near=True, layout="aligned"),
    "none turned": dict(d=48, rot=0, layout="aligned"),
    "odd width": dict(d=17, rot=6),
    "odd width f32 neighbours": dict(d=33, rot=32, near=True, type=F32),
    "width one": dict(d=1),
    "width two": dict(d=2),
    "widest": dict(d=256, layout="aligned"),
    "widest f32, odd": dict(d=255, type=F32),
    "no weights": dict(weights=False),
    "int32 positions": dict(positions="int32"),
    "one row of positions": dict(positions="row"),
    "negative positions": dict(positions="negative", type=F32),
    "far positions": dict(first=1 << 30, type=F32),
    "heads first": dict(layout="heads first"),
    "every other": dict(layout="every other"),
    "odd offset": dict(layout="odd offset"),
    "expanded heads": dict(layout="expanded"),
    "no key heads": dict(hk=0, layout="aligned"),
    "many tokens": dict(b=3, t=701, hq=5, hk=1, d=64, layout="aligned"),
    "many tokens f32": dict(b=1, t=2051, hq=2, hk=2, d=40, rot=20, type=F32),
}


def _close(name, got, ref, size, bf16, rows=1):
    got = _np(got)
    assert got.shape == ref.shape and np.isfinite(got).all(), name
    tol = (32.0 + (8.0 * np.sqrt(rows) if rows > 1 else 0.0)) * 2.0 ** -24 * size
    if bf16:
        tol = tol + 2.0 ** -8 * np.abs(ref)
    over = np.abs(got - ref) - tol
    if over.size and over.max() > 1e-37:
        at = np.unravel_index(np.argmax(over), over.shape)
        raise AssertionError(f"{name} at {at}: got {got[at]!r}, ref {ref[at]!r}, tolerance {tol[at]!r}")


def _positions(s):
    p = _np(s["positions"])
    return np.broadcast_to(p, s["q"].shape[:2])


def _forward(s):
    return sx.head_norm_rotate(s["q"], s["k"], s["positions"], s["turns"], q_weight=s["qw"], k_weight=s["kw"],
                               neighbours=s["near"])


def _backward(s):
    return sx.head_norm_rotate_backward(s["q"], s["k"], s["positions"], s["turns"], s["gq"], s["gk"], q_weight=s["qw"],
                                        k_weight=s["kw"], neighbours=s["near"])


@pytest.mark.parametrize("name", CASES)
def test_forward(name):
    print(f"\n[case] head norm + rotation: {name}", flush=True)
    s = make(**CASES[name])
    for got, x, w in zip(_forward(s), ("q", "k"), ("qw", "kw")):
        args = (_np(s[x]), _positions(s), _np(s["turns"]), _np(s[w]))
        ref = oa.head_norm_rotate(*args, neighbours=s["near"])
        size = oa.head_norm_rotate(*args, neighbours=s["near"], size=True)
        assert got.dtype == s[x].dtype and got.is_contiguous()
        _close(x, got, ref, np.abs(size), s[x].dtype == BF)


@pytest.mark.parametrize("name", CASES)
def test_backward(name):
    print(f"\n[case] head norm + rotation gradient: {name}", flush=True)
    s = make(**CASES[name])
    got = _backward(s)
    for i, (x, w) in enumerate((("q", "qw"), ("k", "kw"))):
        args = (_np(s[x]), _positions(s), _np(s["turns"]), _np(s["g" + x]), _np(s[w]))
        ref = oa.head_norm_rotate_vjp(*args, neighbours=s["near"])
        size = oa.head_norm_rotate_vjp(*args, neighbours=s["near"], size=True)
        _close("grad_" + x, got[i], ref[0], size[0], s[x].dtype == BF)
        if s[w] is None:
            assert got[2 + i] is None
        else:
            rows = int(np.prod(s[x].shape[:3])) + 1
            _close("grad of " + w, got[2 + i], ref[1], size[1], False, rows=rows)


@pytest.mark.parametrize("type", [BF, F32])
def test_no_tokens_and_rows_of_zeros(type):
    s = make(t=0, type=type)
    q, k = _forward(s)
    assert q.shape == (2, 0, 4, 64) and k.shape == (2, 0, 2, 64)
    got = _backward(s)
    assert got[0].shape == q.shape and not got[2].any() and not got[3].any()
    s = make(type=type)
    s["q"], s["k"] = torch.zeros_like(s["q"]), torch.zeros_like(s["k"])
    assert not any(x.any() for x in _forward(s))
    assert torch.isfinite(_backward(s)[0]).all()


def test_infinities_stay_in_their_row():
    s = make(t=20)
    clean = _forward(s)
    s["q"][1, 7, 2, 5], s["k"][0, 3, 1, 0] = float("nan"), float("inf")
    for got, want, at in zip(_forward(s), clean, ((1, 7, 2), (0, 3, 1))):
        assert not torch.isfinite(got[at]).all()
        got[at], want[at] = 0, 0
        assert torch.equal(got, want)


# Rows whose pieces are cut by the turned half, by the row's end or by both, down to a row of one piece, and the
# widest rows of few turned pairs, which take the most lanes.
WIDTHS = {
    "one piece": dict(d=8, rot=8),
    "one piece f32": dict(d=4, rot=2, type=F32),
    "one piece and one": dict(d=9, rot=2),
    "half cut": dict(d=64, rot=36, layout="aligned"),
    "half and end cut": dict(d=114, rot=46),
    "half cut, odd end": dict(d=75, rot=74, layout="odd offset"),
    "end cut, neighbours": dict(d=121, rot=30, near=True),
    "end cut f32": dict(d=58, rot=22, type=F32, layout="odd offset"),
    "odd end f32, neighbours": dict(d=101, rot=100, near=True, type=F32),
    "widest, two turned": dict(d=256, rot=2),
    "widest, two turned f32": dict(d=256, rot=2, type=F32),
    "widest, two turned, every other f32": dict(d=256, rot=2, type=F32, layout="every other"),
    "many tokens, half cut": dict(b=3, t=401, hq=5, hk=1, d=90, rot=12),
}


@pytest.mark.parametrize("name", WIDTHS)
def test_cut_pieces(name):
    print(f"\n[case] head norm + rotation, cut pieces: {name}", flush=True)
    s = make(**WIDTHS[name], seed=50)
    out, grad = _forward(s), _backward(s)
    for i, (x, w) in enumerate((("q", "qw"), ("k", "kw"))):
        args = (_np(s[x]), _positions(s), _np(s["turns"]), _np(s[w]))
        ref = oa.head_norm_rotate(*args, neighbours=s["near"])
        size = oa.head_norm_rotate(*args, neighbours=s["near"], size=True)
        _close(x, out[i], ref, np.abs(size), s[x].dtype == BF)
        args = args[:3] + (_np(s["g" + x]), args[3])
        ref = oa.head_norm_rotate_vjp(*args, neighbours=s["near"])
        size = oa.head_norm_rotate_vjp(*args, neighbours=s["near"], size=True)
        _close("grad_" + x, grad[i], ref[0], size[0], s[x].dtype == BF)
        _close("grad_" + w, grad[2 + i], ref[1], size[1], False, rows=s[x].shape[0] * s[x].shape[1] * s[x].shape[2])


@pytest.mark.parametrize("type", [BF, F32])
@pytest.mark.parametrize("near", [False, True])
def test_an_infinity_behind_the_turned_part_stays_alone(type, near):
    s = make(type=type, rot=10, near=near)
    s["q"][1, 3, 2, 20] = float("inf")
    row = _forward(s)[0][1, 3, 2].clone()
    assert torch.isnan(row[20])  # infinity times a root of zero
    row[20] = 0
    assert not row.any()


def test_autograd_gives_the_backward_call():
    s = make(t=30, type=F32)
    leaves = [s[n].clone().requires_grad_() for n in ("q", "k", "qw", "kw")]
    q, k = sx.head_norm_rotate(leaves[0], leaves[1], s["positions"], s["turns"], q_weight=leaves[2], k_weight=leaves[3])
    ((q * s["gq"]).sum() + (k * s["gk"]).sum()).backward()
    # the same layout for both: another alignment takes another order of the sums
    s.update({n: x.detach() for n, x in zip(("q", "k", "qw", "kw"), leaves)})
    for leaf, want in zip(leaves, _backward(s)):
        assert torch.equal(leaf.grad, want)


def test_autograd_with_one_result_used():
    s = make(t=30, type=F32)
    q = s["q"].clone().requires_grad_()
    got, _ = sx.head_norm_rotate(q, s["k"], s["positions"], s["turns"], q_weight=s["qw"], k_weight=s["kw"])
    got.backward(s["gq"])
    s["q"] = q.detach()
    s["gk"] = torch.zeros_like(s["gk"])
    assert torch.equal(q.grad, _backward(s)[0])


def test_replays_of_a_graph_and_results_repeat():
    s = make(b=2, t=1100, d=64, layout="aligned")
    eager = (*_forward(s), *_backward(s))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = (*_forward(s), *_backward(s))
    for _ in range(4):
        for a, b in zip(eager, (*_forward(s), *_backward(s))):
            assert torch.equal(a, b)
        torch.cuda.synchronize()
        for c in captured:
            c.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager, captured):
            assert torch.equal(a, b)


def test_far_apart_rows():
    s = make(t=33)
    want = (*_forward(s), *_backward(s))
    apart = (1 << 31) + 4096
    room = torch.empty(apart + 33 * 256, dtype=BF, device=DEV)
    for name in ("q", "gq"):
        x = room.as_strided((2, 33, 4, 64), (apart, 256, 64, 1))
        x.copy_(s[name])
        kept, s[name] = s[name], x
        for a, b in zip(want, (*_forward(s), *_backward(s))):
            assert torch.equal(a, b)
        s[name] = kept


# One token in f32, and token groups enough that a workgroup of the gradient takes several (1024 of them at most take
# part on 256 compute units; with 130 heads a group is one token).
MORE = {
    "one token f32": dict(b=1, t=1, type=F32),
    "one token f32, far": dict(b=1, t=1, type=F32, first=1 << 20, layout="aligned", d=128),
    "one token f32 neighbours, odd width": dict(b=1, t=1, type=F32, near=True, d=33, rot=20),
    "several groups a workgroup": dict(b=2, t=1300, hq=130, hk=2, d=8, layout="aligned"),
    "several groups a workgroup f32": dict(b=1, t=2100, hq=2, hk=130, d=10, rot=6, type=F32),
}


@pytest.mark.parametrize("name", MORE)
def test_single_tokens_and_many_groups(name):
    print(f"\n[case] head norm + rotation: {name}", flush=True)
    s = make(**MORE[name], seed=70)
    out, grad = _forward(s), _backward(s)
    for i, (x, w) in enumerate((("q", "qw"), ("k", "kw"))):
        args = (_np(s[x]), _positions(s), _np(s["turns"]), _np(s[w]))
        size = oa.head_norm_rotate(*args, neighbours=s["near"], size=True)
        _close(x, out[i], oa.head_norm_rotate(*args, neighbours=s["near"]), np.abs(size), s[x].dtype == BF)
        args = args[:3] + (_np(s["g" + x]), args[3])
        ref = oa.head_norm_rotate_vjp(*args, neighbours=s["near"])
        size = oa.head_norm_rotate_vjp(*args, neighbours=s["near"], size=True)
        _close("grad_" + x, grad[i], ref[0], size[0], s[x].dtype == BF)
        _close("grad_" + w, grad[2 + i], ref[1], size[1], False, rows=s[x].shape[0] * s[x].shape[1] * s[x].shape[2])
