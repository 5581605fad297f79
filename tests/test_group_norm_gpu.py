"""Group norm on the GPU against the 64-bit oracle.

Tolerances, from the arithmetic: the mean and variance of m values come from
sums in 32 bits in an order of their own, n = m roundings that are independent: eight
standard deviations, 8 sqrt(m) 2^-24, of the mean of the absolute values and of the
variance. x - mean is exact to a step of its own and the mean's error, so u is off by
(8 sqrt(m) + 16) 2^-24 of (|x| + mean |x|) / root |weight| + |bias|, with SiLU 8 steps more;
a gradient by twice as many of what its terms add up to, plus what n's error (the same
over root) does through SiLU's second derivative (at most 0.5). Sums over all rows: their number more. bf16 results are
rounded once: 2^-8 of themselves.
"""

import numpy as np
import pytest
import torch

import scan_primitives_amd as sx
from oracle import state_space as os_
from tests.test_causal_conv_gpu import BF, DEV, F32, _np, close

pytestmark = pytest.mark.gpu


def make(shape=(40, 64), groups=4, type=BF, act=None, weight=True, bias=True, eps=1e-5, layout="plain", offset=0.0,
         seed=0):
    gen = torch.Generator().manual_seed(4000 + seed)
    c = shape[-1]

    def laid():
        if layout == "half of a projection":
            return (torch.randn(*shape[:-1], 2 * c, generator=gen) + offset).to(type).to(DEV)[..., c:]
        if layout == "odd offset":
            return (torch.randn(*shape[:-1], c + 3, generator=gen) + offset).to(type).to(DEV)[..., 1:c + 1]
        if layout == "channels first":
            return (torch.randn(shape[0], c, *shape[1:-1], generator=gen) + offset).to(type).to(DEV).movedim(1, -1)
        if layout == "samples inside":
            return (torch.randn(shape[1], shape[0], *shape[2:], generator=gen) + offset).to(type).to(DEV).transpose(0, 1)
        return (torch.randn(*shape, generator=gen) + offset).to(type).to(DEV)

    return dict(x=laid(), groups=groups, weight=torch.randn(c, generator=gen).to(DEV) if weight else None,
                bias=torch.randn(c, generator=gen).to(DEV) if bias else None, eps=eps, activation=act), laid()


CASES = {
    "rows": dict(),
    "rows f32 silu": dict(type=F32, act="silu"),
    "one row": dict(shape=(1, 64)),
    "one group": dict(shape=(33, 64), groups=1, type=F32),
    "a channel a group": dict(shape=(9, 24), groups=24, type=F32),
    "two channels a group": dict(shape=(70, 24), groups=12, act="silu"),
    "odd groups": dict(shape=(50, 185), groups=5, type=F32),
    "odd groups bf16": dict(shape=(50, 111), groups=3, act="silu"),
    "groups of 24": dict(shape=(100, 192), groups=8),
    "groups of 20 f32": dict(shape=(100, 60), groups=3, type=F32),
    "wide rows": dict(shape=(20, 2048), groups=2, act="silu"),
    "wide rows f32": dict(shape=(10, 3000), groups=1, type=F32),
    "very wide rows": dict(shape=(5, 8192), groups=1),
    "very wide rows f32": dict(shape=(3, 4096), groups=1, type=F32, act="silu"),
    "odd wide rows": dict(shape=(7, 1021), groups=1),
    "rows too wide for a workgroup": dict(shape=(4, 9000), groups=1, type=F32),
    "odd rows too wide for a workgroup": dict(shape=(3, 2 * 1501), groups=2),
    "many rows": dict(shape=(5000, 32), groups=2, type=F32),
    "more groups than slots": dict(shape=(30, 1600), groups=100),
    "sequences": dict(shape=(3, 50, 64)),
    "sequences f32 silu": dict(shape=(2, 333, 48), groups=6, type=F32, act="silu"),
    "maps": dict(shape=(2, 9, 7, 40), groups=5, act="silu"),
    "volumes": dict(shape=(1, 3, 4, 5, 16), groups=2, type=F32),
    "one position": dict(shape=(6, 1, 64), groups=2),
    "one position a row": dict(shape=(6, 1, 1, 10), groups=5, type=F32),
    "long sequences": dict(shape=(1, 20000, 32), groups=8, act="silu"),
    "sequences of many channels": dict(shape=(2, 100, 4096), groups=32),
    "sequences of wide groups": dict(shape=(2, 10, 6000), groups=2, type=F32),
    "sequences of odd wide groups": dict(shape=(2, 11, 1006), groups=2, act="silu"),
    "sequences of odd groups": dict(shape=(3, 65, 33), groups=3, type=F32, act="silu"),
    "no weight": dict(weight=False),
    "no bias": dict(bias=False, shape=(2, 30, 16), act="silu"),
    "neither": dict(weight=False, bias=False, type=F32),
    "a far mean": dict(offset=300.0, type=F32, shape=(30, 256), groups=2),
    "a far mean of sequences": dict(offset=300.0, type=F32, shape=(2, 500, 64), groups=2),
    "half of a projection": dict(layout="half of a projection", act="silu"),
    "half of a projection, sequences": dict(layout="half of a projection", shape=(2, 40, 64), type=F32),
    "odd offset": dict(layout="odd offset"),
    "channels first": dict(layout="channels first", shape=(2, 40, 64)),
    "samples inside": dict(layout="samples inside", shape=(3, 40, 64), type=F32),
    "samples inside of maps": dict(layout="samples inside", shape=(3, 4, 5, 16)),
}


def _size(s):
    """What u's parts add up to, and the count a group's sums go over."""
    x, g = np.abs(_np(s["x"])), s["groups"]
    c = x.shape[-1]
    v = x.reshape(x.shape[0], -1, g, c // g)
    full = _np(s["x"]).reshape(v.shape)
    root = np.sqrt(full.var((1, 3), keepdims=True) + s["eps"])
    w = np.ones(c) if s["weight"] is None else np.abs(_np(s["weight"]))
    b = np.zeros(c) if s["bias"] is None else np.abs(_np(s["bias"]))
    n = (v + v.mean((1, 3), keepdims=True)) / root
    return (n * w.reshape(g, -1) + b.reshape(g, -1)).reshape(x.shape), n.reshape(x.shape), v.shape[1] * v.shape[3], root


def _host(s):
    return {k: (_np(v) if isinstance(v, torch.Tensor) else v) for k, v in s.items()}


@pytest.mark.parametrize("name", CASES)
def test_forward(name):
    s, _ = make(**CASES[name])
    size, _, m, _ = _size(s)
    close("out", sx.group_norm(**s), os_.group_norm(**_host(s)), size, 1.1 * (8 * np.sqrt(m) + 16) + 8)


@pytest.mark.parametrize("name", CASES)
def test_backward(name):
    s, go = make(**CASES[name])
    got = sx.group_norm_backward(grad_out=go, **s)
    ref, size = os_.group_norm_vjp(grad_out=_np(go), **_host(s))
    usize, nsize, m, root = _size(s)
    steps = 2 * (8 * np.sqrt(m) + 16) + 30
    # n's error, over root and through the slope of SiLU, of the largest row and element
    g, c = s["groups"], s["x"].shape[-1]
    lead = (go.shape[0], -1, g, c // g)
    w = (np.ones(c) if s["weight"] is None else np.abs(_np(s["weight"]))).reshape(g, -1)
    part = np.abs(_np(go)).reshape(lead) * w * (usize + nsize).reshape(lead)
    full = np.broadcast_to(part.max((1, 3), keepdims=True) / root, part.shape).reshape(go.shape)
    close("grad_x", got[0], ref[0], size[0] + full, steps)
    rows = go.numel() // c
    for what, a, r, z, p in (("grad_weight", got[1], ref[1], size[1], usize * (1 + nsize)),
                             ("grad_bias", got[2], ref[2], size[2], usize)):
        if a is None:
            assert s[what[5:]] is None
            continue
        extra = (np.abs(_np(go)) * p).reshape(-1, c).sum(0)
        close(what, a, r, z + extra, steps + 8 * np.sqrt(rows))


def test_every_row_of_rows_is_a_sample_of_one_position():
    s, go = make(shape=(12, 96), groups=3, type=F32, act="silu")
    t = dict(s, x=s["x"][:, None])
    assert torch.equal(sx.group_norm(**s), sx.group_norm(**t)[:, 0])


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("shape", [(5, 64), (3, 20, 64)])
def test_an_infinity_stays_in_its_group(shape, value):
    s, go = make(shape=shape, type=F32, act="silu")
    clean, grads = sx.group_norm(**s), sx.group_norm_backward(grad_out=go, **s)
    s["x"][(1,) + (0,) * (len(shape) - 2) + (20,)] = value
    out, got = sx.group_norm(**s), sx.group_norm_backward(grad_out=go, **s)
    bad = torch.zeros_like(out, dtype=torch.bool)
    bad[1, ..., 16:32] = True
    assert torch.isnan(out[bad]).all() and torch.equal(out[~bad], clean[~bad])
    assert torch.equal(got[0][~bad], grads[0][~bad])
    keep = torch.arange(64, device=DEV) // 16 != 1
    assert torch.equal(got[1][keep], grads[1][keep]) and torch.equal(got[2][keep], grads[2][keep])


@pytest.mark.parametrize("shape", [(6, 32), (2, 40, 32)])
def test_a_group_without_variance(shape):
    s, go = make(shape=shape, type=F32)
    s["x"].fill_(7.25)
    out = sx.group_norm(**s)
    assert torch.equal(out, s["bias"].expand(shape))
    assert torch.isfinite(sx.group_norm_backward(grad_out=go, **s)[0]).all()


def test_nothing_to_norm():
    for shape in ((0, 64), (3, 0, 64), (0, 5, 64)):
        s, go = make(shape=shape, type=F32)
        assert sx.group_norm(**s).shape == shape
        gx, gw, gb = sx.group_norm_backward(grad_out=go, **s)
        assert gx.shape == shape and not gw.any() and not gb.any()


def test_autograd_gives_the_backward_call():
    for shape in ((30, 64), (2, 21, 64)):
        s, go = make(shape=shape, type=F32, act="silu")
        leaves = {n: s[n].clone().requires_grad_() for n in ("x", "weight", "bias")}
        sx.group_norm(**{**s, **leaves}).backward(go)
        for a, n in zip(sx.group_norm_backward(grad_out=go, **s), leaves):
            assert torch.equal(leaves[n].grad, a), n


@pytest.mark.parametrize("shape", [(10, 24), (2, 9, 24)])
@pytest.mark.parametrize("act", [None, "silu"])
def test_gradient_matches_differences_of_the_forward_call(shape, act):
    s, go = make(shape=shape, type=F32, act=act)
    grads = sx.group_norm_backward(grad_out=go, **s)
    gen = torch.Generator().manual_seed(5)
    for n, grad in zip(("x", "weight", "bias"), grads):
        step = torch.randn(s[n].shape, generator=gen).to(DEV)
        e = 1e-2
        up, down = ((sx.group_norm(**{**s, n: s[n] + k * e * step}).double() * go).sum().item() for k in (1, -1))
        want = (grad.double() * step.double()).sum().item()
        # the third derivative's share e^2, and f32 roundings over 2 e
        assert abs((up - down) / (2 * e) - want) <= 2e-3 * abs(want) + 5e-3 * grad.double().norm().item(), n


def test_far_apart_samples():
    far = (1 << 31) + 40
    s, go = make(shape=(2, 30, 32), type=BF)
    want = (sx.group_norm(**s), *sx.group_norm_backward(grad_out=go, **s))
    room = torch.empty(far + 4 * 30 * 32, dtype=BF, device=DEV)
    x, g = (room.as_strided((2, 30, 32), (far, 32, 1), k * 30 * 32) for k in (0, 1))
    x.copy_(s["x"])
    g.copy_(go)
    s["x"] = x
    for a, b in zip((sx.group_norm(**s), *sx.group_norm_backward(grad_out=g, **s)), want):
        assert torch.equal(a, b)
