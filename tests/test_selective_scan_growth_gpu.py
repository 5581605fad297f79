"""The selective scan with states that grow (positive rates, or negative steps), across segments: a zero stays zero and
a small state comes out as token by token, also where the growth alone passes f32's range."""

import pytest
import torch

import scan_primitives_amd as sx
from oracle import state_space as os_
from tests import test_selective_scan_gpu as scan
from tests.test_causal_conv_gpu import BF, DEV, F32, close, host

pytestmark = pytest.mark.gpu

# dt a = 6.3 to 6.6 a token: 16 tokens, the shortest segment, grow by more than 2^145. The last has segments of 64.
SIZES = [dict(b=1, t=700, d=40, n=4), dict(b=2, t=300, d=70, n=10, g=2, gate=False),
         dict(b=1, t=400, d=24, n=29, layout="channels first"), dict(b=4, t=128, d=256, n=16, g=64, skip=False)]


def _make(how, size, type=F32, seed=0):
    """Rates and steps whose product is positive: by the rates, under softplus or not, or by the steps."""
    s, g = scan.make(type=type, softplus=how == "softplus", bias=False, initial=True, seed=seed, **size)
    s["a"] = 1.05 + 0.04 * torch.rand(s["a"].shape, generator=torch.Generator().manual_seed(seed)).to(DEV)
    if how == "steps":
        s["a"] = -s["a"]
    return s, g


def _grow(s, how, tokens):
    """A step of 6 in `tokens`, of 1e-4 elsewhere."""
    sign = -1 if how == "steps" else 1
    s["delta"].fill_(-9.0 if how == "softplus" else sign * 1e-4)
    s["delta"][:, tokens] = sign * 6.0


def _check(s, g, tokens):
    """`tokens`: how many grow at most in a chain that is not zero."""
    # the exponents, up to 6.6 of each such token: a rate's and a product's rounding, and one of each of a sum's terms
    more = 6.6 * tokens * (tokens + 3)
    out, last = sx.selective_scan(return_state=True, **s)
    (ref, want), (size, sstate) = (os_.selective_scan(size=z, **host(s)) for z in (False, True))
    close("out", out, ref, size, scan._steps(s) + more)
    close("last state", last, want, sstate, scan._steps(s) + more)
    got = sx.selective_scan_backward(**s, **g)
    ref, size = (os_.selective_scan_vjp(size=z, **host(s), **host(g)) for z in (False, True))
    for i, what in enumerate(scan.NAMES):
        if got[i] is not None:
            close(what, got[i], ref[i], size[i], 2 * (scan._steps(s, tokens=True, rows=True) + more))


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("how", ["softplus", "rates", "steps"])
def test_nothing_grows_to_nothing(how, size):
    s, g = _make(how, size)
    _grow(s, how, slice(None))
    # inputs at the last tokens alone, and the result's gradient at the first
    s["initial"].zero_()
    g["grad_state"].zero_()
    s["x"][:, :-8] = 0
    g["grad_out"][:, 8:] = 0
    _check(s, g, 8)


@pytest.mark.parametrize("type", [F32, BF])
@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("how", ["softplus", "rates", "steps"])
def test_small_states_that_grow_past_the_range(how, size, type):
    # 16 tokens grow by 2^145: states before them and gradients behind them are of 1e-30, in one segment and over the
    # border of two
    t = size["t"]
    for first in (t // 2 // 64 * 64, t // 2 // 64 * 64 - 6):
        s, g = _make(how, size, type)
        _grow(s, how, slice(first, first + 16))
        s["initial"] *= 1e-30
        s["x"][:, first:first + 16] = 0
        g["grad_out"][:, first:first + 16] = 0
        s["x"][:, :first] *= 1e-30
        g["grad_out"][:, first + 16:] *= 1e-30
        g["grad_state"] *= 1e-30
        _check(s, g, 16)


def test_growth_that_decays_again_within_a_segment():
    s, g = _make("rates", SIZES[3])
    _grow(s, "rates", slice(70, 86))
    s["delta"][:, 86:102] = -6.0
    # states grow to 1e34 and come back. Gradients behind go back over the same tokens, to 1e-34 and back.
    s["initial"] *= 1e-10
    s["x"][:, 64:102] = 0
    s["x"][:, :64] *= 1e-10
    g["grad_out"][:, 64:102] = 0
    g["grad_out"][:, 102:] *= 1e10
    g["grad_state"] *= 1e10
    _check(s, g, 32)
