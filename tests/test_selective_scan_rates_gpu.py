"""The selective scan with rates whose product with log2(e) passes f32's range, or that are infinite: a state that
forgets at once, and one that a step of zero leaves as it is."""

import pytest
import torch

import scan_primitives_amd as sx
from tests import test_selective_scan_gpu as scan
from tests.test_causal_conv_gpu import BF, F32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("type", [BF, F32])
@pytest.mark.parametrize("rate", [float("-inf"), -3e38])
@pytest.mark.parametrize("kwargs", [dict(t=20, lengths=[20, 9]), dict(b=1, t=900), dict(b=3, t=333, lengths=[0, 333, 100], n=6)])
def test_a_rate_without_bound_is_a_large_one(kwargs, rate, type):
    s, g = scan.make(type=type, initial=True, d=40, **kwargs)
    s["a"][:, 3] = -1e30  # exp(dt a) is zero for every step there is
    want = (*sx.selective_scan(return_state=True, **s), *sx.selective_scan_backward(**s, **g))
    assert all(torch.isfinite(t).all() for t in want)
    s["a"][:, 3] = rate
    got = (*sx.selective_scan(return_state=True, **s), *sx.selective_scan_backward(**s, **g))
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_a_step_of_zero_keeps_the_state():
    for rate in (-3e38, float("-inf")):
        one = scan.make_step(type=F32, softplus=False, slots=None, pool=3)
        one["a"][:, 3] = rate
        one["delta"] = torch.zeros_like(one["delta"])
        one["delta_bias"] = None
        state = one["state"].clone()
        sx.selective_scan_step(**one)
        assert torch.equal(one["state"], state)
        p, _ = scan.make(type=F32, softplus=False, bias=False, initial=True, t=20)
        p["a"][:, 3] = rate
        p["delta"].zero_()
        assert torch.equal(sx.selective_scan(return_state=True, **p)[1], p["initial"])
