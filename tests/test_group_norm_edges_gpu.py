"""Group norm where its arithmetic ends: no eps, infinities anywhere in a group, squares past f32's range."""

import pytest
import torch

import scan_primitives_amd as sx
from oracle import state_space as os_
from scan_primitives_amd import _binding as B
from tests import test_group_norm_gpu as norm
from tests.test_causal_conv_gpu import BF, DEV, F32, close

pytestmark = pytest.mark.gpu


# rows that fill the last step of the workgroups' rows in part; wide rows; samples of several positions
@pytest.mark.parametrize("type", [BF, F32])
@pytest.mark.parametrize("act", [None, "silu"])
@pytest.mark.parametrize("shape,groups", [((1, 64), 1), ((500, 64), 4), ((37, 96), 3), ((1000, 200), 10), ((5, 3000), 1),
                                          ((7, 1021), 1), ((3, 50, 64), 4), ((1, 4000, 48), 3)])
def test_no_eps(shape, groups, act, type, monkeypatch):
    monkeypatch.setitem(norm.CASES, "no eps", dict(shape=shape, groups=groups, act=act, type=type, eps=0.0))
    norm.test_forward("no eps")
    norm.test_backward("no eps")


# x, groups, and positions of an infinity: [.., channel of the group's sixteen or more]
PLACES = [((3, 20, 64), 4, [(1, 0, 20), (1, 0, 21), (1, 7, 18), (1, 19, 31)]),               # a workgroup a sample
          ((2, 20000, 32), 2, [(1, 0, 17), (1, 9, 21), (1, 12345, 16), (1, 19999, 31)]),     # many chunks a sample
          ((2, 10, 6000), 2, [(1, 0, 3001), (1, 9, 3777), (1, 4, 5999)]),                    # groups wider than a workgroup
          ((3, 9000), 1, [(1, 0), (1, 1), (1, 5003), (1, 8999)]),                            # rows wider than one
          ((40, 64), 4, [(1, 16), (1, 21), (1, 31)])]


@pytest.mark.parametrize("type", [BF, F32])
@pytest.mark.parametrize("act", [None, "silu"])
@pytest.mark.parametrize("shape,groups,places", PLACES)
def test_an_infinity_anywhere_turns_its_group_to_nan(shape, groups, places, act, type):
    s, go = norm.make(shape=shape, groups=groups, act=act, type=type)
    clean, grads, x = sx.group_norm(**s), sx.group_norm_backward(grad_out=go, **s), s["x"].clone()
    per = shape[-1] // groups
    for place in places:
        for value in (float("inf"), float("-inf"), float("nan")):
            s["x"].copy_(x)
            s["x"][place] = value
            first = place[-1] // per * per
            bad = torch.zeros_like(clean, dtype=torch.bool)
            bad[place[0], ..., first:first + per] = True
            out, got = sx.group_norm(**s), sx.group_norm_backward(grad_out=go, **s)
            for a, b in ((out, clean), (got[0], grads[0])):
                assert torch.isnan(a[bad]).all() and torch.equal(a[~bad], b[~bad]), (place, value)
            keep = torch.ones(shape[-1], dtype=torch.bool, device=DEV)
            keep[first:first + per] = False
            assert torch.equal(got[1][keep], grads[1][keep]) and torch.equal(got[2][keep], grads[2][keep])


@pytest.mark.parametrize("type", [BF, F32])
@pytest.mark.parametrize("shape,groups", [((40, 64), 4), ((3, 20, 64), 4), ((1, 20000, 32), 2), ((2, 10, 6000), 2),
                                          ((3, 9000), 1)])
def test_squares_past_the_range_are_an_infinite_variance(shape, groups, type):
    s, go = norm.make(shape=shape, groups=groups, type=type)
    for size in (1e20, 1e30):
        big = dict(s, x=s["x"] * size)
        out, got = sx.group_norm(**big), sx.group_norm_backward(grad_out=go, **big)
        assert torch.equal(out, s["bias"].expand(shape).to(type))
        assert not got[0].any() and not got[1].any()
        assert torch.isfinite(got[2]).all() and got[2].any()


def test_group_counts_past_64_bits():
    s, go = norm.make(shape=(6, 32), type=F32)
    for groups in (2 ** 64 + 4, 4 - 2 ** 64, 2 ** 63, 4.0, "4", None):
        for call in (lambda g: sx.group_norm(s["x"], g), lambda g: sx.group_norm_backward(s["x"], g, go)):
            with pytest.raises(sx.SxError) as e:
                call(groups)
            assert e.value.code == B.SX_E_DIM_001, groups
    want = sx.group_norm(s["x"], 4)
    for groups in (torch.tensor([4, 8]).numpy()[0], torch.tensor(4)):
        assert torch.equal(sx.group_norm(s["x"], groups), want)


@pytest.mark.parametrize("far", [300.0, 1e5])
@pytest.mark.parametrize("shape,groups,first", [((1, 200000, 16), 4, 800), ((1, 1000000, 4), 1, 4000),
                                                ((2, 4096, 512), 32, 16), ((2, 4096, 512), 32, 1), ((4, 9000), 1, 8)])
def test_what_stands_first_may_lie_far_from_the_rest(shape, groups, first, far):
    # A thread sums at most 64 values (of a wide row 36) and a workgroup its 256 threads' about references that one
    # outlier does not move far, chunks are joined in 64 bits: 8 (sqrt(64) + sqrt(256)) steps of the variance, half as many
    # of its root, and 16 for the rest.
    s, _ = norm.make(shape=shape, groups=groups, type=F32)
    s["x"][:, :first] += far
    size, *_ = norm._size(s)
    close("out", sx.group_norm(**s), os_.group_norm(**norm._host(s)), size, 4 * (64 ** 0.5 + 256 ** 0.5) + 16)


@pytest.mark.parametrize("value", [0.1, 2e38, -3.3e38])
@pytest.mark.parametrize("shape,groups", [((3, 20, 64), 4), ((1, 20000, 32), 2), ((2, 10, 6000), 2), ((2, 300, 33), 3)])
def test_equal_values_of_any_size_have_no_variance(shape, groups, value):
    s, go = norm.make(shape=shape, groups=groups, type=F32)
    s["x"].fill_(value)
    assert torch.equal(sx.group_norm(**s), s["bias"].expand(shape))
    assert all(torch.isfinite(t).all() for t in sx.group_norm_backward(grad_out=go, **s))
