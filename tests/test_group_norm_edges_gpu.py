"""Group norm where its arithmetic ends: no eps, infinities anywhere in a group, squares past f32's range."""

import pytest
import torch

import scan_primitives_amd as sx
from scan_primitives_amd import _binding as B
from tests import test_group_norm_gpu as norm
from tests.test_causal_conv_gpu import BF, DEV, F32

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
