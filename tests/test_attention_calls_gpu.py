"""How decay attention and head norm + rotation are called: optional values of any truth."""

import numpy as np
import pytest
import torch

import scan_primitives_amd as sx
from tests.test_decay_attention_gpu import make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("true,false", [(1, 0), (np.bool_(True), np.bool_(False)), ("yes", "")])
def test_whether_the_state_is_wanted_goes_by_truth(true, false):
    s = make(t=70, initial=True)
    args = dict(initial=s["initial"], scale=s["scale"])
    out, state = sx.decay_attention(s["q"], s["k"], s["v"], s["g"], return_state=True, **args)
    got = sx.decay_attention(s["q"], s["k"], s["v"], s["g"], return_state=true, **args)
    assert torch.equal(got[0], out) and torch.equal(got[1], state)
    assert torch.equal(sx.decay_attention(s["q"], s["k"], s["v"], s["g"], return_state=false, **args), out)
