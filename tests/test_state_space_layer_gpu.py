"""The example layer: convolution, scan and norm together, as a server and a trainer use them; and the norm behind
decay attention."""

import pytest
import torch

import scan_primitives_amd as sx
from examples.state_space_layer import StateSpaceLayer, prompt_then_tokens, train

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("type", [torch.float32, torch.bfloat16])
def test_tokens_after_a_prompt_are_the_prompt(type):
    torch.manual_seed(1)
    layer = StateSpaceLayer(width=64, inner=96, states=8, groups=2).to("cuda")
    if type == torch.bfloat16:
        layer.bfloat16_projections()
    x = torch.randn(3, 90, 64, device="cuda", dtype=type)
    got = prompt_then_tokens(layer, x, [70, 1, 64], 16)
    with torch.no_grad():
        whole = layer(x)
    want = torch.stack([whole[i, n:n + 16] for i, n in enumerate([70, 1, 64])]).float()
    # f32: sums of up to 90 tokens and 96 inputs in another order. bf16: every stage rounds (three projections, the
    # convolution, the scan, the norm, which divides by a group's spread), and the two ways round the same values
    # apart by a step of 2^-7 here and there.
    tol = 2e-5 if type == torch.float32 else 6 * 2.0 ** -7
    assert (got.float() - want).abs().max() <= tol * want.abs().max()


def test_training_runs():
    torch.manual_seed(2)
    losses = train(StateSpaceLayer(width=32, inner=64, states=4).to("cuda"), steps=5)
    assert all(torch.isfinite(torch.tensor(losses)))


def test_gradients_match_differences():
    torch.manual_seed(3)
    layer = StateSpaceLayer(width=16, inner=32, states=4, groups=2).to("cuda")
    x = torch.randn(2, 70, 16, device="cuda")
    weight = torch.randn(2, 70, 16, device="cuda")
    loss = lambda: (layer(x).double() * weight).sum()  # noqa: E731
    loss().backward()
    for name, p in layer.named_parameters():
        d = torch.randn_like(p)
        e = 1e-2 / d.abs().max().item()
        with torch.no_grad():
            p.add_(e * d)
            up = loss()
            p.sub_(2 * e * d)
            down = loss()
            p.add_(e * d)
        want, got = ((up - down) / (2 * e)).item(), (p.grad.double() * d).sum().item()
        # the third derivative's share e^2 times what a norm's root makes of it, and f32 sums of 2 x 70 x 16 terms
        # over 2 e
        assert abs(got - want) <= 2e-2 * abs(want) + 3e-2 * p.grad.double().norm().item(), name


def test_the_norm_of_heads_behind_decay_attention():
    torch.manual_seed(4)
    q, k, v = (torch.randn(2, 50, 4, 32, device="cuda") for _ in range(3))
    g = -torch.rand(2, 50, 4, device="cuda")
    leaves = [x.requires_grad_() for x in (q, k, v, g)]
    o = sx.decay_attention(q, k, v, g)
    got = sx.group_norm(o.reshape(100, 128), 4, eps=1e-6)
    o64 = o.detach().double().reshape(100, 4, 32)
    want = (o64 - o64.mean(-1, keepdim=True)) / (o64.var(-1, unbiased=False, keepdim=True) + 1e-6).sqrt()
    # means and variances of 32 values: 8 sqrt(32) + 24 steps of 2^-24 of values up to (|o| + mean) / root
    size = (o64.abs() + o64.abs().mean(-1, keepdim=True)) / (o64.var(-1, unbiased=False, keepdim=True) + 1e-6).sqrt()
    assert ((got.double().reshape(want.shape) - want).abs() <= 70 * 2.0 ** -24 * size).all()
    weight = torch.randn_like(got)
    (got * weight).sum().backward()
    go = sx.group_norm_backward(o.detach().reshape(100, 128), 4, weight, eps=1e-6)[0].reshape(o.shape)
    for leaf, grad in zip(leaves, sx.decay_attention_backward(q.detach(), k.detach(), v.detach(), g.detach(), go)):
        assert torch.equal(leaf.grad, grad)
