"""The example layer: the operators together, as a server and a trainer use them."""

import pytest
import torch

from examples.linear_attention_layer import LinearAttentionLayer, prompt_then_tokens, train

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("type", [torch.float32, torch.bfloat16])
def test_tokens_after_a_prompt_are_the_prompt(type):
    torch.manual_seed(1)
    layer = LinearAttentionLayer(width=64, heads=4, key_heads=2, head_width=32).to("cuda")
    if type == torch.bfloat16:
        layer.bfloat16_projections()
    x = torch.randn(3, 90, 64, device="cuda", dtype=type)
    got = prompt_then_tokens(layer, x, [70, 1, 64], 16)
    with torch.no_grad():
        whole = layer(x, torch.arange(90, device="cuda"))
    want = torch.stack([whole[i, n:n + 16] for i, n in enumerate([70, 1, 64])]).float()
    # f32: sums of up to 90 tokens and 128 inputs in another order. bf16: every stage rounds (projection, norm,
    # attention, projection), and the two ways round the same values apart by a step of 2^-7 here and there.
    tol = 1e-5 if type == torch.float32 else 4 * 2.0 ** -7
    assert (got.float() - want).abs().max() <= tol * want.abs().max()


def test_training_learns_the_token_before():
    torch.manual_seed(2)
    layer = LinearAttentionLayer(width=32, heads=4, key_heads=2, head_width=32).to("cuda")
    losses = train(layer, steps=40)
    assert losses[-1] < 0.8 * losses[0]


def test_gradients_match_differences():
    torch.manual_seed(3)
    layer = LinearAttentionLayer(width=16, heads=4, key_heads=2, head_width=16).to("cuda")
    x = torch.randn(2, 70, 16, device="cuda")
    positions = torch.arange(70, device="cuda")
    weight = torch.randn(2, 70, 16, device="cuda")
    loss = lambda: (layer(x, positions).double() * weight).sum()  # noqa: E731
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
        # the third derivative's share e^2, and f32 sums of 2 x 70 x 16 terms over 2 e
        assert abs(got - want) <= 1e-2 * abs(want) + 2e-2 * p.grad.double().norm().item(), name
