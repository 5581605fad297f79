"""A linear-attention layer on the package's operators: a prompt, single tokens, a training step.

``python examples/linear_attention_layer.py`` (one MI355X) runs a padded batch
of prompts through the layer, goes on token by token from the states the
prompts left in a pool, checks that against the same tokens run as one prompt,
and takes a few training steps on a toy task.
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import scan_primitives_amd as sx  # noqa: E402


class LinearAttentionLayer(torch.nn.Module):
    """Queries and keys are normed a head and turned by position; each value head forgets at a rate that the
    token sets. The state, [heads, width, width] in f32, is all that a request leaves behind."""

    def __init__(self, width: int, heads: int, key_heads: int, head_width: int, base: float = 10000.0):
        super().__init__()
        self.heads, self.key_heads, self.head_width = heads, key_heads, head_width
        self.qkv = torch.nn.Linear(width, (2 * key_heads + heads) * head_width, bias=False)
        self.forget = torch.nn.Linear(width, heads)
        self.out = torch.nn.Linear(heads * head_width, width, bias=False)
        self.q_weight = torch.nn.Parameter(torch.ones(head_width))
        self.k_weight = torch.nn.Parameter(torch.ones(head_width))
        self.register_buffer("turns", sx.rotation_turns(head_width, base), persistent=False)
        torch.nn.init.constant_(self.forget.bias, 4.0)

    def bfloat16_projections(self):
        """The projections in bf16; the norms' weights (f32) and the turns (f64) stay as the operators take them."""
        for linear in (self.qkv, self.forget, self.out):
            linear.to(torch.bfloat16)
        return self

    def project(self, x, positions):
        """q, k, v and the log decay of x [B, T, width]."""
        b, t, _ = x.shape
        h, hk, d = self.heads, self.key_heads, self.head_width
        qkv = self.qkv(x)
        q, k = qkv[..., :hk * d].view(b, t, hk, d), qkv[..., hk * d:2 * hk * d].view(b, t, hk, d)
        v = qkv[..., 2 * hk * d:].view(b, t, h, d)
        q, k = sx.head_norm_rotate(q, k, positions, self.turns, q_weight=self.q_weight, k_weight=self.k_weight)
        return q, k, v, torch.nn.functional.logsigmoid(self.forget(x).float())

    def forward(self, x, positions, initial=None, lengths=None, return_state=False):
        b, t, _ = x.shape
        q, k, v, g = self.project(x, positions)
        o, state = sx.decay_attention(q, k, v, g, initial=initial, lengths=lengths, scale=self.head_width ** -0.5,
                                      return_state=True)
        y = self.out(o.reshape(b, t, -1))
        return (y, state) if return_state else y

    def step(self, x, positions, pool, slots):
        """The next token of each row, x [B, width]: its state in the pool is read and updated."""
        q, k, v, g = self.project(x[:, None], positions[:, None])
        o = sx.decay_attention_step(q[:, 0], k[:, 0], v[:, 0], g[:, 0], pool, slots=slots,
                                    scale=self.head_width ** -0.5)
        return self.out(o.reshape(x.shape[0], -1))


def prompt_then_tokens(layer, x, prompt_lengths, tokens):
    """Prompts of the given lengths (the start of each row of x), then `tokens` tokens one by one: their outputs."""
    b, dev = x.shape[0], x.device
    most = max(prompt_lengths)
    lengths = torch.tensor(prompt_lengths, dtype=torch.int32, device=dev)
    positions = torch.arange(x.shape[1], device=dev).expand(b, -1)
    with torch.no_grad():
        _, state = layer(x[:, :most].contiguous(), positions[:, :most], lengths=lengths, return_state=True)
        pool = torch.zeros(b + 2, *state.shape[1:], device=dev)  # a server's pool: two more states than requests
        slots = torch.arange(b, dtype=torch.int32, device=dev) + 1
        pool[1:b + 1] = state
        rows, at, out = torch.arange(b, device=dev), lengths.long(), []
        for _ in range(tokens):
            out.append(layer.step(x[rows, at], at, pool, slots))
            at = at + 1
    return torch.stack(out, 1)


def train(layer, steps=20, seed=0):
    """Learns to answer each token with the one before it; the losses."""
    gen = torch.Generator().manual_seed(seed)
    dev = layer.turns.device
    width = layer.qkv.in_features
    opt = torch.optim.Adam(layer.parameters(), lr=3e-3)
    positions = torch.arange(96, device=dev)
    losses = []
    for _ in range(steps):
        x = torch.randn(4, 96, width, generator=gen).to(dev)
        want = torch.cat([torch.zeros_like(x[:, :1]), x[:, :-1]], 1)
        loss = (layer(x, positions) - want).square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.item())
    return losses


def main():
    torch.manual_seed(0)
    layer = LinearAttentionLayer(width=64, heads=4, key_heads=2, head_width=32).to("cuda").bfloat16_projections()
    x = torch.randn(3, 80, 64, device="cuda", dtype=torch.bfloat16)
    got = prompt_then_tokens(layer, x, [50, 7, 64], 12)
    with torch.no_grad():
        whole = layer(x, torch.arange(80, device="cuda"))
    want = torch.stack([whole[i, n:n + 12] for i, n in enumerate([50, 7, 64])])
    print(f"12 tokens after prompts of 50, 7 and 64: {(got - want).abs().max().item():.1e} from the same tokens as "
          f"one prompt (outputs of {want.float().std().item():.1e})")
    layer = LinearAttentionLayer(width=64, heads=4, key_heads=2, head_width=32).to("cuda")
    losses = train(layer)
    print(f"training: loss {losses[0]:.3f} to {losses[-1]:.3f} in {len(losses)} steps")


if __name__ == "__main__":
    main()
