"""A layer on a selective state space, on the package's operators: a prompt, single tokens, a training step.

``python examples/state_space_layer.py`` (one MI355X) runs a padded batch of
prompts through the layer, goes on token by token from what the prompts left in
two pools, checks that against the same tokens run as one prompt, and takes a
few training steps on a toy task.
"""

import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import scan_primitives_amd as sx  # noqa: E402


class StateSpaceLayer(torch.nn.Module):
    """A short convolution, the scan, gated, and a norm of groups of channels. A request leaves behind the
    convolution's last inputs, [taps - 1, inner], and the states, [inner, states] in f32."""

    def __init__(self, width: int, inner: int, states: int = 16, groups: int = 1, taps: int = 4, norm_groups: int = 4):
        super().__init__()
        self.inner, self.states, self.groups, self.norm_groups = inner, states, groups, norm_groups
        self.narrow = max(1, width // 16)
        self.into = torch.nn.Linear(width, 2 * inner, bias=False)
        self.rows = torch.nn.Linear(inner, self.narrow + 2 * groups * states, bias=False)
        self.delta = torch.nn.Linear(self.narrow, inner, bias=False)
        self.out = torch.nn.Linear(inner, width, bias=False)
        self.taps = torch.nn.Parameter((2 * torch.rand(inner, taps) - 1) * taps ** -0.5)
        self.taps_bias = torch.nn.Parameter(torch.zeros(inner))
        # steps of 1e-3 to 1e-1 and rates of 1 to `states`
        dt = torch.exp(torch.rand(inner) * math.log(100.0) + math.log(1e-3))
        self.delta_bias = torch.nn.Parameter(dt + torch.log(-torch.expm1(-dt)))
        self.log_rates = torch.nn.Parameter(torch.arange(1, states + 1).float().log().repeat(inner, 1))
        self.skip = torch.nn.Parameter(torch.ones(inner))
        self.norm_weight = torch.nn.Parameter(torch.ones(inner))
        self.norm_bias = torch.nn.Parameter(torch.zeros(inner))

    def bfloat16_projections(self):
        """The projections in bf16; everything else stays f32, as the operators take it."""
        for linear in (self.into, self.rows, self.delta, self.out):
            linear.to(torch.bfloat16)
        return self

    def row_parts(self, x):
        """delta, b and c of the convolution's outputs [.., inner]."""
        rows = self.rows(x)
        n = self.groups * self.states
        b, c = (rows[..., self.narrow + i * n:self.narrow + (i + 1) * n].unflatten(-1, (self.groups, self.states))
                for i in (0, 1))
        return self.delta(rows[..., :self.narrow]), b, c

    def leave(self, y):
        """The norm of each token's groups of channels and the last projection, of y [.., inner]."""
        n = sx.group_norm(y.reshape(-1, self.inner), self.norm_groups, weight=self.norm_weight, bias=self.norm_bias)
        return self.out(n.reshape(y.shape))

    def forward(self, x, states=(None, None), lengths=None, return_states=False):
        inner = self.into(x)
        u, inputs = sx.causal_conv(inner[..., :self.inner], self.taps, bias=self.taps_bias, initial=states[0],
                                   lengths=lengths, activation="silu", return_state=True)
        delta, b, c = self.row_parts(u)
        y, h = sx.selective_scan(u, delta, -self.log_rates.exp(), b, c, skip=self.skip, z=inner[..., self.inner:],
                                 delta_bias=self.delta_bias, initial=states[1], lengths=lengths, return_state=True)
        out = self.leave(y)
        return (out, (inputs, h)) if return_states else out

    def step(self, x, pools, slots):
        """The next token of each row, x [B, width]: its states in the two pools are read and updated."""
        inner = self.into(x)
        u = sx.causal_conv_step(inner[..., :self.inner], self.taps, pools[0], bias=self.taps_bias, slots=slots,
                                activation="silu")
        delta, b, c = self.row_parts(u)
        y = sx.selective_scan_step(u, delta, -self.log_rates.exp(), b, c, pools[1], slots=slots, skip=self.skip,
                                   z=inner[..., self.inner:], delta_bias=self.delta_bias)
        return self.leave(y)


def prompt_then_tokens(layer, x, prompt_lengths, tokens):
    """Prompts of the given lengths (the start of each row of x), then `tokens` tokens one by one: their outputs."""
    b, dev = x.shape[0], x.device
    lengths = torch.tensor(prompt_lengths, dtype=torch.int32, device=dev)
    with torch.no_grad():
        _, states = layer(x[:, :max(prompt_lengths)], lengths=lengths, return_states=True)
        # a server's pools: two more states than requests
        pools = [torch.zeros(b + 2, *s.shape[1:], dtype=s.dtype, device=dev) for s in states]
        slots = torch.arange(b, dtype=torch.int32, device=dev) + 1
        for pool, s in zip(pools, states):
            pool[1:b + 1] = s
        rows, at, out = torch.arange(b, device=dev), lengths.long(), []
        for _ in range(tokens):
            out.append(layer.step(x[rows, at], pools, slots))
            at = at + 1
    return torch.stack(out, 1)


def train(layer, steps=20, seed=0):
    """Learns to answer each token with the one before it; the losses."""
    gen = torch.Generator().manual_seed(seed)
    dev, width = layer.skip.device, layer.into.in_features
    opt = torch.optim.Adam(layer.parameters(), lr=3e-3)
    losses = []
    for _ in range(steps):
        x = torch.randn(4, 96, width, generator=gen).to(dev)
        want = torch.cat([torch.zeros_like(x[:, :1]), x[:, :-1]], 1)
        loss = (layer(x) - want).square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.item())
    return losses


def main():
    torch.manual_seed(0)
    layer = StateSpaceLayer(width=64, inner=128).to("cuda").bfloat16_projections()
    x = torch.randn(3, 80, 64, device="cuda", dtype=torch.bfloat16)
    got = prompt_then_tokens(layer, x, [50, 7, 64], 12)
    with torch.no_grad():
        whole = layer(x)
    want = torch.stack([whole[i, n:n + 12] for i, n in enumerate([50, 7, 64])])
    print(f"12 tokens after prompts of 50, 7 and 64: {(got - want).abs().max().item():.1e} from the same tokens as "
          f"one prompt (outputs of {want.float().std().item():.1e})")
    layer = StateSpaceLayer(width=64, inner=128).to("cuda")
    losses = train(layer)
    print(f"training: loss {losses[0]:.3f} to {losses[-1]:.3f} in {len(losses)} steps")


if __name__ == "__main__":
    main()
