"""A small model of multi-head scan layers: training, a prompt, single tokens.

Each layer is the norm with its residual add (AddNorm), one projection into
z, x, B, C and the step, the multi-head scan (HeadsScan), the norm with the
gate (GatedNorm) and the projection back.  The model learns to answer with the
token it saw `LAG` positions before; then a prompt is run as a whole, its states are
kept, and the tokens after it go through the single-token entry points.  Both
ways give the same logits up to rounding.

    python examples/heads_block.py [--steps 200] [--dtype bf16|f32]
"""
import argparse
import math
import os
import sys

import torch
from torch import nn
from torch.nn import functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from selective_state_space_63_amd import block  # noqa: E402

LAG = 2


class HeadsLayer(nn.Module):
    def __init__(self, dim, heads, headdim, groups, dstate, dtype):
        super().__init__()
        self.heads, self.headdim, self.groups, self.dstate = heads, headdim, groups, dstate
        self.inner, self.state_row = heads * headdim, groups * dstate
        self.norm = nn.Parameter(torch.ones(dim))
        self.gate_norm = nn.Parameter(torch.ones(self.inner))
        self.widths = [self.inner, self.inner, self.state_row, self.state_row, heads]
        self.row = sum(self.widths) + -sum(self.widths) % 8  # rows of 16 bytes
        self.w_in = nn.Parameter(torch.randn(self.row, dim) / math.sqrt(dim))
        self.w_out = nn.Parameter(torch.randn(dim, self.inner) / math.sqrt(self.inner))
        self.A_log = nn.Parameter(torch.linspace(0, math.log(8), heads))
        self.D = nn.Parameter(torch.ones(heads))
        self.delta_bias = nn.Parameter(torch.full((heads,), -1.0))
        self.dtype = dtype

    def project(self, u):
        """z, x, delta, B, C as slices of one row per token."""
        row = F.linear(u, self.w_in.to(self.dtype))
        z, x, B, C, delta = row[..., :sum(self.widths)].split(self.widths, -1)
        groups = (self.groups, self.dstate)
        return z, x.unflatten(-1, (self.heads, self.headdim)), delta, B.unflatten(-1, groups), C.unflatten(-1, groups)

    def forward(self, u, residual, h0=None):
        """u, residual: (batch, seqlen, dim) -> the same, and the states after
        the last token."""
        u, residual = block.AddNorm.apply(u, self.norm, residual)
        z, x, delta, B, C = self.project(u)
        y, h = block.HeadsScan.apply(x, delta, -self.A_log.exp(), B, C, self.D, h0, self.delta_bias, True)
        out = block.GatedNorm.apply(y.flatten(-2), z, self.gate_norm)
        return F.linear(out, self.w_out.to(self.dtype)), residual, h

    def step(self, u, residual, h):
        """One token: u, residual: (batch, dim); h is advanced in place."""
        u, residual = block.add_norm_fwd(u, self.norm, residual=residual)
        z, x, delta, B, C = self.project(u)
        y = block.heads_state_update(h, x, delta, -self.A_log.exp(), B, C, D=self.D, delta_bias=self.delta_bias,
                                     delta_softplus=True)
        out = block.gated_norm_fwd(y.flatten(-2), z, self.gate_norm)
        return F.linear(out, self.w_out.to(self.dtype)), residual


class Model(nn.Module):
    def __init__(self, vocab=32, dim=128, layers=2, heads=4, headdim=64, groups=1, dstate=64, dtype=torch.bfloat16):
        super().__init__()
        self.dtype = dtype
        self.embed = nn.Parameter(torch.randn(vocab, dim))
        self.layers = nn.ModuleList(HeadsLayer(dim, heads, headdim, groups, dstate, dtype) for _ in range(layers))
        self.norm = nn.Parameter(torch.ones(dim))
        self.head = nn.Parameter(torch.randn(vocab, dim) / math.sqrt(dim))

    def forward(self, tokens, states=None):
        """Logits of (batch, seqlen) tokens and every layer's final state."""
        u, residual, out = F.embedding(tokens, self.embed).to(self.dtype), None, []
        for i, layer in enumerate(self.layers):
            u, residual, h = layer(u, residual, None if states is None else states[i])
            out.append(h)
        u, _ = block.AddNorm.apply(u, self.norm, residual)
        return F.linear(u, self.head.to(self.dtype)).float(), out

    @torch.no_grad()
    def step(self, tokens, states):
        """Logits of one token per sequence; the states are advanced in place."""
        u, residual = F.embedding(tokens, self.embed).to(self.dtype), None
        for layer, h in zip(self.layers, states):
            u, residual = layer.step(u, residual, h)
        u, _ = block.add_norm_fwd(u, self.norm, residual=residual)
        return F.linear(u, self.head.to(self.dtype)).float()


def train(model, steps, batch=16, seqlen=96, vocab=32, lr=3e-3, seed=0):
    """The losses of `steps` steps."""
    gen = torch.Generator("cuda").manual_seed(seed)
    opt = torch.optim.Adam(model.parameters(), lr=lr)
    losses = []
    for _ in range(steps):
        tokens = torch.randint(vocab, (batch, seqlen), device="cuda", generator=gen)
        logits, _ = model(tokens)
        loss = F.cross_entropy(logits[:, LAG:].flatten(0, 1), tokens[:, :-LAG].flatten())
        opt.zero_grad(set_to_none=True)
        loss.backward()
        opt.step()
        losses.append(loss.detach())
    return torch.stack(losses).tolist()


@torch.no_grad()
def prompt_then_tokens(model, tokens, prompt):
    """Logits of tokens[:, prompt:], one token at a time after a prompt."""
    _, states = model(tokens[:, :prompt])
    return torch.stack([model.step(tokens[:, t], states) for t in range(prompt, tokens.shape[1])], 1)


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--dtype", choices=("bf16", "f32"), default="bf16")
    a = ap.parse_args()
    torch.manual_seed(0)
    model = Model(dtype=torch.bfloat16 if a.dtype == "bf16" else torch.float32).cuda()
    losses = train(model, a.steps)
    for i in range(0, len(losses), max(1, len(losses) // 10)):
        print(f"step {i}: loss {losses[i]:.3f}")
    tokens = torch.randint(32, (4, 120), device="cuda")
    got = prompt_then_tokens(model, tokens, 70)
    with torch.no_grad():
        want = model(tokens)[0][:, 70:]
    print(f"answers right: {(got.argmax(-1) == tokens[:, 70 - LAG:-LAG]).float().mean().item():.3f}; logits of prompt and "
          f"tokens against the whole sequence: {((got - want).norm() / want.norm()).item():.1e}")


if __name__ == "__main__":
    main()
