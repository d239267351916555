"""A small language model on the library's layer norm, causal convolution,
norms of queries and keys with rotation, and gated delta rule: trained for a
few steps on a toy task, then served one token at a time from a prompt's
states.

    python examples/delta_block.py            # on a GB300
"""
import os
import sys

import torch
from torch import nn

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from bidirectional_masked_linear_gb300 import delta, ssm  # noqa: E402


class Block(nn.Module):
    """x + out(delta rule(norms(convolution(in(norm(x)))))), decays and step sizes from the same in-projection."""

    def __init__(self, width, heads, d, K=4):
        super().__init__()
        self.heads, self.d, self.inner = heads, d, heads * d
        self.norm_weight, self.norm_bias = nn.Parameter(torch.ones(width)), nn.Parameter(torch.zeros(width))
        self.in_proj = nn.Linear(width, 3 * self.inner + 2 * heads, bias=False)
        self.taps = nn.Parameter(torch.randn(3 * self.inner, K) / K)
        self.rate = nn.Parameter(torch.linspace(-4.0, -1.0, heads))   # a head's decay without its input
        self.register_buffer("freqs", 100.0 ** (-torch.arange(d // 2) / (d // 2)))
        self.out_proj = nn.Linear(self.inner, width, bias=False)

    def project(self, x):
        """(what the convolution takes, the decays' logarithms, beta)."""
        p = self.in_proj(ssm.LayerNorm.apply(x, self.norm_weight, self.norm_bias, 1e-5))
        g = -nn.functional.softplus(p[..., 3 * self.inner:-self.heads] + self.rate)
        return p[..., :3 * self.inner], g, torch.sigmoid(p[..., -self.heads:])

    def split(self, u):
        """q, k and v, slices of one tensor."""
        return (t.unflatten(-1, (self.heads, self.d)) for t in u.split(self.inner, -1))

    def forward(self, x, lengths=None):
        u, g, beta = self.project(x)
        q, k, v = self.split(ssm.CausalConv.apply(u, self.taps, None, "silu", None, lengths))
        q, k = delta.QKNorm.apply(q, k, None, None, "l2", 1e-6, self.freqs)
        y = delta.GatedDelta.apply(q, k, v, g, beta, None, None, lengths)
        return x + self.out_proj(y.flatten(2))

    def prompt(self, x, lengths=None):
        """As forward, with the states that decoding goes on from."""
        u, g, beta = self.project(x)
        u, conv = ssm.conv_fwd(u, self.taps, lengths=lengths, return_state=True)
        q, k, v = self.split(u)
        q, k = delta.qknorm_fwd(q, k, freqs=self.freqs)
        f = delta.delta_fwd(q, k, v, g, beta, lengths=lengths, return_state=True)
        return x + self.out_proj(f.out.flatten(2)), (conv, f.h)

    def step(self, x, states, positions):
        """One token of each sequence, at `positions` [B, 1]."""
        conv, h = states
        u, g, beta = self.project(x)
        u = ssm.conv_step(u.contiguous(), conv, self.taps)
        q, k, v = self.split(u.unsqueeze(1))
        q, k = delta.qknorm_fwd(q, k, freqs=self.freqs, positions=positions)
        y = delta.delta_step(h, q[:, 0], k[:, 0], v[:, 0].contiguous(), g, beta)
        return x + self.out_proj(y.flatten(1))


class Model(nn.Module):
    def __init__(self, vocab=16, width=64, heads=2, d=32, depth=2):
        super().__init__()
        self.embed = nn.Embedding(vocab, width)
        self.blocks = nn.ModuleList(Block(width, heads, d) for _ in range(depth))
        self.head = nn.Linear(width, vocab, bias=False)

    def forward(self, tokens, lengths=None):
        x = self.embed(tokens)
        for b in self.blocks:
            x = b(x, lengths)
        return self.head(x)

    def prompt(self, tokens, lengths=None):
        x, states = self.embed(tokens), []
        for b in self.blocks:
            x, s = b.prompt(x, lengths)
            states.append(s)
        return self.head(x), states

    def step(self, tokens, states, positions):
        x = self.embed(tokens)
        for b, s in zip(self.blocks, states):
            x = b.step(x, s, positions)
        return self.head(x)


def batch(n, pairs, vocab, generator):
    """Keys with values, then the keys again: the values are what follows them."""
    keys = torch.stack([torch.randperm(vocab // 2, generator=generator)[:pairs] for _ in range(n)])
    values = vocab // 2 + torch.randint(vocab // 2, (n, pairs), generator=generator)
    seen = torch.stack((keys, values), -1).flatten(1)
    return torch.cat((seen, seen), 1)


def train(model, steps, lr=3e-3, seed=0):
    gen = torch.Generator().manual_seed(seed)
    opt = torch.optim.AdamW(model.parameters(), lr=lr)
    losses = []
    for _ in range(steps):
        t = batch(32, 6, 16, gen).cuda()
        logits = model(t[:, :-1].contiguous())[:, 12::2]   # where a key was seen before
        loss = nn.functional.cross_entropy(logits.flatten(0, 1), t[:, 13::2].flatten())
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(float(loss.detach()))
    return losses


@torch.no_grad()
def serve_error(model, seed=1):
    """How far a prompt followed by single tokens is from the whole sequences, ragged ones."""
    gen = torch.Generator().manual_seed(seed)
    t = torch.randint(0, 16, (3, 60), generator=gen).cuda()
    n = torch.tensor([50, 7, 33], dtype=torch.int32, device="cuda")
    whole = model(t)
    got, states = model.prompt(t[:, :50].contiguous(), n)
    off = max(float((got[b, :n[b]] - whole[b, :n[b]]).abs().max()) for b in range(3))
    rows = torch.arange(3, device="cuda")
    for k in range(10):
        at = (n + k).long()
        got = model.step(t[rows, at], states, (n + k).unsqueeze(1))
        off = max(off, float((got - whole[rows, at]).abs().max()))
    return off / float(whole.abs().max())


if __name__ == "__main__":
    torch.manual_seed(0)
    m = Model().cuda()
    losses = train(m, 300)
    print(f"loss {losses[0]:.3f} -> {losses[-1]:.3f}")
    print(f"tokens after a prompt are {serve_error(m):.1e} off the whole sequence")
