"""A small state space model on the library's layer norm, causal convolution
and selective scan: trained for a few steps on a toy task, then served one
token at a time from a prompt's states.

    python examples/ssm_block.py            # on a GB300

``Block(..., directions=2)`` also walks the tokens from the last to the first
and adds the two, as an encoder of images or text does; such a block has no
one-token form.
"""
import os
import sys

import torch
from torch import nn

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from bidirectional_masked_linear_gb300 import ssm  # noqa: E402


class Mixer(nn.Module):
    """Convolution and scan in one direction, on the two halves of the in-projection."""

    def __init__(self, inner, N, rank, K=4):
        super().__init__()
        self.N, self.rank = N, rank
        self.taps = nn.Parameter(torch.randn(inner, K) / K)
        self.tap_bias = nn.Parameter(torch.zeros(inner))
        self.x_proj = nn.Linear(inner, rank + 2 * N, bias=False)
        self.dt_proj = nn.Linear(rank, inner, bias=False)
        step = torch.exp(torch.empty(inner).uniform_(-6.9, -2.3))   # 0.001 .. 0.1
        self.dt_bias = nn.Parameter(step + torch.log(-torch.expm1(-step)))
        self.A_log = nn.Parameter(torch.log(torch.arange(1.0, N + 1)).repeat(inner, 1))
        self.D = nn.Parameter(torch.ones(inner))

    def steps(self, u):
        """(dt, B, C) of the convolution's output; B and C stay slices of one tensor."""
        p = self.x_proj(u)
        return self.dt_proj(p[..., :self.rank]), p[..., self.rank:self.rank + self.N], p[..., self.rank + self.N:]

    def forward(self, x, z, lengths, reverse):
        u = ssm.CausalConv.apply(x, self.taps, self.tap_bias, "silu", None, lengths, reverse)
        dt, Bm, Cm = self.steps(u)
        return ssm.SelectiveScan.apply(u, dt, -torch.exp(self.A_log), Bm, Cm, self.D, z, self.dt_bias, True, None,
                                       lengths, reverse)

    def prompt(self, x, z, lengths):
        """As forward from the left, with the states that decoding goes on from."""
        u, conv = ssm.conv_fwd(x, self.taps, self.tap_bias, lengths=lengths, return_state=True)
        dt, Bm, Cm = self.steps(u)
        f = ssm.scan_fwd(u, dt, -torch.exp(self.A_log), Bm, Cm, self.D, z, self.dt_bias, lengths=lengths,
                         return_state=True)
        return f.out, (conv, f.h)

    def step(self, x, z, states):
        conv, h = states
        u = ssm.conv_step(x, conv, self.taps, self.tap_bias)
        dt, Bm, Cm = self.steps(u)
        return ssm.scan_step(h, u, dt, -torch.exp(self.A_log), Bm.contiguous(), Cm.contiguous(), self.D, z,
                             self.dt_bias)


class Block(nn.Module):
    def __init__(self, width, N=16, directions=1):
        super().__init__()
        self.inner = 2 * width
        self.norm_weight, self.norm_bias = nn.Parameter(torch.ones(width)), nn.Parameter(torch.zeros(width))
        self.in_proj = nn.Linear(width, 2 * self.inner, bias=False)
        self.mixers = nn.ModuleList(Mixer(self.inner, N, max(8, width // 16)) for _ in range(directions))
        self.out_proj = nn.Linear(self.inner, width, bias=False)

    def halves(self, x):
        n = ssm.LayerNorm.apply(x, self.norm_weight, self.norm_bias, 1e-5)
        xz = self.in_proj(n)
        return xz[..., :self.inner], xz[..., self.inner:]

    def forward(self, x, lengths=None):
        u, z = self.halves(x)
        y = sum(m(u, z, lengths, k == 1) for k, m in enumerate(self.mixers))
        return x + self.out_proj(y)

    def prompt(self, x, lengths=None):
        u, z = self.halves(x)
        y, states = self.mixers[0].prompt(u, z, lengths)
        return x + self.out_proj(y), states

    def step(self, x, states):
        u, z = self.halves(x)
        return x + self.out_proj(self.mixers[0].step(u.contiguous(), z.contiguous(), states))


class Model(nn.Module):
    def __init__(self, vocab=16, width=64, depth=2, directions=1):
        super().__init__()
        self.embed = nn.Embedding(vocab, width)
        self.blocks = nn.ModuleList(Block(width, directions=directions) for _ in range(depth))
        self.head = nn.Linear(width, vocab)

    def forward(self, tokens, lengths=None):
        x = self.embed(tokens)
        for b in self.blocks:
            x = b(x, lengths)
        return self.head(x)

    @torch.no_grad()
    def prompt(self, tokens, lengths=None):
        """(logits of every token, states of every block)."""
        x, states = self.embed(tokens), []
        for b in self.blocks:
            x, s = b.prompt(x, lengths)
            states.append(s)
        return self.head(x), states

    @torch.no_grad()
    def step(self, token, states):
        """Logits after one more token of each sequence; states move on in place."""
        x = self.embed(token)
        for b, s in zip(self.blocks, states):
            x = b.step(x, s)
        return self.head(x)


def batch(B, L, vocab, gen):
    """Tokens, and at each place the token that stood `lag` places before (the first token says how many)."""
    t = torch.randint(0, vocab, (B, L), generator=gen, device="cuda")
    lag = torch.randint(1, 4, (B,), generator=gen, device="cuda")
    t[:, 0] = lag
    at = (torch.arange(L, device="cuda") - lag[:, None]).clamp(min=0)
    return t, t.gather(1, at)


def train(model, steps=150, B=32, L=64, vocab=16, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    opt = torch.optim.AdamW(model.parameters(), lr=3e-3)
    losses = []
    for _ in range(steps):
        t, want = batch(B, L, vocab, gen)
        loss = nn.functional.cross_entropy(model(t)[:, 4:].flatten(0, 1), want[:, 4:].flatten())
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.detach())
    return torch.stack(losses).tolist()


def serve_error(model, B=3, L=40, prompt=25, vocab=16, seed=1):
    """The largest difference between the logits of token-by-token decoding after a prompt and those of the whole
    sequence, relative to the largest logit."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    t, _ = batch(B, L, vocab, gen)
    with torch.no_grad():
        whole = model(t)
    got, states = model.prompt(t[:, :prompt].contiguous())
    got = [got] + [model.step(t[:, i], states)[:, None] for i in range(prompt, L)]
    return float((torch.cat(got, 1) - whole).abs().max() / whole.abs().max())


if __name__ == "__main__":
    torch.manual_seed(0)
    torch.backends.cuda.matmul.allow_tf32 = False
    m = Model().cuda()
    losses = train(m)
    print(f"loss {losses[0]:.3f} -> {losses[-1]:.3f}")
    print(f"decoding against the whole sequence: {serve_error(m):.1e} of the largest logit")
    enc = Model(directions=2).cuda()
    losses = train(enc, 50)
    print(f"both directions: loss {losses[0]:.3f} -> {losses[-1]:.3f}")
