"""The small model of examples/delta_block.py: convolution, norms with
rotation, delta rule and layer norm as one uses them.  It trains, its gradients
are those of plain torch operations in 64 bits, a ragged prompt followed by
single tokens gives the whole sequences' logits, and a step of training and a
token can be captured."""
import os
import sys

import pytest
import torch
from torch import nn

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bidirectional_masked_linear_gb300 import build, lion
    lion.load(build.build())
    import delta_block
    return delta_block


def test_runs(example):
    torch.manual_seed(0)
    losses = example.train(example.Model().cuda(), 5)
    assert all(map(lambda x: x == x and abs(x) < 100, losses))


def _plain_block(b, x):
    """The block in elementary operations, token by token."""
    H, d = b.heads, b.d
    n = (x - x.mean(-1, keepdim=True)) / torch.sqrt(x.var(-1, unbiased=False, keepdim=True) + 1e-5)
    p = (n * b.norm_weight + b.norm_bias) @ b.in_proj.weight.T
    u, g, beta = p[..., :3 * b.inner], -nn.functional.softplus(p[..., 3 * b.inner:-H] + b.rate), torch.sigmoid(p[..., -H:])
    K, L = b.taps.shape[1], x.shape[1]
    line = torch.cat((u.new_zeros(u.shape[0], K - 1, u.shape[2]), u), 1)
    u = sum(b.taps[:, k] * line[:, k:k + L] for k in range(K))
    q, k, v = (t.unflatten(-1, (H, d)) for t in (u * torch.sigmoid(u)).split(b.inner, -1))
    angle = torch.arange(L, device=x.device)[:, None] * b.freqs
    c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]

    def norm(t):
        t = t / torch.sqrt((t * t).sum(-1, keepdim=True) + 1e-6)
        a, e = t.chunk(2, -1)
        return torch.cat((a * c - e * s, a * s + e * c), -1)

    q, k = norm(q), norm(k)
    S, out = x.new_zeros(x.shape[0], H, d, d), []
    for t in range(L):
        S = torch.exp(g[:, t])[..., None, None] * S
        miss = v[:, t] - (S * k[:, t].unsqueeze(-1)).sum(2)
        S = S + k[:, t].unsqueeze(-1) * (beta[:, t].unsqueeze(-1) * miss).unsqueeze(2)
        out.append((S * q[:, t].unsqueeze(-1)).sum(2) * d ** -0.5)
    return x + torch.stack(out, 1).flatten(2) @ b.out_proj.weight.T


def test_gradients(example):
    """Every parameter's, against 64 bits.  float32 results of the operators are within 1e-5 of theirs, torch's sums and
    products within as much; eight of them follow one another from a loss to the embedding: 1e-4 of the largest."""
    torch.manual_seed(3)
    m = example.Model().cuda()
    t = torch.randint(0, 16, (2, 45), device="cuda")
    w = torch.randn(2, 45, 16, device="cuda")
    (m(t) * w).sum().backward()
    ref = example.Model().cuda().double()
    ref.load_state_dict(m.state_dict())
    x = ref.embed(t)
    for b in ref.blocks:
        x = _plain_block(b, x)
    (ref.head(x) * w).sum().backward()
    for (name, p), r in zip(m.named_parameters(), ref.parameters()):
        assert float((p.grad - r.grad).abs().max()) <= 1e-4 * float(r.grad.abs().max()), name


def test_prompt_and_steps_give_the_whole(example):
    torch.manual_seed(1)
    assert example.serve_error(example.Model().cuda()) <= 1e-4   # fp32 products in another order, two blocks


def test_ragged_batch_is_its_sequences(example):
    torch.manual_seed(2)
    m = example.Model().cuda()
    t, n = torch.randint(0, 16, (3, 70), device="cuda"), [70, 1, 33]
    with torch.no_grad():
        whole = m(t, torch.tensor(n, dtype=torch.int32, device="cuda"))
        for b, k in enumerate(n):
            alone = m(t[b:b + 1, :k].contiguous())
            assert float((whole[b:b + 1, :k] - alone).abs().max()) <= 1e-4 * float(alone.abs().max())


def test_a_captured_token(example):
    """A decoding step as a graph, replayed from token to token on states in place."""
    torch.manual_seed(4)
    m = example.Model().cuda()
    t = torch.randint(0, 16, (2, 12), device="cuda")
    with torch.no_grad():
        whole = m(t)
        _, states = m.prompt(t[:, :4].contiguous())
        token, pos = t[:, 4].clone(), torch.full((2, 1), 4, dtype=torch.int32, device="cuda")
        kept = [[x.clone() for x in s] for s in states]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            m.step(token, states, pos)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = m.step(token, states, pos)
        for s, k in zip(states, kept):
            for x, z in zip(s, k):
                x.copy_(z)
        for i in range(4, 12):
            token.copy_(t[:, i])
            pos.fill_(i)
            graph.replay()
            assert float((y - whole[:, i]).abs().max()) <= 1e-4 * float(whole.abs().max())
