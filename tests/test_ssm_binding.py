"""The state space block's Python binding without a GPU: what its autograd
functions and argument checks do before anything reaches the library."""
import pytest
import torch

from bidirectional_masked_linear_gb300 import ssm


def _cube(monkeypatch, name):
    """The autograd function `name` on y = x^3 in place of its kernels, applied to x."""
    if name == "LayerNorm":
        monkeypatch.setattr(ssm, "layernorm_fwd", lambda x, *a, **k: (x ** 3, x[..., 0], x[..., 0]))
        monkeypatch.setattr(ssm, "layernorm_bwd", lambda dy, x, *a, **k: (3 * x * x * dy, None, None))
        return lambda x: ssm.LayerNorm.apply(x, x[0].detach(), None)
    if name == "CausalConv":
        monkeypatch.setattr(ssm, "conv_fwd", lambda x, *a, **k: x ** 3)
        monkeypatch.setattr(ssm, "conv_bwd", lambda dy, x, *a, **k: ssm.ConvGrads(3 * x * x * dy, None, None, None))
        return lambda x: ssm.CausalConv.apply(x, x[0].detach(), None)
    monkeypatch.setattr(ssm, "scan_fwd", lambda u, *a, **k: ssm.ScanOut(u ** 3, None, u.detach()))
    monkeypatch.setattr(ssm, "scan_bwd",
                        lambda do, u, *a, **k: ssm.ScanGrads(3 * u * u * do, *[None] * 8))
    return lambda x: ssm.SelectiveScan.apply(x, *[x.detach()] * 4)


@pytest.mark.parametrize("name", ("LayerNorm", "CausalConv", "SelectiveScan"))
def test_second_derivatives_are_refused(monkeypatch, name):
    """The gradients' kernels have none of their own: a second derivative must not come out without their terms."""
    f = _cube(monkeypatch, name)
    x = torch.tensor([[1.0, 2.0]], requires_grad=True)
    g, = torch.autograd.grad(f(x).sum(), x)
    assert torch.equal(g, 3 * x.detach() ** 2)
    g, = torch.autograd.grad(f(x).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="differentiated again"):
        (g.sum() + (x ** 2).sum()).backward()
    # one that does not need them is not refused
    (g.detach().sum() + (x ** 2).sum()).backward()
    assert torch.equal(x.grad, 2 * x.detach())
    # nor is one with nothing to differentiate
    dy = torch.ones_like(x)
    assert not torch.autograd.grad(f(x), x, dy)[0].requires_grad
