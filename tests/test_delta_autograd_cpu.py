"""The delta rule's autograd functions without a GPU: the calls that they make,
stood in for by formulas."""
import pytest
import torch

from bidirectional_masked_linear_gb300 import delta


@pytest.fixture
def calls(monkeypatch):
    made = []
    monkeypatch.setattr(delta, "qknorm_fwd", lambda q, k, *a, **kw: (2 * q, 3 * k))
    monkeypatch.setattr(delta, "qknorm_bwd", lambda dq, dk, q, k, *a, **kw: delta.QKNormGrads(2 * dq, 3 * dk, None, None))
    monkeypatch.setattr(delta, "delta_fwd",
                        lambda q, *a, **kw: made.append(kw) or delta.DeltaOut(2 * q, None, q.detach() if kw.get("save") else None))
    monkeypatch.setattr(delta, "delta_bwd", lambda do, *a, **kw: delta.DeltaGrads(2 * do, *[torch.zeros_like(do)] * 4, None))
    return made


def test_a_gradient_that_there_is_none_of_raises(calls):
    """Learned frequencies or a learned scale would otherwise stay as they are in silence."""
    q, f = torch.ones(3, requires_grad=True), torch.ones(4, requires_grad=True)
    norm = lambda f: delta.QKNorm.apply(q, q, None, None, "l2", 1e-6, f)  # noqa: E731
    with pytest.raises(RuntimeError, match="freqs has no gradient"):
        sum(y.sum() for y in norm(f)).backward()
    sum(y.sum() for y in norm(f.detach())).backward()
    assert torch.equal(q.grad, torch.full((3,), 5.0)) and f.grad is None
    with torch.no_grad():
        assert torch.equal(norm(f)[0], 2 * q)
    scale, rest = torch.tensor(2.0, requires_grad=True), [torch.ones(3)] * 4
    with pytest.raises(RuntimeError, match="scale has no gradient"):
        delta.GatedDelta.apply(q, *rest, scale).sum().backward()
    q.grad = None
    delta.GatedDelta.apply(q, *rest, scale.detach()).sum().backward()
    assert torch.equal(q.grad, torch.full((3,), 2.0))


def test_nothing_is_kept_where_no_gradient_is_wanted(calls):
    """What the forward keeps is twice its inputs and more: 408 MB beside 201 at 16 x 4096 x 8 x 64 in bfloat16."""
    x = [torch.ones(3)] * 5
    delta.GatedDelta.apply(*x)
    with torch.no_grad():
        delta.GatedDelta.apply(*(2 * torch.ones(3, requires_grad=True) for _ in x))
    delta.GatedDelta.apply(*x[:4], torch.ones(3, requires_grad=True)).sum().backward()
    assert [c["save"] for c in calls] == [False, False, True]
