"""Results that would be written over what others still read are refused, and
nothing is written: crossed outputs of the norms, the one-token step's output
in place of its query, and the gradients in place of what they are made of."""
import pytest
import torch

from bidirectional_masked_linear_gb300 import delta, lion

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bidirectional_masked_linear_gb300 import build
    lion.load(build.build())


def _refused(call, *tensors):
    before = [t.clone() for t in tensors]
    with pytest.raises(lion.LionError) as e:
        call()
    assert e.value.status == lion.ERR_INVALID_ARG
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(before, tensors))


def _inputs(L):
    gen = torch.Generator(device="cuda").manual_seed(1)
    mk = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    one = lambda *s: mk(2, L, *s) if L else mk(2, *s)  # noqa: E731
    q, k = (torch.nn.functional.normalize(one(3, 64), dim=-1) for _ in range(2))
    return dict(q=q, k=k, v=one(3, 64), g=-one(3).abs(), beta=torch.sigmoid(one(3)))


def test_norms():
    q, k = torch.randn(2, 5, 32, 64, device="cuda"), torch.randn(2, 5, 32, 64, device="cuda")
    out = torch.zeros_like(q)
    for how in (dict(q_out=k), dict(k_out=q), dict(q_out=k, k_out=q), dict(q_out=q), dict(k_out=k),
                dict(q_out=out, k_out=out)):
        _refused(lambda: delta.qknorm_fwd(q, k, **how), q, k, out)
    assert delta.qknorm_fwd(q, q, q_out=out)[0] is out   # inputs may be the same


def _with_results(monkeypatch, call, results):
    """The call with given tensors for the results that it would allocate, in their order."""
    left = list(results)
    monkeypatch.setattr(delta, "_like", lambda stream, x: left.pop(0))
    try:
        call()
    finally:
        monkeypatch.undo()
        assert not left


def test_norm_gradients(monkeypatch):
    q, k, dqo, dko, x, y = (torch.randn(2, 5, 32, 64, device="cuda") for _ in range(6))
    for results in ((k, x), (x, q), (dko, x), (x, dqo), (q, x), (dqo, x), (x, k), (x, dko), (x, x)):
        _refused(lambda: _with_results(monkeypatch, lambda: delta.qknorm_bwd(dqo, dko, q, k), results), q, k, dqo, dko, x)
    _with_results(monkeypatch, lambda: delta.qknorm_bwd(dqo, dko, q, k), (x, y))
    assert torch.equal(x, delta.qknorm_bwd(dqo, dko, q, k).dq)


def test_delta_gradients(monkeypatch):
    a = _inputs(70)
    dout = torch.randn_like(a["v"])
    saved = delta.delta_fwd(**a, save=True).saved
    x = [torch.zeros_like(a[n]) for n in ("q", "k", "v", "g", "beta")]
    for i, others in ((0, (dout, a["q"], a["k"], x[1], x[2])), (1, (dout, a["q"], a["k"], x[2])),
                      (2, (dout, a["q"], a["k"])), (3, (a["g"], a["beta"], x[4])), (4, (a["g"], a["beta"]))):
        for other in others:
            results = [other if j == i else y for j, y in enumerate(x)]
            for s in (saved, None):
                _refused(lambda: _with_results(monkeypatch, lambda: delta.delta_bwd(dout, **a, saved=s), results),
                         dout, *a.values(), *x)
    want = delta.delta_bwd(dout, **a, saved=saved)
    _with_results(monkeypatch, lambda: delta.delta_bwd(dout, **a, saved=saved), x)
    assert all(torch.equal(s, t) for s, t in zip(x, want))


def test_step():
    a = _inputs(0)
    h = torch.randn(2, 3, 64, 64, device="cuda")
    for n in ("q", "k"):
        _refused(lambda: delta.delta_step(h, **a, out=a[n]), h, *a.values())
    # a value's own columns are read by the threads that write them
    other = h.clone()
    want = delta.delta_step(other, **a)
    assert torch.equal(delta.delta_step(h, **a, out=a["v"]), want) and torch.equal(h, other)
