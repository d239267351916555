"""The gated delta rule against its recurrence in 64 bits where many heads
share a walk's SMs and where long sequences are cut into segments, with decays
and step sizes so small that a state lasts a thousand tokens and more: every
segment's part is in all that follow it.

Bounds, set before the first run, on the 2-norm of the error, in which
roundings add as their squares do.  States (float32 from bfloat16 inputs): a
chunk takes out and writes in products of factors of two planes, three
roundings of at most 2^-18 of them, 3 x 2^-18 = 1.1e-5 at the very most where all
of them were at their bound; 1e-5, as the sequences of the other tests have.
Results and gradients in float32 the same.  bfloat16 results: four factors'
and their own rounding of 2^-9 at most, 2^-9 sqrt(5), and dq, dk, dg and dbeta,
whose terms come from both sides of a token, all four factors' at once,
2^-7."""
import pytest
import torch

from bidirectional_masked_linear_gb300 import delta, lion
from delta_recurrence import recurrence
from test_gpu_ssm import T

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bidirectional_masked_linear_gb300 import build
    lion.load(build.build())


def _inputs(B, L, Hk, Hv, dk, dv, dtype, seed):
    """Step sizes of about e^-4: keys of a head of 64 take thousands of tokens to erase what a state holds."""
    gen = torch.Generator().manual_seed(seed)
    mk = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    unit = lambda t: t / t.norm(dim=-1, keepdim=True)  # noqa: E731
    a = dict(q=unit(mk(B, L, Hk, dk)), k=unit(mk(B, L, Hk, dk)), v=mk(B, L, Hv, dv),
             g=-torch.log1p(torch.exp(-8 - mk(B, L, Hv))), beta=torch.sigmoid(mk(B, L, Hv) - 4))
    a = {x: y.to(T[dtype]).cuda() for x, y in a.items()}
    return a, mk(B, Hv, dk, dv).cuda(), mk(B, L, Hv, dv).to(T[dtype]).cuda()


def _near(name, got, want, limit):
    off, size = float((got.double() - want).norm()), float(want.norm())
    assert off <= limit * size, (name, off / size)


def _compare(a, h0, dout, how, dtype):
    r = recurrence(**a, scale=how["scale"], h0=h0, lengths=how["n"], reverse=how["reverse"], dout=dout)
    n = how.pop("n")
    if n is not None:
        for b, m in enumerate(n):
            for x in (*a.values(), dout):
                x[b, m:] = float("nan")
        how["lengths"] = torch.tensor(n, dtype=torch.int32, device="cuda")
    f = delta.delta_fwd(**a, h0=h0, **how, return_state=True, save=True)
    g = delta.delta_bwd(dout, **a, h0=h0, **how, saved=f.saved)
    for x, y in (("out", f.out), ("h", f.h), *((x, getattr(g, x)) for x in ("dq", "dk", "dv", "dg", "dbeta", "dh0"))):
        limit = 1e-5 if y.dtype == torch.float32 else 5 ** 0.5 * 2.0 ** -9 if x in ("out", "dv") else 2.0 ** -7
        _near(x, y, r[x], limit)
    # without what the forward kept
    plain = delta.delta_fwd(**a, h0=h0, **how, return_state=True)
    assert torch.equal(plain.out, f.out) and torch.equal(plain.h, f.h)
    again = delta.delta_bwd(dout, **a, h0=h0, **how)
    assert all(torch.equal(x, y) for x, y in zip(again, g))


# More CTAs of 32 columns than the 152 SMs, and at most 304 of 64: four pairs of warps a CTA in bfloat16.
@pytest.mark.parametrize("dtype", ("bf16", "fp32"))
@pytest.mark.parametrize("B,L,Hk,Hv,dk,dv,ragged,reverse", (
    (40, 100, 1, 2, 64, 64, True, False), (20, 257, 2, 8, 64, 64, False, True), (20, 130, 1, 2, 128, 128, True, True),
    (26, 97, 1, 3, 72, 40, True, False), (20, 161, 2, 2, 40, 104, False, False), (50, 64, 2, 6, 128, 64, True, False)))
def test_walks_of_many_heads(B, L, Hk, Hv, dk, dv, ragged, reverse, dtype):
    a, h0, dout = _inputs(B, L, Hk, Hv, dk, dv, dtype, dk + dv + L)
    n = [(41 * b + 1) % (L + 1) for b in range(B)] if ragged else None
    _compare(a, h0, dout, dict(scale=dk ** -0.5, n=n, reverse=reverse), dtype)


# Segments of 19, 17, 18, 17 and 16 chunks, of which the odd ones end inside a block of 64 tokens; two pairs of warps a
# CTA in the first and the last row, four in the others.
@pytest.mark.parametrize("B,L,Hk,Hv,dk,dv,n,reverse", (
    (1, 2400, 1, 1, 64, 64, None, False), (2, 2605, 4, 8, 64, 64, (2605, 1111), True),
    (2, 5000, 2, 4, 128, 128, (4999, 3000), False), (3, 2605, 2, 4, 24, 72, (2605, 544, 0), True),
    (2, 4096, 1, 1, 128, 40, None, False)))
def test_many_segments(B, L, Hk, Hv, dk, dv, n, reverse):
    a, h0, dout = _inputs(B, L, Hk, Hv, dk, dv, "bf16", dk + dv + L)
    _compare(a, h0, dout, dict(scale=dk ** -0.5, n=n, reverse=reverse), "bf16")
