"""Decays above 1, whose product over 32 adjacent tokens is finite in float32
but over a block of the gradients or a segment of a cut walk is not: states and
gradients that are finite all the same, small before they grow, are right.

Bounds, on the 2-norm over the tokens between two growths, whose values are of
one size.  An exponent of up to 80 is held to 2^-18, 4e-6 of its power, and up
to ten such powers stand in a product beside the other roundings: 1e-4 in
float32.  bfloat16 results: 2^-9 sqrt(5), dq and dk 2^-7, as in the tests of
walks.  dg and dbeta of a token are single sums, which may cancel.  What the
roundings of their factors (R, dR, a block's first state and last gradient,
each at most 2^-9 and independent of the others) make of such a sum is to first
order d = sum x_i delta_i, and |d| > 4 x 2^-9 |x| has a probability below
2 e^-8 (Hoeffding): that, with the |x| of `_sizes`, and a rounding of the
result."""
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


def _sizes(a, reverse, walk):
    """For dg and dbeta of each token the length of all x_i, where a factor's rounding of 1 + delta_i makes x_i delta_i
    of the sum.  In a block of 64 tokens the state before token t consists of the block's first state and of what
    tokens before t wrote, R; its gradient of the block's last one and of what tokens from t on add, dO and dR."""
    states, R, dR, dstates = (x if isinstance(x, list) else x[:, 0, 0] for x in walk)
    k, g, beta = ((a[x].flip(1) if reverse else a[x])[0, :, 0].double() for x in "k g beta".split())
    dg, db = torch.zeros_like(g), torch.zeros_like(g)
    for c in range(0, len(g), 64):
        e = min(len(g), c + 64)
        G = g[c:e].cumsum(0)
        first, last = states[c][0, 0], dstates[e][0, 0]
        for t in range(c, e):
            old, new = g[t].exp() * states[t][0, 0], dstates[t][0, 0] / g[t].exp()
            to, on = (G[t - c] - G[:t - c]).exp()[:, None], (G[t - c:] - G[t - c]).exp()[:, None]
            end = (G[-1] - G[t - c]).exp()
            for x in (to * beta[c:t, None] * R[c:t] * (k[c:t] @ new), on * dR[t:e] * (k[t:e] @ old),
                      G[t - c].exp() * first * new, end * last * old):
                dg[t] += (x * x).sum()
            for x in (R[t] * dR[t] / beta[t], end * last * k[t][:, None] * R[t],
                      (on * dR[t:e] * (k[t:e] @ k[t])[:, None] * R[t])[1:]):
                db[t] += (x * x).sum()
    return {"dg": dg.sqrt(), "dbeta": db.sqrt()}


def _grown(L, dk, dv, dtype, up, down, reverse, by=55.0):
    """Growths of e^by at `up`, values of 1e-16 beside them, and decays as large at `down`.  Between growths of less than
    e^55 values are of many sizes: the tokens before the first and after the last of those are compared."""
    gen = torch.Generator().manual_seed(dk + L)
    mk = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    unit = lambda t: t / t.norm(dim=-1, keepdim=True)  # noqa: E731
    a = dict(q=unit(mk(1, L, 1, dk)), k=unit(mk(1, L, 1, dk)), v=1e-16 * mk(1, L, 1, dv),
             g=-0.001 * torch.rand(1, L, 1, generator=gen), beta=torch.sigmoid(mk(1, L, 1)))
    a["g"][:, list(up)], a["g"][:, list(down)] = by, -by
    dout = 1e-16 * mk(1, L, 1, dv)
    a = {x: (y.flip(1) if reverse else y).to(T[dtype]).cuda() for x, y in a.items()}
    dout, h0 = dout.to(T[dtype]).cuda(), 1e-16 * mk(1, 1, dk, dv).cuda()
    how = dict(scale=dk ** -0.5, reverse=reverse, h0=h0)
    r = recurrence(**a, **how, dout=dout)
    f = delta.delta_fwd(**a, **how, return_state=True, save=True)
    g = delta.delta_bwd(dout, **a, **how, saved=f.saved)
    cuts = [0, *up, *down, L]
    groups = list(zip(cuts, cuts[1:])) if by == 55.0 else [(0, up[0]), (up[-1], L)]
    sizes = _sizes(a, reverse, r["walk"])
    for x in ("h", "dh0"):
        off, size = float(((f.h if x == "h" else g.dh0).double() - r[x]).norm()), float(r[x].norm())
        assert 0 < size < 1e37 and off <= 1e-4 * size, (x, off, size)
    for x, y in (("out", f.out), *((x, getattr(g, x)) for x in ("dq", "dk", "dv", "dg", "dbeta"))):
        y, want = ((t.flip(1) if reverse else t)[0].double() for t in (y, r[x]))
        for i, j in groups:
            off, size = float((y[i:j] - want[i:j]).norm()), float(want[i:j].norm())
            if dtype == "fp32":
                limit = 1e-4 * size
            elif x in sizes:
                limit = 2.0 ** -9 * (4 * float(sizes[x][i:j].norm()) + size)
            else:
                limit = (5 ** 0.5 if x in ("out", "dv") else 4) * 2.0 ** -9 * size
            assert 0 < size < 1e37 and off <= limit, (x, i, off, limit, size)


@pytest.mark.parametrize("dtype", ("bf16", "fp32"))
@pytest.mark.parametrize("reverse", (False, True))
@pytest.mark.parametrize("dk,dv,up", ((64, 64, (10, 50)), (24, 40, (3, 35)), (128, 128, (70, 127))))
def test_growth_inside_a_block(dk, dv, up, reverse, dtype):
    _grown(150, dk, dv, dtype, up, (), reverse)


# Three segments of 18 chunks, 576 tokens: all growths are in the second one.
@pytest.mark.parametrize("reverse", (False, True))
@pytest.mark.parametrize("down", ((), (900, 1000)))
@pytest.mark.parametrize("dk,dv", ((64, 64), (128, 72)))
def test_growth_inside_a_segment(dk, dv, down, reverse):
    _grown(1700, dk, dv, "bf16", (700, 800), down, reverse)


@pytest.mark.parametrize("reverse", (False, True))
@pytest.mark.parametrize("L,at,dtype", ((150, 34, "fp32"), (150, 34, "bf16"), (150, 70, "bf16"), (1700, 674, "bf16")))
def test_growth_up_to_the_bound(L, at, dtype, reverse):
    """Ten decays of e^8.5 among 32 tokens: 8e36 of the 3e38 that their product may be."""
    _grown(L, 64, 64, dtype, range(at, at + 20, 2), (), reverse, by=8.5)
