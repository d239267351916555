"""The delta rule's operators on the GPU against 64-bit references written
token by token from the formulas (delta_reference.py, which derives the bounds
of the delta rule).

Bounds of the norms, set before the first run, with e = 2^-24: the sum of a
head's squares is eight terms a lane and five exchanges, root and quotient
exact to a rounding, so 1 / length is off by 16 e; a product more makes 2 e,
the angle, its cosine and sine and the turn 8 e of the pair's two values.
y: 32 e of the pair; dx: 48 e of its two terms' absolute values; dw: 64 e and
one e for each row of the sum.  The step: a sum of dk products, 2 dk + 32
roundings of the formula of absolute values."""
import math

import numpy as np
import pytest
import torch

import delta_reference as ref
from bidirectional_masked_linear_gb300 import delta, lion
from test_gpu_ssm import E, T, _check, _f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bidirectional_masked_linear_gb300 import build
    lion.load(build.build())


def _equal(a, b):
    return all(x is y is None or torch.equal(x, y) for x, y in zip(a, b))


# ------------------------------------------------------- norms of q and k

QK = [  # B, L, Hq, Hk, d, rot, norm, weight, interleaved, far
    (1, 1, 1, 1, 8, 0, "l2", False, False, False), (2, 3, 3, 1, 16, 8, "rms", True, False, True),
    (1, 5, 2, 5, 24, 24, "l2", True, True, False), (3, 7, 12, 12, 64, 64, "rms", True, False, True),
    (2, 200, 5, 3, 72, 40, "l2", False, False, False), (1, 9, 4, 2, 128, 128, "rms", True, True, True),
    (2, 4, 1, 3, 136, 8, "rms", False, False, False), (1, 6, 2, 2, 256, 256, "l2", True, False, True),
    (4, 2500, 2, 1, 40, 16, "rms", True, True, False),
]


def _pairs(d, rot, interleaved):
    """Each value's partner in its turn (itself where it does not turn)."""
    at = np.arange(d)
    m = rot // 2
    if interleaved:
        at[:rot] ^= 1
    else:
        at[:m], at[m:rot] = np.arange(m, rot), np.arange(m)
    return at


@pytest.mark.parametrize("dtype", ("bf16", "fp32"))
@pytest.mark.parametrize("B,L,Hq,Hk,d,rot,norm,weight,interleaved,far", QK)
def test_qknorm(B, L, Hq, Hk, d, rot, norm, weight, interleaved, far, dtype):
    gen = torch.Generator().manual_seed(d + L)
    mk = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    x = [(2 * mk(B, L, h, d)).to(T[dtype]) for h in (Hq, Hk)]
    dy = [mk(B, L, h, d).to(T[dtype]) for h in (Hq, Hk)]
    w = [1 + 0.3 * mk(d) if weight else None for _ in range(2)]
    freqs = 10000.0 ** (-torch.arange(rot // 2) / max(1, rot // 2)) if rot else None
    pos = torch.arange(L).expand(B, L)
    if far:
        pos = pos + (torch.rand(B, 1, generator=gen) * (2 ** 31 - 1 - L)).long()
    c = lambda t: None if t is None else t.cuda()  # noqa: E731
    kw = dict(q_weight=c(w[0]), k_weight=c(w[1]), norm=norm, eps=1e-6, freqs=c(freqs), interleaved=interleaved,
              positions=pos.int().cuda() if rot and far else None)
    y = delta.qknorm_fwd(x[0].cuda(), x[1].cuda(), **kw)
    g = delta.qknorm_bwd(dy[0].cuda(), dy[1].cuda(), x[0].cuda(), x[1].cuda(), **kw)
    at, n = _pairs(d, rot, interleaved), d if norm == "rms" else 1
    for i in range(2):
        X, W, DY = _f64(x[i]), _f64(w[i]), _f64(dy[i])
        r = ref.qknorm(X, W, norm, 1e-6, _f64(freqs), pos.numpy(), interleaved, DY)
        W = np.ones(d) if W is None else W
        size = np.abs(X * r["r"] * W)
        _check("y", y[i], r["y"], 32 * E * (size + size[..., at]))
        dz = np.abs(DY) + np.abs(DY[..., at])
        gs = dz * np.abs(W)
        along = (gs * np.abs(X)).sum(-1, keepdims=True) / n
        _check("dx", g[i], r["dx"], 48 * E * (r["r"] * gs + np.abs(X) * r["r"] ** 3 * along))
        if weight:
            _check("dw", g[2 + i], r["dw"], (64 + X.size // d) * E * (dz * np.abs(X) * r["r"]).sum((0, 1, 2)))
        else:
            assert g[2 + i] is None
    assert _equal(y, delta.qknorm_fwd(x[0].cuda(), x[1].cuda(), **kw))
    assert _equal(g, delta.qknorm_bwd(dy[0].cuda(), dy[1].cuda(), x[0].cuda(), x[1].cuda(), **kw))


@pytest.mark.parametrize("dtype", ("bf16", "fp32"))
@pytest.mark.parametrize("at", (0, 8, 2, 3))
def test_qknorm_of_slices(at, dtype):
    """Slices of a projection, also off the vectors' alignment, equal their copies bit for bit."""
    B, L, Hq, Hk, d = 3, 11, 4, 2, 64
    wide = torch.randn(B, L, at + (Hq + Hk) * d + 5, device="cuda").to(T[dtype])
    q, k = (wide[..., at + a:at + b].unflatten(2, (-1, d)) for a, b in ((0, Hq * d), (Hq * d, (Hq + Hk) * d)))
    w, freqs = torch.randn(d, device="cuda"), torch.rand(16, device="cuda")
    kw = dict(q_weight=w, freqs=freqs, norm="rms")
    dq, dk = torch.randn(B, L, Hq, d, device="cuda").to(T[dtype]), torch.randn(B, L, Hk, d, device="cuda").to(T[dtype])
    assert _equal(delta.qknorm_fwd(q, k, **kw), delta.qknorm_fwd(q.contiguous(), k.contiguous(), **kw))
    a, b = delta.qknorm_bwd(dq, dk, q, k, **kw), delta.qknorm_bwd(dq, dk, q.contiguous(), k.contiguous(), **kw)
    assert _equal(a, b) and a.dk_weight is None


def test_qknorm_edges():
    """A head of zeros stays one; a position and its frequency turn whole turns away; outputs that are given."""
    q = torch.zeros(1, 2, 1, 16, device="cuda")
    q[0, 1] = 3.0
    y, _ = delta.qknorm_fwd(q, q)
    assert bool((y[0, 0] == 0).all()) and float((y[0, 1] - 0.25).abs().max()) <= 32 * E
    # frequencies of powers of two: position 2^30 f turns as one of f does 2^30 times, in exact arithmetic mod 1
    f = torch.tensor([0.5, 0.125, 2.0 ** -9, 1.0], device="cuda")
    pos = torch.tensor([[2 ** 30 + 7, 2 ** 31 - 1]], dtype=torch.int32, device="cuda")
    q = torch.zeros(1, 2, 1, 8, device="cuda")
    q[..., :4] = 0.5
    y, _ = delta.qknorm_fwd(q, q, freqs=f, positions=pos)
    a = _f64(pos)[0][:, None] * _f64(f)
    want = 0.5 * np.concatenate([np.cos(a), np.sin(a)], 1)
    _check("turn", y[0, :, 0], want, 32 * E)
    out = torch.empty_like(q)
    got = delta.qknorm_fwd(q, q, freqs=f, positions=pos, q_out=out)
    assert got[0] is out and torch.equal(out, y)


def test_qknorm_refusals():
    q = torch.zeros(1, 2, 2, 16, device="cuda")
    for kw, status in ((dict(q=q[..., :12].contiguous(), k=q[..., :12].contiguous()), lion.ERR_UNSUPPORTED),
                       (dict(freqs=torch.zeros(6, device="cuda")), lion.ERR_UNSUPPORTED),
                       (dict(freqs=torch.zeros(12, device="cuda")), lion.ERR_INVALID_ARG),
                       (dict(eps=-1.0), lion.ERR_INVALID_ARG), (dict(freqs=torch.zeros(4)), lion.ERR_INVALID_ARG)):
        with pytest.raises(lion.LionError) as e:
            delta.qknorm_fwd(**{**dict(q=q, k=q), **kw})
        assert e.value.status == status, kw


# ------------------------------------------------------------ the delta rule

def _inputs(B, L, Hk, Hv, dk, dv, dtype, seed, decay=3.0):
    gen = torch.Generator().manual_seed(seed)
    mk = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    unit = lambda t: t / t.norm(dim=-1, keepdim=True)  # noqa: E731
    a = dict(q=unit(mk(B, L, Hk, dk)), k=unit(mk(B, L, Hk, dk)), v=mk(B, L, Hv, dv),
             g=-torch.log1p(torch.exp(-decay - mk(B, L, Hv))), beta=torch.sigmoid(mk(B, L, Hv)))
    a = {x: y.to(T[dtype]) for x, y in a.items()}
    return a, mk(B, Hv, dk, dv), mk(B, L, Hv, dv).to(T[dtype])


DELTA = [  # B, L, Hk, Hv, dk, dv, lengths, state, reverse, decay
    (1, 1, 1, 1, 8, 8, None, False, False, 3.0), (2, 2, 1, 2, 64, 64, None, True, True, 3.0),
    (2, 31, 2, 2, 16, 24, None, True, False, 0.0), (1, 32, 1, 1, 64, 64, None, True, False, 3.0),
    (3, 33, 1, 3, 40, 72, (33, 0, 1), True, True, 3.0), (2, 64, 1, 1, 128, 64, None, False, False, 6.0),
    (3, 65, 2, 4, 64, 128, (65, 64, 32), True, False, -3.0), (2, 96, 1, 1, 72, 8, (96, 95), True, True, 3.0),
    (2, 97, 1, 2, 128, 128, None, True, False, 3.0), (2, 197, 3, 3, 64, 64, (197, 100), True, False, 6.0),
    (1, 200, 1, 1, 8, 128, None, True, True, -6.0),
]


@pytest.mark.parametrize("dtype", ("bf16", "fp32"))
@pytest.mark.parametrize("B,L,Hk,Hv,dk,dv,lens,state,reverse,decay", DELTA)
def test_delta(B, L, Hk, Hv, dk, dv, lens, state, reverse, decay, dtype):
    a, h0, dout = _inputs(B, L, Hk, Hv, dk, dv, dtype, L * 7 + dk, decay)
    A = {x: _f64(y) for x, y in a.items()}
    DO = _f64(dout)
    if lens:
        for b in range(B):   # what a padded place holds does not matter
            for x in (*a.values(), dout):
                x[b, lens[b]:] = float("nan")
    scale = 0.3
    r = ref.delta(**A, scale=scale, h0=_f64(h0) if state else None, lengths=lens, reverse=reverse, dout=DO,
                  bf16=dtype == "bf16")
    dev = {x: y.cuda() for x, y in a.items()}
    how = dict(scale=scale, h0=h0.cuda() if state else None, reverse=reverse,
               lengths=torch.tensor(lens, dtype=torch.int32, device="cuda") if lens else None)
    f = delta.delta_fwd(**dev, **how, return_state=True, save=True)
    g = delta.delta_bwd(dout.cuda(), **dev, **how, saved=f.saved)
    assert (g.dh0 is not None) == state
    for x, y in (("out", f.out), ("h", f.h), *((x, getattr(g, x)) for x in ("dq", "dk", "dv", "dg", "dbeta", "dh0"))):
        if y is not None:
            _check(x, y, r[x], r["~" + x])
            if x in ("out", "dv") or y.dtype == torch.float32:
                _exact_enough(x, y, r[x])
    # without what the forward kept, into workspaces of the caller's, and again
    plain = delta.delta_fwd(**dev, **how, return_state=True)
    assert plain.saved is None and _equal(plain[:2], f[:2])
    code = lion.DTYPE_BF16 if dtype == "bf16" else lion.DTYPE_FP32
    ws = torch.empty(delta.delta_bwd_workspace_bytes(B, L, Hk, Hv, dk, dv, code, False), dtype=torch.uint8, device="cuda")
    ws.fill_(255)
    assert _equal(delta.delta_bwd(dout.cuda(), **dev, **how, workspace=ws), g)
    ws = torch.full((delta.delta_workspace_bytes(B, L, Hk, Hv, dk, dv, code),), 255, dtype=torch.uint8, device="cuda")
    assert _equal(delta.delta_fwd(**dev, **how, workspace=ws)[:1], f[:1])


def _exact_enough(name, got, want):
    """What the bounds of single values, in which all errors add up, leave open.  The 2-norm of the error, where
    roundings add as their squares do: bfloat16 results are five roundings of at most 2^-9 off (four factors' and their
    own), 2^-9 sqrt(5) of the norm of their terms, float32 results, a bfloat16 call's states among them, 1e-5.  The
    terms of dq, dk, dg and dbeta come from both sides of a token and may cancel where there are two or three of them;
    of many tokens' sums they are as large as the result."""
    off = np.linalg.norm(_f64(got) - want)
    limit = 1e-5 if got.dtype == torch.float32 else 5 ** 0.5 * 2.0 ** -9
    assert off <= limit * np.linalg.norm(want), (name, off / np.linalg.norm(want))


@pytest.mark.parametrize("dtype", ("bf16", "fp32"))
@pytest.mark.parametrize("L,dk,dv", ((513, 64, 64), (300, 128, 128)))
def test_delta_over_many_chunks(L, dk, dv, dtype):
    a, h0, dout = _inputs(2, L, 1, 2, dk, dv, dtype, 11)
    r = ref.delta(**{x: _f64(y) for x, y in a.items()}, scale=dk ** -0.5, h0=_f64(h0), dout=_f64(dout))
    dev = {x: y.cuda() for x, y in a.items()}
    f = delta.delta_fwd(**dev, h0=h0.cuda(), return_state=True, save=True)
    g = delta.delta_bwd(dout.cuda(), **dev, h0=h0.cuda(), saved=f.saved)
    for x, y in (("out", f.out), ("h", f.h), ("dq", g.dq), ("dk", g.dk), ("dv", g.dv), ("dg", g.dg),
                 ("dbeta", g.dbeta), ("dh0", g.dh0)):
        _exact_enough(x, y, r[x])


@pytest.mark.parametrize("dtype", ("bf16", "fp32"))
def test_delta_gradients_under_strong_decay(dtype):
    """Decays of e^-7 and less: a decay's gradient is a single small pair beside products that cancel."""
    a, _, dout = _inputs(1, 100, 1, 1, 64, 64, dtype, 2, decay=-8.0)
    r = ref.delta(**{x: _f64(y) for x, y in a.items()}, scale=0.125, dout=_f64(dout))
    dev = {x: y.cuda() for x, y in a.items()}
    g = delta.delta_bwd(dout.cuda(), **dev, saved=delta.delta_fwd(**dev, save=True).saved)
    off = np.linalg.norm(_f64(g.dg) - r["dg"]) / np.linalg.norm(r["dg"])
    # bfloat16: four roundings of 2^-9 at most; float32: sums of 64 rows and columns, 2^-24 each of terms e^-7 and less
    assert off <= (2.0 ** -7 if dtype == "bf16" else 1e-5), off


@pytest.mark.parametrize("dtype", ("bf16", "fp32"))
@pytest.mark.parametrize("at", (0, 8, 2, 3))
def test_delta_of_slices(at, dtype):
    """Slices of projections, also off the vectors' alignment, equal their copies bit for bit."""
    B, L, Hk, Hv, dk, dv = 2, 70, 2, 4, 24, 40
    a, h0, dout = _inputs(B, L, Hk, Hv, dk, dv, dtype, 3)
    flat = [a[x].flatten(2) if a[x].dim() == 4 else a[x] for x in ("q", "k", "v", "g", "beta")]
    wide = torch.cat([torch.zeros(B, L, at).to(T[dtype]), *flat, torch.zeros(B, L, 3).to(T[dtype])], 2).cuda()
    cut, first = {}, at
    for x, y in zip(("q", "k", "v", "g", "beta"), flat):
        t = wide[..., first:first + y.shape[2]]
        first += y.shape[2]
        cut[x] = t.unflatten(2, a[x].shape[2:]) if a[x].dim() == 4 else t
    dev = {x: y.cuda() for x, y in a.items()}
    f, s = (delta.delta_fwd(**d, h0=h0.cuda(), return_state=True, save=True) for d in (dev, cut))
    assert _equal(f[:2], s[:2])
    off = torch.empty(dout.numel() + 1, dtype=T[dtype], device="cuda")[1:].view(dout.shape)
    assert _equal(delta.delta_bwd(dout.cuda(), **dev, saved=f.saved), delta.delta_bwd(off.copy_(dout), **cut, saved=s.saved))
    assert torch.equal(delta.delta_fwd(**cut, h0=h0.cuda(), out=off).out, f.out)


def test_ragged_reversed_and_alone():
    """A padded batch gives each sequence's own bits, and walking back those of the flipped sequence."""
    n = (130, 1, 0, 64)
    a, h0, dout = _inputs(4, 130, 1, 2, 64, 64, "bf16", 5)
    dev, h0, dout = {x: y.cuda() for x, y in a.items()}, h0.cuda(), dout.cuda()
    lens = torch.tensor(n, dtype=torch.int32, device="cuda")
    for rev in (False, True):
        f = delta.delta_fwd(**dev, h0=h0, lengths=lens, reverse=rev, return_state=True, save=True)
        g = delta.delta_bwd(dout, **dev, h0=h0, lengths=lens, reverse=rev, saved=f.saved)
        for b, m in enumerate(n):
            for x in (f.out, g.dq, g.dk, g.dv, g.dg, g.dbeta):
                assert bool((x[b, m:] == 0).all())
            if m == 0:
                assert torch.equal(f.h[b], h0[b]) and bool((g.dh0[b] == 0).all())
                continue
            flip = (lambda t: t.flip(1)) if rev else (lambda t: t)
            one = {x: flip(y[b:b + 1, :m]).contiguous() for x, y in dev.items()}
            s = delta.delta_fwd(**one, h0=h0[b:b + 1], return_state=True, save=True)
            assert torch.equal(flip(s.out), f.out[b:b + 1, :m]) and torch.equal(s.h[0], f.h[b])
            e = delta.delta_bwd(flip(dout[b:b + 1, :m]).contiguous(), **one, h0=h0[b:b + 1], saved=s.saved)
            for x in ("dq", "dk", "dv", "dg", "dbeta"):
                assert torch.equal(flip(getattr(e, x)), getattr(g, x)[b:b + 1, :m]), x
            assert torch.equal(e.dh0[0], g.dh0[b])
    # lengths out of range are clamped into it
    wild = torch.tensor([999, 1, -3, 64], dtype=torch.int32, device="cuda")
    assert _equal(delta.delta_fwd(**dev, h0=h0, lengths=wild, return_state=True)[:2],
                  delta.delta_fwd(**dev, h0=h0, lengths=lens, return_state=True)[:2])


@pytest.mark.parametrize("dtype", ("bf16", "fp32"))
@pytest.mark.parametrize("at", (1, 31, 32, 33, 64, 70))
def test_a_decay_of_zero_starts_anew(at, dtype):
    """g = -inf forgets all: what follows is a sequence of its own, to the roundings that the chunks' cuts decide."""
    a, _, dout = _inputs(1, 100, 1, 1, 64, 32, dtype, 9)
    a["g"][:, at] = -float("inf")
    dev, dout = {x: y.cuda() for x, y in a.items()}, dout.cuda()
    f = delta.delta_fwd(**dev, return_state=True, save=True)
    g = delta.delta_bwd(dout, **dev, saved=f.saved)
    r = ref.delta(**{x: np.where(np.isinf(y), -2000.0, y) for x, y in ((x, _f64(y)) for x, y in a.items())},
                  scale=0.125, dout=_f64(dout), bf16=dtype == "bf16")
    _check("out", f.out, r["out"], r["~out"])
    _check("h", f.h, r["h"], r["~h"])
    for x in ("dq", "dk", "dv", "dg", "dbeta"):
        _check(x, getattr(g, x), r[x], r["~" + x])
    assert float(g.dg[0, at, 0]) == 0


def test_tokens_that_write_nothing():
    """beta = 0 leaves the state to its decay, and its gradient is that of the value it would have written."""
    a, h0, dout = _inputs(1, 50, 1, 1, 64, 64, "fp32", 4)
    a["beta"].zero_()
    dev = {x: y.cuda() for x, y in a.items()}
    f = delta.delta_fwd(**dev, h0=h0.cuda(), return_state=True, save=True)
    g = delta.delta_bwd(dout.cuda(), **dev, h0=h0.cuda(), saved=f.saved)
    r = ref.delta(**{x: _f64(y) for x, y in a.items()}, scale=0.125, h0=_f64(h0), dout=_f64(dout))
    _check("h", f.h, r["h"], r["~h"])
    _check("dbeta", g.dbeta, r["dbeta"], r["~dbeta"])
    assert float(np.abs(r["dbeta"]).max()) > 0 and bool((g.dk == 0).all()) and bool((g.dv == 0).all())


# ------------------------------------------------------------------ the step

@pytest.mark.parametrize("dtype", ("bf16", "fp32"))
@pytest.mark.parametrize("B,Hk,Hv,dk,dv", ((1, 1, 1, 8, 8), (3, 2, 4, 24, 40), (2, 3, 3, 64, 64), (5, 1, 3, 72, 128),
                                           (2, 1, 1, 128, 8), (7, 2, 2, 128, 128)))
def test_delta_step(B, Hk, Hv, dk, dv, dtype):
    a, h0, _ = _inputs(B, 1, Hk, Hv, dk, dv, dtype, dk + dv)
    a["g"][0, 0, 0] = -float("inf")
    one = {x: y[:, 0].contiguous() for x, y in a.items()}
    h = h0.cuda()
    y = delta.delta_step(h, **{x: t.cuda() for x, t in one.items()}, scale=0.3)
    A = {x: _f64(t) for x, t in one.items()}
    for b in range(B):
        for v in range(Hv):
            k, q, S = A["k"][b, v // (Hv // Hk)], A["q"][b, v // (Hv // Hk)], _f64(h0)[b, v]
            al, be = np.exp(A["g"][b, v]), A["beta"][b, v]
            o, new = ref.step(S, q, k, A["v"][b, v], A["g"][b, v], be, 0.3)
            u = be * (np.abs(A["v"][b, v]) + al * (np.abs(S).T @ np.abs(k)))
            tol = (2 * dk + 32) * E
            _check("h", h[b, v], new, tol * (al * np.abs(S) + np.outer(np.abs(k), u)))
            _check("out", y[b, v], o, tol * 0.3 * (al * (np.abs(S).T @ np.abs(q)) + np.abs(k) @ np.abs(q) * u))


def test_steps_after_a_prompt():
    """A prompt's state and single tokens give the whole sequence, to the chunks' roundings."""
    L, cut = 80, 70
    a, _, _ = _inputs(2, L, 1, 2, 64, 64, "fp32", 6)
    dev = {x: y.cuda() for x, y in a.items()}
    r = ref.delta(**{x: _f64(y) for x, y in a.items()}, scale=0.125)
    h = delta.delta_fwd(**{x: y[:, :cut].contiguous() for x, y in dev.items()}, return_state=True).h
    for t in range(cut, L):
        y = delta.delta_step(h, **{x: v[:, t].contiguous() for x, v in dev.items()})
        _check("out", y, r["out"][:, t], r["~out"][:, t])
    _check("h", h, r["h"], r["~h"])


# ------------------------------------------------- streams, graphs, autograd, size

def test_on_another_stream():
    a, h0, dout = _inputs(2, 100, 1, 2, 64, 64, "bf16", 8)
    dev, h0, dout = {x: y.cuda() for x, y in a.items()}, h0.cuda(), dout.cuda()
    want = delta.delta_fwd(**dev, h0=h0, return_state=True, save=True)
    grads = delta.delta_bwd(dout, **dev, h0=h0, saved=want.saved)
    norms = delta.qknorm_fwd(dev["q"], dev["k"])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = delta.delta_fwd(**dev, h0=h0, return_state=True, save=True, stream=s)
    back = delta.delta_bwd(dout, **dev, h0=h0, saved=got.saved, stream=s)
    other = delta.qknorm_fwd(dev["q"], dev["k"], stream=s)
    s.synchronize()
    assert _equal(got[:2], want[:2]) and _equal(back, grads) and _equal(other, norms)


def test_captured_and_replayed():
    """Two graphs of calls on the same inputs, each with its own memory, replayed on new values."""
    a, h0, dout = _inputs(2, 100, 1, 2, 64, 64, "bf16", 8)
    b, h1, dout1 = _inputs(2, 100, 1, 2, 64, 64, "bf16", 9)
    dev, h0, dout = {x: y.cuda() for x, y in a.items()}, h0.cuda(), dout.cuda()
    step = {x: y[:, 0].contiguous() for x, y in dev.items()}
    h = h0.clone()

    def train():
        q, k = delta.qknorm_fwd(dev["q"], dev["k"])
        f = delta.delta_fwd(q, k, dev["v"], dev["g"], dev["beta"], h0=h0, return_state=True, save=True)
        g = delta.delta_bwd(dout, q, k, dev["v"], dev["g"], dev["beta"], h0=h0, saved=f.saved)
        return (*f[:2], *g, *delta.qknorm_bwd(g.dq, g.dk, dev["q"], dev["k"])[:2])

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        train()
        delta.delta_step(h, **step)
    torch.cuda.synchronize()
    one, two = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(one):
        got = train()
    with torch.cuda.graph(two):
        y = delta.delta_step(h, **step)
    for x in dev:
        dev[x].copy_(b[x])
        step[x].copy_(b[x][:, 0])
    h0.copy_(h1)
    h.copy_(h1)
    dout.copy_(dout1)
    one.replay()
    two.replay()
    torch.cuda.synchronize()
    assert _equal(got, train())
    fresh = h0.clone()
    assert torch.equal(y, delta.delta_step(fresh, **step)) and torch.equal(h, fresh)


@pytest.mark.parametrize("dtype", ("bf16", "fp32"))
def test_autograd(dtype):
    """The differentiable ops give the calls' gradients, also of leaves that reach them by two ways."""
    a, h0, dout = _inputs(2, 70, 1, 2, 64, 64, dtype, 12)
    dev = {x: y.cuda().requires_grad_() for x, y in a.items()}
    h0 = h0.cuda().requires_grad_()
    w = torch.ones(64, device="cuda", requires_grad=True)
    freqs = torch.rand(32, device="cuda")
    q, k = delta.QKNorm.apply(dev["q"], dev["k"], w, w, "rms", 1e-6, freqs)
    y = delta.GatedDelta.apply(q, 0.125 * k, dev["v"], dev["g"], dev["beta"], 0.5, h0)
    y.backward(dout.cuda())
    with torch.no_grad():
        kw = dict(q_weight=w, k_weight=w, norm="rms", freqs=freqs)
        q, k = delta.qknorm_fwd(dev["q"], dev["k"], **kw)
        g = delta.delta_bwd(dout.cuda(), q, 0.125 * k, dev["v"], dev["g"], dev["beta"], 0.5, h0)
        n = delta.qknorm_bwd(g.dq, 0.125 * g.dk, dev["q"], dev["k"], **kw)
    for x, z in (("q", n.dq), ("k", n.dk), ("v", g.dv), ("g", g.dg), ("beta", g.dbeta)):
        assert torch.equal(dev[x].grad, z), x
    assert torch.equal(h0.grad, g.dh0) and torch.equal(w.grad, n.dq_weight + n.dk_weight)


def test_delta_refusals():
    a, h0, dout = _inputs(1, 4, 1, 1, 16, 16, "fp32", 1)
    dev, h0 = {x: y.cuda() for x, y in a.items()}, h0.cuda()
    narrow = {**dev, "q": dev["q"][..., :12].contiguous(), "k": dev["k"][..., :12].contiguous()}
    wide = {**dev, "v": torch.zeros(1, 4, 1, 136, device="cuda")}
    three = {**dev, "q": torch.zeros(1, 4, 2, 16, device="cuda"), "k": torch.zeros(1, 4, 2, 16, device="cuda")}
    for kw, status in ((narrow, lion.ERR_UNSUPPORTED), (wide, lion.ERR_UNSUPPORTED), (three, lion.ERR_INVALID_ARG),
                       ({**dev, "scale": float("nan")}, lion.ERR_INVALID_ARG),
                       ({**dev, "workspace": torch.empty(256, dtype=torch.uint8, device="cuda")}, lion.ERR_INVALID_ARG),
                       ({**dev, "lengths": torch.ones(1, dtype=torch.int32)}, lion.ERR_INVALID_ARG)):
        with pytest.raises(lion.LionError) as e:
            delta.delta_fwd(**kw)
        assert e.value.status == status
    with pytest.raises(ValueError):
        delta.delta_bwd(dout.cuda(), **dev, saved=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        delta.delta_step(h0[..., ::2], **{x: y[:, 0].contiguous() for x, y in dev.items()})


def test_delta_of_more_than_two_to_the_31_values():
    """Heads are what they are alone, wherever they lie."""
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 100e9:
        pytest.skip("not enough free memory")
    L, H, d = 280000, 64, 128
    gen = torch.Generator(device="cuda").manual_seed(1)
    mk = lambda *s: torch.randn(*s, generator=gen, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    q, v = mk(1, L, H, d), mk(1, L, H, d)
    assert q.numel() > 2 ** 31
    q, k = delta.qknorm_fwd(q, q.flip(2))
    g, beta = -torch.rand(1, L, H, device="cuda").bfloat16(), torch.rand(1, L, H, device="cuda").bfloat16()
    f = delta.delta_fwd(q, k, v, g, beta, return_state=True, save=True)
    r = delta.delta_bwd(v, q, k, v, g, beta, saved=f.saved)
    for h in (0, 63):
        one = [x[:, :, h:h + 1].contiguous() for x in (q, k, v, g, beta)]
        s = delta.delta_fwd(*one, return_state=True, save=True)
        assert torch.equal(s.out, f.out[:, :, h:h + 1]) and torch.equal(s.h[0, 0], f.h[0, h])
        e = delta.delta_bwd(one[2], *one, saved=s.saved)
        for x in ("dq", "dk", "dv", "dg", "dbeta"):
            assert torch.equal(getattr(e, x), getattr(r, x)[:, :, h:h + 1]), x


@pytest.mark.parametrize("reverse", (False, True))
@pytest.mark.parametrize("dk,dv", ((64, 64), (128, 72), (24, 8)))
def test_delta_in_segments(dk, dv, reverse):
    """Long sequences of few heads are walked in segments; some of the batch end before the last ones, one has none."""
    n = (1700, 620, 32, 0)
    a, h0, dout = _inputs(4, 1700, 1, 1, dk, dv, "bf16", dk, decay=6.0)
    r = ref.delta(**{x: _f64(y) for x, y in a.items()}, scale=dk ** -0.5, h0=_f64(h0), lengths=n, reverse=reverse,
                  dout=_f64(dout), bf16=True)
    for b in range(4):
        for x in (*a.values(), dout):
            x[b, n[b]:] = float("nan")
    dev = {x: y.cuda() for x, y in a.items()}
    how = dict(h0=h0.cuda(), lengths=torch.tensor(n, dtype=torch.int32, device="cuda"), reverse=reverse)
    f = delta.delta_fwd(**dev, **how, return_state=True, save=True)
    g = delta.delta_bwd(dout.cuda(), **dev, **how, saved=f.saved)
    for x, y in (("out", f.out), ("h", f.h), ("dq", g.dq), ("dk", g.dk), ("dv", g.dv), ("dg", g.dg),
                 ("dbeta", g.dbeta), ("dh0", g.dh0)):
        _exact_enough(x, y, r[x])
    assert torch.equal(f.h[3], h0[3].cuda()) and bool((f.out[2, 32:] == 0).all())
    assert _equal(delta.delta_fwd(**dev, **how, return_state=True)[:2], f[:2])


@pytest.mark.parametrize("dtype", ("bf16", "fp32"))
@pytest.mark.parametrize("B,Hv,dk,dv,reverse", ((160, 2, 64, 64, False), (102, 3, 40, 24, True), (90, 2, 128, 128, False)))
def test_delta_of_many_sequences(B, Hv, dk, dv, reverse, dtype):
    """More walks than an SM holds at once, of batches above and below the 128 sequences that are ordered by length."""
    L = 70
    a, h0, dout = _inputs(B, L, 1, Hv, dk, dv, dtype, B)
    n = [(37 * b) % (L + 1) for b in range(B)]
    r = ref.delta(**{x: _f64(y) for x, y in a.items()}, scale=dk ** -0.5, h0=_f64(h0), lengths=n, reverse=reverse,
                  dout=_f64(dout), bf16=dtype == "bf16")
    for b in range(B):
        for x in (*a.values(), dout):
            x[b, n[b]:] = float("nan")
    dev = {x: y.cuda() for x, y in a.items()}
    how = dict(h0=h0.cuda(), lengths=torch.tensor(n, dtype=torch.int32, device="cuda"), reverse=reverse)
    f = delta.delta_fwd(**dev, **how, return_state=True, save=True)
    g = delta.delta_bwd(dout.cuda(), **dev, **how, saved=f.saved)
    for x, y in (("out", f.out), ("h", f.h), ("dq", g.dq), ("dk", g.dk), ("dv", g.dv), ("dg", g.dg),
                 ("dbeta", g.dbeta), ("dh0", g.dh0)):
        _check(x, y, r[x], r["~" + x])
        _exact_enough(x, y, r[x])
    assert _equal(delta.delta_fwd(**dev, **how, return_state=True)[:2], f[:2])


def test_results_in_place_of_inputs_are_refused():
    """A token's results are written while others are still read."""
    a, h0, _ = _inputs(1, 40, 1, 1, 64, 64, "bf16", 1)
    dev = {x: y.cuda() for x, y in a.items()}
    before = {x: y.clone() for x, y in dev.items()}
    for call in (*(lambda x=x: delta.delta_fwd(**dev, out=dev[x]) for x in "qkv"),
                 lambda: delta.qknorm_fwd(dev["q"], dev["k"], q_out=dev["q"]),
                 lambda: delta.qknorm_fwd(dev["q"], dev["k"], k_out=dev["k"])):
        with pytest.raises(lion.LionError) as e:
            call()
        assert e.value.status == lion.ERR_INVALID_ARG and _equal(before.values(), dev.values())


def test_two_streams_at_once():
    """Calls on two streams, each with its own workspaces, do not meet."""
    sets = [_inputs(2, 900, 2, 4, 64, 64, "bf16", s) for s in (1, 2)]
    sets = [({x: y.cuda() for x, y in a.items()}, h.cuda(), d.cuda()) for a, h, d in sets]

    def train(a, h0, dout, s=None):
        f = delta.delta_fwd(**a, h0=h0, return_state=True, save=True, stream=s)
        return (*f[:2], *delta.delta_bwd(dout, **a, h0=h0, saved=f.saved, stream=s))

    want = [train(*x) for x in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(3):
        got = [train(*x, s) for x, s in zip(sets, streams)]
        torch.cuda.synchronize()
        assert all(_equal(x, y) for x, y in zip(got, want))


@pytest.mark.parametrize("dk,dv", ((64, 64), (40, 24)))
def test_segments_in_a_workspace_of_the_callers(dk, dv):
    """What a workspace held before does not matter, and gradients without the forward's `saved` are the same."""
    B, L, Hk, Hv = 2, 1666, 1, 2
    a, h0, dout = _inputs(B, L, Hk, Hv, dk, dv, "bf16", 17, decay=6.0)
    dev, dout = {x: y.cuda() for x, y in a.items()}, dout.cuda()
    how = dict(h0=h0.cuda(), lengths=torch.tensor([L, 777], dtype=torch.int32, device="cuda"))
    f = delta.delta_fwd(**dev, **how, return_state=True, save=True)
    g = delta.delta_bwd(dout, **dev, **how, saved=f.saved)
    code = lion.DTYPE_BF16
    nan = lambda n: torch.full((n,), 255, dtype=torch.uint8, device="cuda")  # noqa: E731
    ws = nan(delta.delta_workspace_bytes(B, L, Hk, Hv, dk, dv, code))
    assert _equal(delta.delta_fwd(**dev, **how, return_state=True, workspace=ws)[:2], f[:2])
    for saved in (f.saved, None):
        ws = nan(delta.delta_bwd_workspace_bytes(B, L, Hk, Hv, dk, dv, code, saved is not None))
        assert _equal(delta.delta_bwd(dout, **dev, **how, saved=saved, workspace=ws), g)
    # captured and replayed on other values
    one = torch.cuda.CUDAGraph()
    with torch.cuda.graph(one):
        x = delta.delta_fwd(**dev, **how, return_state=True, save=True)
        y = delta.delta_bwd(dout, **dev, **how, saved=x.saved)
    dev["v"].mul_(2)
    dout.neg_()
    one.replay()
    f = delta.delta_fwd(**dev, **how, return_state=True, save=True)
    assert _equal(x[:2], f[:2]) and _equal(y, delta.delta_bwd(dout, **dev, **how, saved=f.saved))
