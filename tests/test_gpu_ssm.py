"""The state space block on the GPU against 64-bit references written token by
token from the formulas (ssm_reference.py).

Bounds, set before the first run.  With e = 2^-24 and, for every result, its
magnitude (the same formulas with every term's absolute value):
  scan         e (64 + 16 L + 2 (N + D + B L)) magnitude: 16 roundings of a
               decay's exponent a step (|delta A| <= 8 here, two roundings of
               it), 64 for the nonlinearities, and one for each term of a sum;
  convolution  e (64 + 2 B L) magnitude;
  layer norm   the rounding of mean and variance carried through (below);
A bfloat16 result lies between the bound's two ends rounded to bfloat16
(rounding keeps the order)."""
import numpy as np
import pytest
import torch

import ssm_reference as ref
from bidirectional_masked_linear_gb300 import lion, ssm

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
T = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bidirectional_masked_linear_gb300 import build
    lion.load(build.build())


def _check(name, got, want, tol):
    got = got.detach()
    g = got.double().cpu().numpy()
    assert g.shape == want.shape, (name, g.shape, want.shape)
    tol = np.broadcast_to(tol, want.shape) + 1e-30
    if got.dtype == torch.bfloat16:
        low, high = (torch.from_numpy(np.ascontiguousarray(v)).bfloat16().double().numpy()
                     for v in (want - tol, want + tol))
        inside = (g >= low) & (g <= high)
    else:
        inside = np.abs(g - want) <= tol   # NaN fails too
    assert inside.all(), f"{name}: {np.sum(~inside)} of {inside.size} off, by up to {np.nanmax(np.abs(g - want) / tol)} of the bound"


def _f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


# ------------------------------------------------------------------ layer norm

NORM = [(1, 1), (3, 7), (5, 64), (197, 192), (33, 256), (7, 257), (9, 768), (4, 1000), (70, 1024), (6, 1025),
        (5, 2048), (3, 4095), (4, 8192), (2, 16384), (2500, 40)]


@pytest.mark.parametrize("dtype", ("bf16", "fp32"))
@pytest.mark.parametrize("rows,cols", NORM)
def test_layernorm(rows, cols, dtype):
    g = torch.Generator().manual_seed(rows * 7 + cols)
    x = (3.0 + 2.0 * torch.randn(rows, cols, generator=g)).to(T[dtype]).cuda()
    dy = torch.randn(rows, cols, generator=g).to(T[dtype]).cuda()
    w, b = (1 + 0.3 * torch.randn(cols, generator=g)).cuda(), torch.randn(cols, generator=g).cuda()
    eps = 1e-5
    y, mean, rstd = ssm.layernorm_fwd(x, w, b, eps, save_stats=True)
    dx, dw, db = ssm.layernorm_bwd(dy, x, w, mean, rstd)
    X, DY, W, Bb = _f64(x), _f64(dy), _f64(w), _f64(b)
    r = ref.layernorm(X, W, Bb, eps, DY)
    q = (cols / 32 + 16) * E
    rs = 1 / np.sqrt(X.var(-1, keepdims=True) + eps)
    xh = (X - X.mean(-1, keepdims=True)) * rs
    exh = q * rs * (np.abs(X) + np.abs(X).mean(-1, keepdims=True)) + 2 * q * np.abs(xh)
    # a mean off by m shifts the centred values and, with them, the variance
    exh = exh + np.abs(xh) * exh.mean(-1, keepdims=True)
    _check("y", y, r["y"], np.abs(W) * exh + 4 * E * np.abs(r["y"]) + 4 * E * np.abs(Bb))
    G = np.abs(DY * W)
    m1, m2 = G.mean(-1, keepdims=True), (G * np.abs(xh)).mean(-1, keepdims=True)
    e2 = (G * exh).mean(-1, keepdims=True)
    _check("dx", dx, r["dx"], rs * (q * (G + m1 + np.abs(xh) * m2) + exh * m2 + np.abs(xh) * e2)
           + q * np.abs(r["dx"]))
    n = rows + 64
    _check("dweight", dw, r["dweight"], (np.abs(DY) * exh).sum(0) + n * E * (np.abs(DY * xh)).sum(0))
    _check("dbias", db, r["dbias"], n * E * np.abs(DY).sum(0))
    assert torch.equal(ssm.layernorm_fwd(x, w, b, eps), y)
    again = ssm.layernorm_bwd(dy, x, w, mean, rstd)
    assert all(torch.equal(p, s) for p, s in zip(again, (dx, dw, db)))


def test_layernorm_without_bias_of_strided_rows():
    """A column slice, and one that starts off 16 bytes, equal their copies bit for bit."""
    wide = torch.randn(37, 300, device="cuda").bfloat16()
    w = torch.randn(128, device="cuda")
    for at in (0, 8, 3):
        x = wide[:, at:at + 128]
        a, b = ssm.layernorm_fwd(x, w, save_stats=True), ssm.layernorm_fwd(x.contiguous(), w, save_stats=True)
        assert all(torch.equal(p, s) for p, s in zip(a, b))
        dy = torch.randn(37, 128, device="cuda").bfloat16()
        p = ssm.layernorm_bwd(dy, x, w, a[1], a[2], bias=False)
        s = ssm.layernorm_bwd(dy, x.contiguous(), w, a[1], a[2], bias=True)
        assert p[2] is None and torch.equal(p[0], s[0]) and torch.equal(p[1], s[1])


def test_layernorm_constant_row():
    """A row without variance: xh = 0 up to the rounding of the mean, times 1/sqrt(eps)."""
    x = torch.full((2, 100), 5.0, device="cuda")
    w, b = torch.ones(100, device="cuda"), torch.full((100,), 0.25, device="cuda")
    y = ssm.layernorm_fwd(x, w, b, 1e-5)
    assert float((y - 0.25).abs().max()) <= 5.0 * 20 * E / np.sqrt(1e-5)


# ----------------------------------------------------------------- convolution

CONV = [  # B, L, D, K, ragged, state, reverse
    (1, 1, 1, 4, None, False, False), (2, 3, 8, 4, None, True, False), (2, 16, 24, 3, None, False, True),
    (3, 17, 33, 2, (17, 0, 1), True, False), (3, 18, 40, 4, (2, 18, 0), True, True),
    (4, 130, 264, 4, (130, 3, 64, 1), False, True), (2, 49, 513, 3, (16, 48), True, False),
]


@pytest.mark.parametrize("dtype", ("bf16", "fp32"))
@pytest.mark.parametrize("act", ("silu", "none"))
@pytest.mark.parametrize("B,L,D,K,lens,state,reverse", CONV)
def test_conv(B, L, D, K, lens, state, reverse, act, dtype):
    g = torch.Generator().manual_seed(L * 31 + D)
    mk = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x, dy = mk(B, L, D).to(T[dtype]), mk(B, L, D).to(T[dtype])
    w, b = 0.5 * mk(D, K), mk(D)
    st = mk(B, K - 1, D).to(T[dtype]) if state else None
    n = list(lens) if lens else None
    clean = [_f64(v) for v in (x, w, b, st, dy)]
    if n:
        for q in range(B):   # what a padded place holds does not matter
            x[q, n[q]:] = float("nan")
            dy[q, n[q]:] = float("inf")
            clean[0][q, n[q]:] = clean[4][q, n[q]:] = 0
    X, W, Bb, S, DY = clean
    r = ref.conv(X, W, Bb, act == "silu", S, n, reverse, DY)
    m = ref.conv(X, W, Bb, act == "silu", S, n, reverse, DY, absolute=True)
    c = lambda t: None if t is None else t.cuda()  # noqa: E731
    lt = torch.tensor(n, dtype=torch.int32).cuda() if n else None
    kw = dict(activation=act, state=c(st), lengths=lt, reverse=reverse)
    y, new = ssm.conv_fwd(c(x), c(w), c(b), return_state=True, **kw)
    gr = ssm.conv_bwd(c(dy), c(x), c(w), c(b), **kw)
    f = E * (64 + 2 * B * L)
    _check("y", y, r["y"], f * m["y"])
    _check("state", new, r["state"], 0.0)
    _check("dx", gr.dx, r["dx"], f * m["dx"])
    _check("dweight", gr.dweight, r["dweight"], f * m["dweight"])
    _check("dbias", gr.dbias, r["dbias"], f * m["dbias"])
    if state:
        _check("dstate", gr.dstate, r["dstate"], f * m["dstate"])
    else:
        assert gr.dstate is None
    again = ssm.conv_bwd(c(dy), c(x), c(w), c(b), **kw)
    assert all(p is None or torch.equal(p, s) for p, s in zip(again, gr))


@pytest.mark.parametrize("dtype", ("bf16", "fp32"))
@pytest.mark.parametrize("K", (2, 3, 4))
def test_conv_prompt_then_steps(K, dtype):
    """A prompt, its state, then one token at a time: the outputs of the whole sequence, bit for bit."""
    B, L, D = 3, 21, 70
    x = torch.randn(B, L, D, device="cuda").to(T[dtype])
    w, b = torch.randn(D, K, device="cuda"), torch.randn(D, device="cuda")
    whole, end = ssm.conv_fwd(x, w, b, return_state=True)
    y, st = ssm.conv_fwd(x[:, :9].contiguous(), w, b, return_state=True)
    assert torch.equal(y, whole[:, :9])
    y2, st2 = ssm.conv_fwd(x[:, 9:10].contiguous(), w, b, state=st, return_state=True)
    assert torch.equal(y2, whole[:, 9:10])
    st = st2.clone()
    for t in range(10, L):
        assert torch.equal(ssm.conv_step(x[:, t].contiguous(), st, w, b), whole[:, t])
    assert torch.equal(st, end)


def test_conv_views():
    """Slices of a wider tensor, at and off 16 bytes, equal their copies bit for bit."""
    w, b = torch.randn(64, 4, device="cuda"), torch.randn(64, device="cuda")
    dy = torch.randn(2, 33, 64, device="cuda").bfloat16()
    for B, L in ((2, 33), (1, 33), (2, 1)):
        wide = torch.randn(B, L, 200, device="cuda").bfloat16()
        for at in (0, 8, 5):
            x = wide[..., at:at + 64]
            assert torch.equal(ssm.conv_fwd(x, w, b), ssm.conv_fwd(x.contiguous(), w, b))
            d = dy[:B, :L].contiguous()
            p, s = ssm.conv_bwd(d, x, w, b), ssm.conv_bwd(d, x.contiguous(), w, b)
            assert torch.equal(p.dx, s.dx) and torch.equal(p.dweight, s.dweight)


def test_conv_offsets_past_32_bits():
    """More than 2^31 values: the last sequence equals the same sequence alone, bit for bit."""
    B, L, D = 9, 120000, 2048
    x = torch.empty(B, L, D, dtype=torch.bfloat16, device="cuda").normal_()
    w, b = torch.randn(D, 4, device="cuda"), torch.randn(D, device="cuda")
    y = ssm.conv_fwd(x, w, b)
    assert torch.equal(y[-1:], ssm.conv_fwd(x[-1:], w, b))
    assert torch.equal(y[0, :100], ssm.conv_fwd(x[:1, :100].contiguous(), w, b)[0])


# -------------------------------------------------------------- selective scan

def _scan_inputs(B, L, D, N, G, dtype, gate, skip, bias, state, softplus, seed):
    g = torch.Generator().manual_seed(seed)
    mk = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    t = T[dtype]
    a = dict(u=mk(B, L, D).to(t), dt=(0.5 * mk(B, L, D)).to(t),
             # |delta A| <= 8 with delta = softplus(dt + bias) <= 2.5
             A=-(0.05 + 3.0 * torch.rand(D, N, generator=g)), Bm=mk(B, L, G, N).to(t), Cm=mk(B, L, G, N).to(t))
    a["dt"] = a["dt"].clamp(-2, 1.4) if softplus else a["dt"].abs().clamp(0, 2)
    if bias:
        a["dt_bias"] = (-2.0 * torch.rand(D, generator=g)) if softplus else 0.5 * torch.rand(D, generator=g)
    if skip:
        a["Dskip"] = mk(D)
    if gate:
        a["z"] = mk(B, L, D).to(t)
    if state:
        a["h0"] = mk(B, D, N)
    return a, mk(B, L, D).to(t)


SCAN = [  # B, L, D, N, G, lengths, options off, reverse
    (1, 1, 1, 8, 1, None, "", False),
    (2, 7, 5, 16, 1, None, "", False),
    (1, 16, 64, 16, 1, None, "state", False),
    (2, 17, 33, 16, 3, None, "", True),
    (3, 65, 130, 16, 1, (65, 0, 1), "", False),
    (3, 65, 130, 16, 2, (3, 65, 0), "", True),
    (2, 64, 257, 8, 1, None, "gate", False),
    (2, 130, 40, 32, 1, (129, 33), "skip bias", True),
    (2, 63, 19, 64, 1, None, "softplus", False),
    (2, 100, 34, 64, 2, (64, 100), "gate state", True),
    (1, 600, 24, 16, 1, None, "", False),          # several segments
    (2, 513, 12, 8, 1, (513, 200), "", True),      # several, one sequence not in the first
    (2, 450, 10, 64, 1, (300, 450), "", False),
]


@pytest.mark.parametrize("dtype", ("bf16", "fp32"))
@pytest.mark.parametrize("B,L,D,N,G,lens,off,reverse", SCAN)
def test_scan(B, L, D, N, G, lens, off, reverse, dtype):
    sp = "softplus" not in off
    a, dout = _scan_inputs(B, L, D, N, G, dtype, "gate" not in off, "skip" not in off, "bias" not in off,
                           "state" not in off, sp, seed=B * 1000 + L)
    n = list(lens) if lens else None
    A64 = {k: _f64(v) for k, v in a.items()}
    DO = _f64(dout)
    if n:
        for q in range(B):   # what a padded place holds does not matter
            for k in ("u", "dt", "Bm", "Cm", "z"):
                if k in a:
                    a[k][q, n[q]:] = float("nan")
                    A64[k][q, n[q]:] = 0
            dout[q, n[q]:] = float("-inf")
            DO[q, n[q]:] = 0
    how = dict(dt_softplus=sp, lengths=n, reverse=reverse)
    r, m = ref.scan(**A64, **how, dout=DO), ref.scan(**A64, **how, dout=DO, absolute=True)
    dev = {k: v.cuda() for k, v in a.items()}
    how["lengths"] = torch.tensor(n, dtype=torch.int32).cuda() if n else None
    f = ssm.scan_fwd(**dev, **how, return_state=True, save_states=True)
    gr = ssm.scan_bwd(dout.cuda(), **dev, **how, states=f.states)
    tol = E * (64 + 16 * L + 2 * (N + D + B * L))
    _check("out", f.out, r["out"], tol * m["out"])
    _check("h", f.h, r["h"], tol * m["h"])
    for k in ("du", "ddt", "dA", "dB", "dC"):
        _check(k, getattr(gr, k), r[k], tol * m[k])
    for k, src in (("dDskip", "Dskip"), ("dz", "z"), ("ddt_bias", "dt_bias"), ("dh0", "h0")):
        if src in a:
            _check(k, getattr(gr, k), r[k], tol * m[k])
        else:
            assert getattr(gr, k) is None
    # without the saved states they are computed again, to the same bits; and the same call gives the same bits
    for again in (ssm.scan_bwd(dout.cuda(), **dev, **how), ssm.scan_bwd(dout.cuda(), **dev, **how, states=f.states)):
        assert all(p is None or torch.equal(p, s) for p, s in zip(again, gr))
    assert torch.equal(ssm.scan_fwd(**dev, **how).out, f.out)


@pytest.mark.parametrize("N", (8, 16, 32, 64))
def test_scan_states(N):
    """The saved states are the states before every 16th token."""
    B, L, D, E = 2, 3 * ssm.STATE_EVERY + 5, 37, ssm.STATE_EVERY
    a, _ = _scan_inputs(B, L, D, N, 1, "fp32", True, True, True, True, True, seed=N)
    dev = {k: v.cuda() for k, v in a.items()}
    f = ssm.scan_fwd(**dev, save_states=True)
    assert torch.equal(f.states[:, 0], dev["h0"])
    for k in range(1, f.states.shape[1]):
        cut = {q: v[:, :k * E].contiguous() if q in ("u", "dt", "Bm", "Cm", "z") else v for q, v in dev.items()}
        h = ssm.scan_fwd(**cut, return_state=True).h
        err = (h - f.states[:, k]).abs().max()
        assert float(err) <= 1e-5 * float(h.abs().max())


@pytest.mark.parametrize("dtype", ("bf16", "fp32"))
@pytest.mark.parametrize("N,G", ((8, 1), (16, 2), (32, 1), (64, 3)))
def test_scan_steps(N, G, dtype):
    """One token at a time from a prompt's state, against the reference of the whole sequence."""
    B, L, D = 3, 12, 42
    a, _ = _scan_inputs(B, L, D, N, G, dtype, True, True, True, True, True, seed=N)
    A64 = {k: _f64(v) for k, v in a.items()}
    r, m = ref.scan(**A64), ref.scan(**A64, absolute=True)
    dev = {k: v.cuda() for k, v in a.items()}
    per = ("u", "dt", "Bm", "Cm", "z")
    f = ssm.scan_fwd(**{k: v[:, :7].contiguous() if k in per else v for k, v in dev.items()}, return_state=True)
    h = f.h
    rest = {k: dev[k] for k in ("A", "Dskip", "dt_bias")}
    outs = [f.out]
    for t in range(7, L):
        outs.append(ssm.scan_step(h, **{k: dev[k][:, t].contiguous() for k in per}, **rest)[:, None])
    tol = E * (64 + 16 * L + 2 * N)
    _check("out", torch.cat(outs, 1), r["out"], tol * m["out"])
    _check("h", h, r["h"], tol * m["h"])


def test_scan_step_of_unaligned_rows():
    """B and C off their vectors' alignment: the aligned copies' bits."""
    B, D, N = 5, 33, 8
    a, _ = _scan_inputs(B, 1, D, N, 1, "bf16", True, True, True, True, True, seed=6)
    dev = {k: v.cuda() for k, v in a.items()}
    args = {k: dev[k][:, 0].contiguous() for k in ("u", "dt", "Bm", "Cm", "z")}
    rest = {k: dev[k] for k in ("A", "Dskip", "dt_bias")}
    h1, h2 = dev["h0"].clone(), dev["h0"].clone()
    want = ssm.scan_step(h1, **args, **rest)
    for k in ("u", "dt", "Bm", "Cm", "z"):
        flat = torch.empty(args[k].numel() + 1, dtype=torch.bfloat16, device="cuda")
        flat[1:] = args[k].flatten()
        args[k] = flat[1:].view(args[k].shape)
    assert torch.equal(ssm.scan_step(h2, **args, **rest), want) and torch.equal(h1, h2)


def test_scan_step_captured_in_a_graph():
    B, D, N = 2, 48, 16
    a, _ = _scan_inputs(B, 1, D, N, 1, "bf16", True, True, True, True, True, seed=5)
    dev = {k: v.cuda() for k, v in a.items()}
    args = {k: dev[k][:, 0].contiguous() for k in ("u", "dt", "Bm", "Cm", "z")}
    rest = {k: dev[k] for k in ("A", "Dskip", "dt_bias")}
    h1, h2 = dev["h0"].clone(), dev["h0"].clone()
    want = [ssm.scan_step(h1, **args, **rest) for _ in range(3)]
    out = torch.empty(B, D, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ssm.scan_step(h2, **args, **rest, out=out)
    h2.copy_(dev["h0"])
    for w in want:
        graph.replay()
        assert torch.equal(out, w)
    assert torch.equal(h1, h2)


def test_scan_views_and_streams():
    """Slices of wider projections, at and off 16 bytes, another stream and the caller's own workspace: the copies'
    bits."""
    B, L, D, N, G = 2, 150, 48, 16, 2
    a, dout = _scan_inputs(B, L, D, N, G, "bf16", True, True, True, False, True, seed=9)
    dev = {k: v.cuda() for k, v in a.items()}
    dout = dout.cuda()
    want = ssm.scan_fwd(**dev, save_states=True)
    grads = ssm.scan_bwd(dout, **dev, states=want.states)
    side = torch.cuda.Stream()
    for off in (0, 8, 3):
        v = dict(dev)
        for k in ("u", "dt", "z"):
            wide = torch.full((B, L, 3 * D), float("nan"), dtype=torch.bfloat16, device="cuda")
            wide[..., off:off + D] = dev[k]
            v[k] = wide[..., off:off + D]
        wide = torch.full((B, L, 100), float("nan"), dtype=torch.bfloat16, device="cuda")
        wide[..., off:off + 32], wide[..., off + 32:off + 64] = dev["Bm"].flatten(2), dev["Cm"].flatten(2)
        v["Bm"] = wide[..., off:off + 32].unflatten(2, (G, N))
        v["Cm"] = wide[..., off + 32:off + 64].unflatten(2, (G, N))
        torch.cuda.synchronize()
        ws = torch.empty(max(256, ssm.scan_workspace_bytes(B, L, D, N, G)), dtype=torch.uint8, device="cuda")
        f = ssm.scan_fwd(**v, save_states=True, stream=side, workspace=ws)
        g = ssm.scan_bwd(dout, **v, states=f.states, stream=side)
        side.synchronize()
        assert torch.equal(f.out, want.out) and torch.equal(f.states, want.states)
        assert all(p is None or torch.equal(p, s) for p, s in zip(g, grads))


def test_scan_long():
    """A long sequence of few channels (many segments): against the same recurrence in 64 bits, on the GPU."""
    B, L, D, N = 1, 20011, 24, 16
    a, _ = _scan_inputs(B, L, D, N, 1, "fp32", True, True, True, True, True, seed=3)
    dev = {k: v.cuda() for k, v in a.items()}
    f = ssm.scan_fwd(**dev, return_state=True)
    d = {k: v.double() for k, v in dev.items()}
    delta = torch.nn.functional.softplus(d["dt"] + d["dt_bias"])
    h, mh, ys, ms = d["h0"], d["h0"].abs(), [], []
    for t in range(L):
        e = torch.exp(delta[:, t, :, None] * d["A"])
        x = (delta[:, t] * d["u"][:, t])[..., None] * d["Bm"][:, t]
        h, mh = e * h + x, e * mh + x.abs()
        ys.append((h * d["Cm"][:, t]).sum(-1) + d["Dskip"] * d["u"][:, t])
        ms.append((mh * d["Cm"][:, t].abs()).sum(-1) + (d["Dskip"] * d["u"][:, t]).abs())
    gate = d["z"] * torch.sigmoid(d["z"])
    # a state forgets: the decays are exp(-0.05 delta) and less, so some 2000 steps count
    tol = E * (64 + 16 * 2000)
    assert bool(((f.out - torch.stack(ys, 1) * gate).abs() <= tol * torch.stack(ms, 1) * gate.abs() + 1e-30).all())
    assert bool(((f.h - h).abs() <= tol * mh).all())


def test_lengths_out_of_range_are_clamped():
    B, L, D, N = 3, 40, 24, 16
    a, dout = _scan_inputs(B, L, D, N, 1, "bf16", True, True, True, True, True, seed=21)
    dev = {k: v.cuda() for k, v in a.items()}
    w, b = torch.randn(D, 4, device="cuda"), torch.randn(D, device="cuda")
    got = []
    for n in ([-5, 1000, 7], [0, L, 7]):
        lt = torch.tensor(n, dtype=torch.int32, device="cuda")
        f = ssm.scan_fwd(**dev, lengths=lt, return_state=True, save_states=True)
        g = ssm.scan_bwd(dout.cuda(), **dev, lengths=lt, states=f.states)
        y, st = ssm.conv_fwd(dev["u"], w, b, lengths=lt, return_state=True)
        c = ssm.conv_bwd(dout.cuda(), dev["u"], w, b, lengths=lt)
        got.append([*f, *g, y, st, c.dx, c.dweight, c.dbias])
    assert all(torch.equal(p, s) for p, s in zip(*got))


def test_scan_offsets_past_32_bits():
    """More than 2^31 values: the last sequence against the same sequence alone (cut differently)."""
    B, L, D, N = 3, 360000, 2048, 8
    big = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda").normal_()  # noqa: E731
    u, dt, Bm, Cm = big(B, L, D), big(B, L, D).mul_(0.1), big(B, L, N), big(B, L, N)
    A = -(0.5 + torch.rand(D, N, device="cuda"))
    f = ssm.scan_fwd(u, dt, A, Bm, Cm, return_state=True)
    last = ssm.scan_fwd(u[-1:], dt[-1:], A, Bm[-1:], Cm[-1:], return_state=True)
    # states of order one that forget within some ten tokens: a cut moves the fp32 sums by a few roundings
    assert float((f.h[-1:] - last.h).abs().max()) <= 1e-5 * float(last.h.abs().max())
    for lo in range(0, L, 40000):   # half a bfloat16 unit apart at most where the sums round differently
        p, q = f.out[-1, lo:lo + 40000].float(), last.out[0, lo:lo + 40000].float()
        assert bool(((p - q).abs() <= 2.0 ** -7 * q.abs() + 1e-4).all())


def test_layernorm_offsets_past_32_bits():
    x = torch.empty(280000, 8192, dtype=torch.bfloat16, device="cuda").normal_()
    w = torch.randn(8192, device="cuda")
    y, mean, rstd = ssm.layernorm_fwd(x, w, save_stats=True)
    assert torch.equal(y[-3:], ssm.layernorm_fwd(x[-3:], w))
    dx, _, _ = ssm.layernorm_bwd(x, x, w, mean, rstd, bias=False)
    last, _, _ = ssm.layernorm_bwd(x[-3:], x[-3:], w, mean[-3:], rstd[-3:], bias=False)
    assert torch.equal(dx[-3:], last)


def test_scan_captured_in_a_graph():
    """A prompt's scan with segments, its gradients, conv and norm replay to the same bits."""
    B, L, D, N = 1, 700, 32, 16
    a, dout = _scan_inputs(B, L, D, N, 1, "bf16", True, True, True, True, True, seed=31)
    dev, dout = {k: v.cuda() for k, v in a.items()}, dout.cuda()
    w, nw = torch.randn(D, 4, device="cuda"), torch.randn(D, device="cuda")

    def run():
        f = ssm.scan_fwd(**dev, save_states=True)
        c = ssm.conv_bwd(dout, dev["u"], w)
        return [f.out, f.states, *ssm.scan_bwd(dout, **dev, states=f.states), c.dx, c.dweight,
                ssm.layernorm_fwd(dev["u"], nw)]

    want = run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, s) for p, s in zip(got, want))


def test_scan_growing_states():
    """A > 0 over several segments: nothing before the first input, whatever the factors overflow to."""
    B, L, D, N = 1, 1600, 8, 16
    u, dt = torch.zeros(B, L, D, device="cuda"), torch.ones(B, L, D, device="cuda")
    u[:, -20:] = 1.0
    A = torch.full((D, N), 0.5, device="cuda")
    ones = torch.ones(B, L, N, device="cuda")
    f = ssm.scan_fwd(u, dt, A, ones, ones, dt_softplus=False, return_state=True)
    h = sum(np.exp(0.5 * k) for k in range(20))
    assert bool((f.out[:, :-20] == 0).all())
    assert float((f.h / h - 1).abs().max()) <= 20 * 16 * E


def test_autograd_functions():
    """The three ops in one graph: gradients equal the entry points' own."""
    B, L, D, N = 2, 40, 32, 16
    a, dout = _scan_inputs(B, L, D, N, 1, "fp32", True, True, True, True, True, seed=11)
    dev = {k: v.cuda().requires_grad_() for k, v in a.items()}
    w = torch.randn(D, 4, device="cuda", requires_grad=True)
    nw = torch.ones(D, device="cuda", requires_grad=True)
    nb = torch.zeros(D, device="cuda", requires_grad=True)
    x = torch.randn(B, L, D, device="cuda", requires_grad=True)
    n = ssm.LayerNorm.apply(x, nw, nb, 1e-5)
    u = ssm.CausalConv.apply(n, w, None)
    out = ssm.SelectiveScan.apply(u, *(dev[k] for k in ("dt", "A", "Bm", "Cm", "Dskip", "z", "dt_bias")), True,
                                  dev["h0"])
    out.backward(dout.cuda())
    args = {k: v.detach() for k, v in dev.items()}
    g = ssm.scan_bwd(dout.cuda(), **{**args, "u": u.detach()})
    for k, s in (("dt", g.ddt), ("A", g.dA), ("Bm", g.dB), ("Cm", g.dC), ("Dskip", g.dDskip), ("z", g.dz),
                 ("dt_bias", g.ddt_bias), ("h0", g.dh0)):
        assert torch.equal(dev[k].grad, s), k
    c = ssm.conv_bwd(g.du, n.detach(), w.detach())
    assert torch.equal(w.grad, c.dweight)
    y, mean, rstd = ssm.layernorm_fwd(x.detach(), nw.detach(), nb.detach(), save_stats=True)
    dx, dw, db = ssm.layernorm_bwd(c.dx, x.detach(), nw.detach(), mean, rstd)
    assert torch.equal(x.grad, dx) and torch.equal(nw.grad, dw) and torch.equal(nb.grad, db)


def test_refusals():
    x = torch.randn(2, 4, 8, device="cuda")
    w = torch.randn(8, 4, device="cuda")
    with pytest.raises(lion.LionError) as e:
        ssm.conv_fwd(x, torch.randn(8, 5, device="cuda"))
    assert e.value.status == lion.ERR_UNSUPPORTED
    with pytest.raises(lion.LionError) as e:
        ssm.layernorm_fwd(torch.randn(1, 16385, device="cuda"), torch.randn(16385, device="cuda"))
    assert e.value.status == lion.ERR_UNSUPPORTED
    A, Bm = -torch.ones(8, 12, device="cuda"), torch.randn(2, 4, 1, 12, device="cuda")
    with pytest.raises(lion.LionError) as e:
        ssm.scan_fwd(x, x, A, Bm, Bm)
    assert e.value.status == lion.ERR_UNSUPPORTED
    A, Bm = -torch.ones(8, 16, device="cuda"), torch.randn(2, 4, 1, 16, device="cuda")
    ws = torch.empty(64, dtype=torch.uint8, device="cuda")
    with pytest.raises(lion.LionError) as e:   # a workspace that is too small
        ssm.scan_bwd(x, x, x, A, Bm, Bm, workspace=ws)
    assert e.value.status == lion.ERR_INVALID_ARG
    with pytest.raises(lion.LionError) as e:   # host memory
        ssm.conv_fwd(x, w.cpu())
    assert e.value.status == lion.ERR_INVALID_ARG
    for bad in (lambda: ssm.conv_fwd(x.double(), w), lambda: ssm.conv_fwd(x, w.bfloat16()),
                lambda: ssm.conv_fwd(x, w, lengths=torch.ones(2, device="cuda")),
                lambda: ssm.scan_fwd(x, x.bfloat16(), A, Bm, Bm),
                lambda: ssm.layernorm_fwd(x, w[0].bfloat16())):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: ssm.conv_fwd(x, w[:4]), lambda: ssm.conv_fwd(x.transpose(1, 2), w[:4]),
                lambda: ssm.conv_fwd(x, w, activation="relu"), lambda: ssm.conv_fwd(x.cpu(), w),
                lambda: ssm.conv_fwd(x, w, state=torch.zeros(2, 2, 8, device="cuda")),
                lambda: ssm.scan_fwd(x, x[:, :3], A, Bm, Bm), lambda: ssm.scan_fwd(x, x, A, Bm, Bm, z=x[..., :4]),
                lambda: ssm.layernorm_fwd(x.transpose(1, 2), torch.ones(4, device="cuda")),
                lambda: ssm.scan_fwd(x, x, A, Bm, Bm, h0=torch.zeros(2, 8, 8, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
