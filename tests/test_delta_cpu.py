"""The delta rule's operators without a GPU: the C entry points refuse bad
arguments before anything launches, the size queries answer, the structures
are the header's, the autograd functions refuse second derivatives, and the
64-bit formulas that the GPU tests use agree with differences."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import delta_reference as ref
from bidirectional_masked_linear_gb300 import delta


@pytest.fixture(scope="module")
def lib():
    from bidirectional_masked_linear_gb300 import build, lion
    lion.load(build.build())
    return delta.load()


P = [4096 * (i + 1) for i in range(20)]
QK = dict(q_weight=0, k_weight=0, freqs=0, positions=0, q_token=0, k_token=0, B=1, L=4, Hq=2, Hk=2, d=16, rot=0, norm=0,
          interleaved=0, eps=1e-6, dtype=0, stream=0)
DE = dict(h0=0, lengths=0, saved=0, q_token=0, k_token=0, v_token=0, g_token=0, beta_token=0, B=1, L=4, Hk=2, Hv=4,
          dk=16, dv=16, scale=1.0, reverse=0, dtype=0, workspace=0, workspace_bytes=0, stream=0)
BASE = {
    "qknorm_fwd": ("_QKNormArgs", dict(QK, q=P[0], k=P[1], q_out=P[2], k_out=P[3])),
    "qknorm_bwd": ("_QKNormBwdArgs", dict(QK, dq_out=P[0], dk_out=P[1], q=P[2], k=P[3], dq=P[4], dk=P[5], dq_weight=0,
                                          dk_weight=0, workspace=0, workspace_bytes=0)),
    "delta_fwd": ("_DeltaArgs", dict(DE, q=P[0], k=P[1], v=P[2], g=P[3], beta=P[4], out=P[5], h_out=0)),
    "delta_bwd": ("_DeltaBwdArgs", dict(DE, dout=P[0], q=P[1], k=P[2], v=P[3], g=P[4], beta=P[5], dq=P[6], dk_out=P[7],
                                        dv_out=P[8], dg=P[9], dbeta=P[10], dh0=0)),
    "delta_step": ("_DeltaStepArgs", dict(h=P[0], q=P[1], k=P[2], v=P[3], g=P[4], beta=P[5], out=P[6], B=1, Hk=2, Hv=4,
                                          dk=16, dv=16, scale=1.0, dtype=0, stream=0)),
}


def _call(lib, name, **kw):
    struct, base = BASE[name]
    return getattr(lib, "lion_" + name)(bytes(getattr(delta, struct)(**{**base, **kw})))


@pytest.mark.parametrize("name", sorted(BASE))
def test_refusals(lib, name):
    assert getattr(lib, "lion_" + name)(None) == 1
    assert _call(lib, name) == 1   # pointers that are not device memory
    base = BASE[name][1]
    for field, value in base.items():
        if value in P:
            assert _call(lib, name, **{field: 0}) == 1, field
        elif field in ("B", "L", "Hq", "Hk", "Hv", "d", "dk", "dv"):
            assert _call(lib, name, **{field: 0}) == 1 and _call(lib, name, **{field: -8}) == 1, field
    for field, bad in (("dtype", 2), ("reverse", 2), ("interleaved", -1), ("norm", 2), ("eps", -1.0),
                       ("eps", float("nan")), ("scale", float("nan")), ("scale", float("inf")), ("q_token", 31),
                       ("k_token", -8), ("v_token", 63), ("g_token", 3), ("beta_token", 1), ("Hk", 3), ("rot", -8),
                       ("rot", 24)):
        if field in base and not (field == "Hk" and "qknorm" in name):
            assert _call(lib, name, **{field: bad}) == 1, field


def test_size_queries(lib):
    from bidirectional_masked_linear_gb300 import lion
    assert delta.qknorm_bwd_workspace_bytes(2, 3, 4, 4, 64) >= 2 * 64 * 4
    assert delta.qknorm_bwd_workspace_bytes(2, 3, 4, 4, 64, weights=False) == 0
    for d in (12, 264):
        assert delta.qknorm_bwd_workspace_bytes(2, 3, 4, 4, d) == 0
    ok = (2, 100, 2, 4, 64, 128)
    assert delta.delta_workspace_bytes(*ok) >= 2 * 4 * 4 * 3 * 2048
    assert delta.delta_saved_bytes(*ok) > delta.delta_workspace_bytes(*ok)
    assert delta.delta_saved_bytes(*ok, lion.DTYPE_FP32) > delta.delta_saved_bytes(*ok)
    assert (delta.delta_bwd_workspace_bytes(*ok, have_saved=False)
            == delta.delta_bwd_workspace_bytes(*ok) + delta.delta_saved_bytes(*ok))
    for bad in ((0, 100, 2, 4, 64, 128), (2, 0, 2, 4, 64, 128), (2, 100, 3, 4, 64, 128), (2, 100, 2, 4, 60, 128),
                (2, 100, 2, 4, 64, 136), (2 ** 30, 100, 2, 4, 64, 64), (1, 2 ** 31 - 1, 1, 1, 64, 64),
                (1, 4, 2 ** 26, 2 ** 26, 64, 64)):
        assert delta.delta_workspace_bytes(*bad) == delta.delta_saved_bytes(*bad) == 0, bad
        assert delta.delta_bwd_workspace_bytes(*bad) == 0, bad


def test_struct_layouts_match_the_header():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    txt = re.sub(r"/\*.*?\*/", "", open(os.path.join(root, "include", "lion.h")).read(), flags=re.S)
    for py, c in (("_QKNormArgs", "lion_qknorm_args"), ("_QKNormBwdArgs", "lion_qknorm_bwd_args"),
                  ("_DeltaArgs", "lion_delta_args"), ("_DeltaBwdArgs", "lion_delta_bwd_args"),
                  ("_DeltaStepArgs", "lion_delta_step_args")):
        body = re.search(r"\{([^{}]*)\}\s*" + c + ";", txt).group(1)
        names = [v.strip().lstrip("*").strip() for line in body.split(";") if line.strip()
                 for v in re.sub(r"^\s*(const\s+)?(void|float|int|long long|size_t|cudaStream_t)\b", "",
                                 line.strip()).split(",")]
        assert names == [f[0] for f in getattr(delta, py)._fields_], c
    for name in delta.EXPORTS:
        assert re.search(r"\b" + name + r"\(", txt), name


def test_arguments_are_checked():
    q, k, v = torch.zeros(2, 5, 2, 16), torch.zeros(2, 5, 2, 16), torch.zeros(2, 5, 4, 8)
    g = torch.zeros(2, 5, 4)
    with pytest.raises(ValueError, match="GPU"):
        delta.delta_fwd(q, k, v, g, g)
    with pytest.raises(TypeError):
        delta.delta_fwd(q.double(), k, v, g, g)
    for bad in (dict(k=k[:, :4]), dict(g=g[..., :3]), dict(beta=torch.zeros(2, 5, 4, 1)), dict(v=v.transpose(1, 2)),
                dict(k=k.transpose(2, 3).contiguous().transpose(2, 3)), dict(h0=torch.zeros(2, 4, 8, 16)),
                dict(lengths=torch.zeros(3, dtype=torch.int32))):
        with pytest.raises(ValueError):
            delta._delta_args(**{**dict(q=q, k=k, v=v, g=g, beta=g, h0=None, lengths=None), **bad})
    for bad in (dict(k=k.bfloat16()), dict(g=g.double()), dict(lengths=torch.zeros(2, dtype=torch.int64)),
                dict(h0=torch.zeros(2, 4, 16, 8).bfloat16())):
        with pytest.raises(TypeError):
            delta._delta_args(**{**dict(q=q, k=k, v=v, g=g, beta=g, h0=None, lengths=None), **bad})
    with pytest.raises(ValueError, match="without freqs"):
        delta._qknorm_args(q, k, None, None, None, torch.zeros(2, 5, dtype=torch.int32))
    with pytest.raises(ValueError):
        delta._qknorm_args(q, k, None, None, torch.zeros(2, 4), None)
    with pytest.raises(ValueError, match="'l2' or 'rms'"):
        delta._norm_kind("l1")


@pytest.mark.parametrize("name", ("QKNorm", "GatedDelta"))
def test_second_derivatives_are_refused(monkeypatch, name):
    if name == "QKNorm":
        monkeypatch.setattr(delta, "qknorm_fwd", lambda q, k, *a, **kw: (q ** 3, k ** 3))
        monkeypatch.setattr(delta, "qknorm_bwd",
                            lambda dq, dk, q, k, *a, **kw: delta.QKNormGrads(3 * q * q * dq, 3 * k * k * dk, None, None))
        f = lambda x: delta.QKNorm.apply(x, x.detach())[0]  # noqa: E731
    else:
        monkeypatch.setattr(delta, "delta_fwd", lambda q, *a, **kw: delta.DeltaOut(q ** 3, None, q.detach()))
        monkeypatch.setattr(delta, "delta_bwd",
                            lambda do, q, *a, **kw: delta.DeltaGrads(3 * q * q * do, *[None] * 5))
        f = lambda x: delta.GatedDelta.apply(x, *[x.detach()] * 4)  # noqa: E731
    x = torch.tensor([[1.0, 2.0]], requires_grad=True)
    g, = torch.autograd.grad(f(x).sum(), x, create_graph=True)
    assert torch.equal(g, 3 * x.detach() ** 2)
    with pytest.raises(RuntimeError, match="differentiated again"):
        (g.sum() + (x ** 2).sum()).backward()


# ------------------------------------------------------------------- formulas

def _num(f, x, at, h=1e-5):
    y = x.copy()
    y[at] = x[at] + h
    up = f(y)
    y[at] = x[at] - h
    return (up - f(y)) / (2 * h)


@pytest.mark.parametrize("kind,interleaved,rot", (("l2", False, 8), ("rms", True, 16), ("rms", False, 0)))
def test_qknorm_formulas(kind, interleaved, rot):
    rng = np.random.default_rng(3)
    x, w, dy = rng.standard_normal((2, 3, 2, 16)), 1 + 0.1 * rng.standard_normal(16), rng.standard_normal((2, 3, 2, 16))
    freqs = None if rot == 0 else 10.0 ** -np.arange(rot // 2)
    pos = np.array([[0, 1, 2], [100, 101, 7]])
    f = lambda x, w: (ref.qknorm(x, w, kind, 1e-6, freqs, pos, interleaved)["y"] * dy).sum()  # noqa: E731
    g = ref.qknorm(x, w, kind, 1e-6, freqs, pos, interleaved, dy)
    for at in ((0, 0, 0, 0), (1, 2, 1, 9), (1, 0, 0, 15)):
        assert abs(_num(lambda y: f(y, w), x, at) - g["dx"][at]) <= 1e-8
        assert abs(_num(lambda y: f(x, y), w, at[3:]) - g["dw"][at[3]]) <= 1e-8


@pytest.mark.parametrize("reverse", (False, True))
def test_delta_formulas(reverse):
    rng = np.random.default_rng(5)
    B, L, Hk, Hv, dk, dv = 2, 7, 1, 2, 4, 3
    a = dict(q=rng.standard_normal((B, L, Hk, dk)), k=0.5 * rng.standard_normal((B, L, Hk, dk)),
             v=rng.standard_normal((B, L, Hv, dv)), g=-rng.random((B, L, Hv)), beta=0.3 * rng.random((B, L, Hv)),
             h0=rng.standard_normal((B, Hv, dk, dv)))
    dout, n = rng.standard_normal((B, L, Hv, dv)), [7, 4]
    how = dict(scale=0.7, lengths=n, reverse=reverse)
    r = ref.delta(**a, **how, dout=dout)
    f = lambda **kw: (ref.delta(**{**a, **kw}, **how)["out"] * dout).sum()  # noqa: E731
    for x, dx in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("g", "dg"), ("beta", "dbeta"), ("h0", "dh0")):
        for _ in range(4):
            at = tuple(rng.integers(0, s) for s in a[x].shape)
            assert abs(_num(lambda y: f(**{x: y}), a[x], at) - r[dx][at]) <= 1e-7, (x, at)
    # a token after the others
    o, S = ref.step(r["h"][0, 0], a["q"][0, 0, 0], a["k"][0, 0, 0], a["v"][0, 0, 0], -0.1, 0.2, 0.7)
    more = {x: np.concatenate([y[:1], y[:1, :1]], 1) if not reverse else np.concatenate([y[:1, :1], y[:1]], 1)
            for x, y in a.items() if x != "h0"}
    at = 0 if reverse else L
    more["g"][0, at, 0], more["beta"][0, at, 0] = -0.1, 0.2
    w = ref.delta(**more, h0=a["h0"][:1], scale=0.7, reverse=reverse)
    assert np.allclose(w["out"][0, at, 0], o) and np.allclose(w["h"][0, 0], S)
