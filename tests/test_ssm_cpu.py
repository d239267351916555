"""The state space block without a GPU: its C entry points refuse bad
arguments before anything launches, the workspace queries answer, and the
64-bit gradient formulas that the GPU tests use agree with differences."""
import ctypes

import numpy as np
import pytest

import ssm_reference as ref


@pytest.fixture(scope="module")
def ssm():
    from bidirectional_masked_linear_gb300 import build, lion, ssm
    lion.load(build.build())
    ssm.load()
    return ssm


BASE = {
    "layernorm_fwd": ("_NormArgs", dict(x=4096, weight=8192, bias=0, y=12288, mean=0, rstd=0, x_row=0, rows=2, cols=8,
                                        eps=1e-5, dtype=0, stream=0)),
    "layernorm_bwd": ("_NormBwdArgs", dict(dy=4096, x=8192, weight=12288, mean=16384, rstd=20480, dx=24576,
                                           dweight=28672, dbias=0, x_row=0, rows=2, cols=8, dtype=0, workspace=0,
                                           workspace_bytes=0, stream=0)),
    "conv_fwd": ("_ConvArgs", dict(x=4096, weight=8192, bias=0, state=0, lengths=0, y=12288, state_out=0, x_token=0,
                                   B=1, L=4, D=8, K=4, act=1, reverse=0, dtype=0, stream=0)),
    "conv_bwd": ("_ConvBwdArgs", dict(dy=4096, x=8192, weight=12288, bias=0, state=0, lengths=0, dx=16384,
                                      dweight=20480, dbias=0, dstate=0, x_token=0, B=1, L=4, D=8, K=4, act=1,
                                      reverse=0, dtype=0, workspace=0, workspace_bytes=0, stream=0)),
    "scan_fwd": ("_ScanArgs", dict(u=4096, dt=8192, A=12288, Bm=16384, Cm=20480, Dskip=0, z=0, dt_bias=0, h0=0,
                                   lengths=0, out=24576, h_out=0, states=0, u_token=0, dt_token=0, z_token=0,
                                   b_token=0, c_token=0, B=1, L=4, D=8, N=16, G=1, dt_softplus=1, reverse=0, dtype=0,
                                   workspace=0, workspace_bytes=0, stream=0)),
    "scan_bwd": ("_ScanBwdArgs", dict(dout=4096, u=8192, dt=12288, A=16384, Bm=20480, Cm=24576, Dskip=0, z=0,
                                      dt_bias=0, h0=0, lengths=0, states=0, du=28672, ddt=32768, dA=36864, dB=40960,
                                      dC=45056, dDskip=0, dz=0, ddt_bias=0, dh0=0, u_token=0, dt_token=0, z_token=0,
                                      b_token=0, c_token=0, B=1, L=4, D=8, N=16, G=1, dt_softplus=1, reverse=0,
                                      dtype=0, workspace=0, workspace_bytes=0, stream=0)),
    "scan_step": ("_ScanStepArgs", dict(h=4096, u=8192, dt=12288, A=16384, Bm=20480, Cm=24576, Dskip=0, z=0,
                                        dt_bias=0, out=28672, B=1, D=8, N=16, G=1, dt_softplus=1, dtype=0, stream=0)),
}
NEEDED = {
    "layernorm_fwd": ("x", "weight", "y"), "layernorm_bwd": ("dy", "x", "weight", "mean", "rstd", "dx", "dweight"),
    "conv_fwd": ("x", "weight", "y"), "conv_bwd": ("dy", "x", "weight", "dx", "dweight"),
    "scan_fwd": ("u", "dt", "A", "Bm", "Cm", "out"),
    "scan_bwd": ("dout", "u", "dt", "A", "Bm", "Cm", "du", "ddt", "dA", "dB", "dC"),
    "scan_step": ("h", "u", "dt", "A", "Bm", "Cm", "out"),
}


def _call(ssm, name, **kw):
    struct, base = BASE[name]
    return getattr(ssm.load(), "lion_" + name)(bytes(getattr(ssm, struct)(**{**base, **kw})))


@pytest.mark.parametrize("name", sorted(BASE))
def test_refusals(ssm, name):
    assert getattr(ssm.load(), "lion_" + name)(None) == 1
    assert _call(ssm, name) == 1   # pointers that are not device memory
    for field in NEEDED[name]:
        assert _call(ssm, name, **{field: 0}) == 1, field
    base = BASE[name][1]
    for field in ("B", "L", "D", "rows", "cols", "N", "G", "K"):
        if field in base:
            assert _call(ssm, name, **{field: 0}) == 1, field
            assert _call(ssm, name, **{field: -1}) == 1, field
    for field, bad in (("dtype", 2), ("act", 2), ("reverse", 2), ("dt_softplus", -1), ("x_row", 7), ("x_token", 7),
                       ("u_token", 7), ("z_token", -8), ("b_token", 15)):
        if field in base:
            assert _call(ssm, name, **{field: bad}) == 1, field
    if "G" in base:
        assert _call(ssm, name, G=3) == 1   # does not divide D
    if name == "layernorm_fwd":
        assert _call(ssm, name, eps=-1.0) == 1
        assert _call(ssm, name, eps=float("nan")) == 1
        assert _call(ssm, name, mean=16384) == 1   # without rstd


def test_conv_step_refusals(ssm):
    f = ssm.load().lion_conv_step
    good = [4096, 8192, 12288, None, 16384, 1, 8, 4, 1, 0, None]
    assert f(*good) == 1   # not device memory
    for k, bad in ((0, None), (1, None), (2, None), (4, None), (5, 0), (6, 0), (7, 0), (8, 2), (9, 2)):
        assert f(*(good[:k] + [bad] + good[k + 1:])) == 1


def test_workspace_queries(ssm):
    assert ssm.layernorm_bwd_workspace_bytes(10, 64) >= 2 * 64 * 4
    assert ssm.layernorm_bwd_workspace_bytes(0, 64) == 0
    assert ssm.layernorm_bwd_workspace_bytes(1, 16385) == 0
    assert ssm.conv_bwd_workspace_bytes(1, 4, 8, 4) >= 8 * 5 * 4
    assert ssm.conv_bwd_workspace_bytes(1, 4, 8, 5) == 0
    assert ssm.scan_bwd_workspace_bytes(1, 40, 8, 16) >= (40 * 32 + 8 * 18) * 4
    # without the forward's states: room to compute them
    assert (ssm.scan_bwd_workspace_bytes(1, 40, 8, 16, 1, False)
            >= ssm.scan_bwd_workspace_bytes(1, 40, 8, 16) + 3 * 8 * 16 * 4)
    assert ssm.scan_bwd_workspace_bytes(1, 40, 8, 12) == 0
    assert ssm.scan_workspace_bytes(1, 40, 9, 16, 2) == 0
    # a long sequence of few channels is cut into segments
    assert ssm.scan_workspace_bytes(1, 24337, 64, 16) > 0


def test_struct_layouts_match_the_header(ssm):
    """Field names and order of the ctypes structures are the header's."""
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    txt = re.sub(r"/\*.*?\*/", "", open(os.path.join(root, "include", "lion.h")).read(), flags=re.S)
    for py, c in (("_NormArgs", "lion_layernorm_args"), ("_NormBwdArgs", "lion_layernorm_bwd_args"),
                  ("_ConvArgs", "lion_conv_args"), ("_ConvBwdArgs", "lion_conv_bwd_args"),
                  ("_ScanArgs", "lion_scan_args"), ("_ScanBwdArgs", "lion_scan_bwd_args"),
                  ("_ScanStepArgs", "lion_scan_step_args")):
        body = re.search(r"\{([^{}]*)\}\s*" + c + ";", txt).group(1)
        names = [v.strip().lstrip("*").strip() for line in body.split(";") if line.strip()
                 for v in re.sub(r"^\s*(const\s+)?(void|float|int|long long|size_t|cudaStream_t)\b", "",
                                 line.strip()).split(",")]
        assert names == [f[0] for f in getattr(ssm, py)._fields_], c


# ------------------------------------------- the formulas against differences

def _differences(f, x, dy, eps=1e-5):
    d = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        old = x[i]
        x[i] = old + eps
        up = (f() * dy).sum()
        x[i] = old - eps
        d[i] = (up - (f() * dy).sum()) / (2 * eps)
        x[i] = old
    return d


def _close(got, want):
    # central differences: eps^2 |f'''| / 6 + 2^-53 |f| / eps, far below 1e-7 of the largest
    assert np.max(np.abs(got - want)) <= 1e-7 * max(1.0, np.max(np.abs(want)))


@pytest.mark.parametrize("reverse", (False, True))
@pytest.mark.parametrize("softplus", (False, True))
def test_scan_formulas(reverse, softplus):
    g = np.random.default_rng(1)
    B, L, D, N, G = 2, 5, 4, 3, 2
    a = dict(u=g.normal(size=(B, L, D)), dt=g.normal(size=(B, L, D)), A=-g.uniform(0.2, 2, (D, N)),
             Bm=g.normal(size=(B, L, G, N)), Cm=g.normal(size=(B, L, G, N)), Dskip=g.normal(size=D),
             z=g.normal(size=(B, L, D)), dt_bias=g.normal(size=D), h0=g.normal(size=(B, D, N)))
    how = dict(dt_softplus=softplus, lengths=[5, 2], reverse=reverse)
    dout = g.normal(size=(B, L, D))
    r = ref.scan(**a, **how, dout=dout)
    for name, grad in (("u", "du"), ("dt", "ddt"), ("A", "dA"), ("Bm", "dB"), ("Cm", "dC"), ("Dskip", "dDskip"),
                       ("z", "dz"), ("dt_bias", "ddt_bias"), ("h0", "dh0")):
        _close(r[grad], _differences(lambda: ref.scan(**a, **how)["out"], a[name], dout))


@pytest.mark.parametrize("reverse", (False, True))
@pytest.mark.parametrize("act", (False, True))
def test_conv_formulas(reverse, act):
    g = np.random.default_rng(2)
    B, L, D, K = 2, 5, 3, 4
    a = dict(x=g.normal(size=(B, L, D)), w=g.normal(size=(D, K)), b=g.normal(size=D),
             state=g.normal(size=(B, K - 1, D)))
    how = dict(act=act, lengths=[5, 2], reverse=reverse)
    dy = g.normal(size=(B, L, D))
    r = ref.conv(**a, **how, dy=dy)
    for name, grad in (("x", "dx"), ("w", "dweight"), ("b", "dbias"), ("state", "dstate")):
        _close(r[grad], _differences(lambda: ref.conv(**a, **how)["y"], a[name], dy))


def test_layernorm_formulas():
    g = np.random.default_rng(3)
    x, w, b, dy = g.normal(size=(4, 6)), g.normal(size=6), g.normal(size=6), g.normal(size=(4, 6))
    r = ref.layernorm(x, w, b, 1e-5, dy)
    _close(r["dx"], _differences(lambda: ref.layernorm(x, w, b, 1e-5)["y"], x, dy))
    _close(r["dweight"], _differences(lambda: ref.layernorm(x, w, b, 1e-5)["y"], w, dy))
    _close(r["dbias"], _differences(lambda: ref.layernorm(x, w, b, 1e-5)["y"], b, dy))
