"""The state space block where it is easily wrong: lanes that meet in shared
memory, cut sequences, factors that overflow, empty sequences, sizes past 32
bits.  Bounds as in test_gpu_ssm.py."""
import numpy as np
import pytest
import torch

import ssm_reference as ref
from bidirectional_masked_linear_gb300 import ssm
from test_gpu_ssm import E, T, _check, _f64, _scan_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bidirectional_masked_linear_gb300 import build, lion
    lion.load(build.build())


@pytest.mark.parametrize("dtype", ("bf16", "fp32"))
@pytest.mark.parametrize("N", (8, 16, 32, 64))
def test_equal_sequences_give_equal_bits(N, dtype):
    """The same sequence many times over, with every SM's slots taken: a lane that overwrote what another has yet to
    read would show in some of them."""
    B, L, D = 48, 45, 520
    a, dout = _scan_inputs(1, L, D, N, 1, dtype, True, True, True, True, True, seed=N)
    per = ("u", "dt", "Bm", "Cm", "z", "h0")
    dev = {k: v.expand(B, *v.shape[1:]).contiguous().cuda() if k in per else v.cuda() for k, v in a.items()}
    f = ssm.scan_fwd(**dev, return_state=True, save_states=True)
    g = ssm.scan_bwd(dout.expand(B, L, D).contiguous().cuda(), **dev, states=f.states)
    for name, t in (("out", f.out), ("h", f.h), ("states", f.states), ("du", g.du), ("ddt", g.ddt), ("dB", g.dB),
                    ("dC", g.dC), ("dz", g.dz), ("dh0", g.dh0)):
        assert torch.equal(t, t[:1].expand_as(t)), name


# ------------------------------------------------------ factors that overflow

def _growth(L=1600, D=8, N=16):
    """Two adjacent tokens that each multiply a state by exp(64): their product, the factor of the segment that they
    lie in, is past fp32, what they make of a state of 1e-36 is not."""
    dt, A = torch.zeros(1, L, D, device="cuda"), torch.full((D, N), 64.0, device="cuda")
    dt[:, 200:202] = 1.0
    return dt, A, torch.ones(1, L, N, device="cuda"), 1e-36 * np.exp(128.0)


# two exponents of 92 in base 2 and one of 185, each rounded and each error a factor of ln 2
GROWTH_TOL = 512 * E


def test_scan_chain_of_a_tiny_state():
    dt, A, ones, want = _growth()
    h0 = torch.full((1, 8, 16), 1e-36, device="cuda")
    f = ssm.scan_fwd(torch.zeros_like(dt), dt, A, ones, ones, dt_softplus=False, h0=h0, return_state=True)
    assert float((f.h / want - 1).abs().max()) <= GROWTH_TOL
    assert float((f.out[:, 201:] / (16 * want) - 1).abs().max()) <= GROWTH_TOL


def test_scan_chain_of_a_tiny_gradient():
    dt, A, ones, want = _growth()
    u, dout = torch.zeros_like(dt), torch.zeros_like(dt)
    u[:, 0] = 1.0   # its step is 0: it adds nothing, but its step's gradient is u sum_n G B
    dout[:, -1] = 1e-36
    h0 = torch.zeros(1, 8, 16, device="cuda")
    g = ssm.scan_bwd(dout, u, dt, A, ones, ones, dt_softplus=False, h0=h0)
    assert float((g.dh0 / want - 1).abs().max()) <= GROWTH_TOL
    assert float((g.ddt[:, 0] / (16 * want) - 1).abs().max()) <= GROWTH_TOL
    for t in (g.du[:, :200], g.du[:, 202:], g.ddt[:, 1:], g.dA, g.dB, g.dC):
        assert bool((t == 0).all())


@pytest.mark.parametrize("sign", (1, -1))
def test_scan_chain_past_overflow(sign):
    """Segments whose factor overflows: of a state that is 0 they make 0, of any other what the walk does, inf."""
    L, D, N = 1600, 8, 16
    u, dt = torch.zeros(1, L, D, device="cuda"), torch.ones(1, L, D, device="cuda")
    u[:, -20:] = sign
    A, ones = torch.full((D, N), 2.0, device="cuda"), torch.ones(1, L, N, device="cuda")
    f = ssm.scan_fwd(u, dt, A, ones, ones, dt_softplus=False, return_state=True)
    want = sign * sum(np.exp(2.0 * k) for k in range(20))
    assert bool((f.out[:, :-20] == 0).all())
    assert float((f.h / want - 1).abs().max()) <= 20 * 16 * E
    dout = torch.zeros_like(u)
    dout[:, :20] = sign
    h0 = torch.zeros(1, D, N, device="cuda")
    g = ssm.scan_bwd(dout, u, dt, A, ones, ones, dt_softplus=False, h0=h0)
    want = sign * sum(np.exp(2.0 * (k + 1)) for k in range(20))
    assert float((g.dh0 / want - 1).abs().max()) <= 21 * 16 * E
    assert bool((g.du[:, 20:] == 0).all())
    f = ssm.scan_fwd(torch.zeros_like(u), dt, A, ones, ones, dt_softplus=False, h0=sign * torch.ones_like(h0),
                     return_state=True)
    assert bool((f.h == sign * float("inf")).all())


# ------------------------------------------------------------ empty sequences

@pytest.mark.parametrize("dtype", ("bf16", "fp32"))
@pytest.mark.parametrize("bad", (float("nan"), float("inf")))
def test_conv_gradients_of_an_empty_sequence(bad, dtype):
    """The state before a sequence without tokens reaches no output, whatever it holds."""
    B, L, D, K = 3, 9, 20, 4
    x, dy = (torch.randn(B, L, D, device="cuda").to(T[dtype]) for _ in range(2))
    w, b = torch.randn(D, K, device="cuda"), torch.randn(D, device="cuda")
    st = torch.randn(B, K - 1, D, device="cuda").to(T[dtype])
    lens = torch.tensor([9, 0, 2], dtype=torch.int32, device="cuda")
    want = ssm.conv_bwd(dy, x, w, b, state=st, lengths=lens)
    st[1] = bad
    got = ssm.conv_bwd(dy, x, w, b, state=st, lengths=lens)
    assert all(torch.equal(p, s) for p, s in zip(got, want))
    assert bool((got.dstate[1] == 0).all())


# ---------------------------------------------------- states that forget at once

@pytest.mark.parametrize("dtype", ("bf16", "fp32"))
@pytest.mark.parametrize("L,D,reverse", ((20, 33, False), (20, 33, True), (600, 24, False), (600, 24, True)))
def test_scan_of_states_without_memory(L, D, reverse, dtype):
    """A = -inf keeps nothing (exp(delta A) = 0), and the tokens that a sequence does not have change nothing."""
    N, n = 16, [L, L // 3 + 1]
    a, dout = _scan_inputs(2, L, D, N, 1, dtype, True, True, True, True, True, seed=L)
    a["A"][:, 1::3] = -float("inf")
    lens = torch.tensor(n, dtype=torch.int32)
    A64 = {k: _f64(v) for k, v in a.items()}
    r = ref.scan(**A64, lengths=n, reverse=reverse)
    m = ref.scan(**A64, lengths=n, reverse=reverse, absolute=True)
    dev = {k: v.cuda() for k, v in a.items()}
    how = dict(lengths=lens.cuda(), reverse=reverse)
    f = ssm.scan_fwd(**dev, **how, return_state=True, save_states=True)
    tol = E * (64 + 16 * L + 2 * (N + D + 2 * L))
    _check("out", f.out, r["out"], tol * m["out"])
    _check("h", f.h, r["h"], tol * m["h"])
    # the gradients are those of a decay that is as good as none
    g = ssm.scan_bwd(dout.cuda(), **dev, **how, states=f.states)
    dev["A"].clamp_(min=-1e30)
    want = ssm.scan_bwd(dout.cuda(), **dev, **how, states=f.states)
    assert all(torch.equal(p, s) for p, s in zip(g, want))
    # one token after these
    one = {k: dev[k][:, 0].contiguous() for k in ("u", "dt", "Bm", "Cm", "z")}
    rest = {k: dev[k] for k in ("Dskip", "dt_bias")}
    h1, h2 = f.h.clone(), f.h.clone()
    assert torch.equal(ssm.scan_step(h1, **one, A=a["A"].cuda(), **rest), ssm.scan_step(h2, **one, A=dev["A"], **rest))
    assert torch.equal(h1, h2)


# ------------------------------------------------------- sizes past 32 bits

def _room(gigabytes):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gigabytes * 1e9:
        pytest.skip("not enough free memory")


def test_conv_of_two_to_the_31_sequences():
    """As many runs as the calls take, one less than 2^31: the gradients' walk over them ends."""
    _room(40)
    B = 2 ** 31 - 1
    x = torch.zeros(B, 1, 1, dtype=torch.bfloat16, device="cuda")
    x[-1000:] = 1.0
    dy = torch.ones_like(x)
    w = torch.tensor([[0.5, -0.75]], device="cuda")
    y = ssm.conv_fwd(x, w, activation="none")
    assert bool((y[-1000:] == -0.75).all()) and float(y[:-1000].float().abs().max()) == 0
    del y
    g = ssm.conv_bwd(dy, x, w, activation="none")
    assert float(g.dx.min()) == float(g.dx.max()) == -0.75
    assert g.dweight.tolist() == [[0.0, 1000.0]]


def test_layernorm_of_two_to_the_31_rows():
    _room(40)
    rows = 2 ** 31 - 1
    x = torch.ones(rows, 1, dtype=torch.bfloat16, device="cuda")
    w, b = torch.ones(1, device="cuda"), torch.full((1,), 0.25, device="cuda")
    y, mean, rstd = ssm.layernorm_fwd(x, w, b, 1.0, save_stats=True)   # x - mean is 0
    assert float(y.min()) == float(y.max()) == 0.25
    del y
    x[:-1000] = 0.0   # as dy
    dx, dw, db = ssm.layernorm_bwd(x, x, w, torch.zeros_like(mean), rstd)
    assert bool((dx[-1000:] == -1).all())   # xh = 1 there with a mean of 0: 1 - 1 - 1 * 1
    assert float(dx[:-1000].min()) == float(dx[:-1000].max()) == 0
    assert dw.tolist() == db.tolist() == [1000.0]


def test_scan_step_of_two_to_the_34_states():
    """More groups of four states than 32 bits count: each channel steps once."""
    _room(160)
    D, N = 2 ** 28 + 40, 64
    A = torch.full((D, N), -1.0, device="cuda")
    h = torch.ones(1, D, N, device="cuda")
    u, dt = torch.zeros(1, D, dtype=torch.bfloat16, device="cuda"), torch.ones(1, D, dtype=torch.bfloat16, device="cuda")
    Bm = torch.ones(1, N, dtype=torch.bfloat16, device="cuda")
    y = ssm.scan_step(h, u, dt, A, Bm, Bm, dt_softplus=False)
    want = float(np.exp(-1.0))
    assert abs(float(h.min()) / want - 1) <= 64 * E and abs(float(h.max()) / want - 1) <= 64 * E
    assert float(y.min()) == float(y.max()) == float(torch.tensor(64 * want).bfloat16())


def test_conv_in_place_is_refused():
    """A run would read the outputs of the one before it."""
    from bidirectional_masked_linear_gb300 import lion
    x, w = torch.randn(2, 300, 64, device="cuda"), torch.randn(64, 4, device="cuda")
    before = x.clone()
    with pytest.raises(lion.LionError) as e:
        ssm.conv_fwd(x, w, out=x)
    assert e.value.status == lion.ERR_INVALID_ARG
    torch.cuda.synchronize()
    assert torch.equal(x, before)
    y = torch.empty_like(x)
    assert ssm.conv_fwd(x, w, out=y) is y and torch.equal(y, ssm.conv_fwd(x, w))
