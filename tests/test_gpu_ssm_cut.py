"""The selective scan where its plan cuts sequences into segments and channels
into blocks: values and gradients against the 64-bit reference, and gradients
past 2^31 values.  Bounds as in test_gpu_ssm.py."""
import pytest
import torch

import test_gpu_ssm as base
from bidirectional_masked_linear_gb300 import ssm
from test_scan_plan import plans

CUT = [  # B, L, D, N, G, lengths, options off, reverse; at least this many blocks and segments of the gradients
    ((1, 1600, 24, 16, 1, None, "", False), 1, 17),      # more segments than the chain reads at a time
    ((1, 1600, 24, 32, 1, (1111,), "skip", True), 1, 17),
    ((2, 450, 330, 64, 2, (450, 161), "", True), 2, 2),
    ((1, 500, 200, 32, 2, None, "", False), 2, 2),
    ((2, 400, 300, 8, 1, (400, 90), "gate", False), 2, 2),
    ((1, 500, 600, 16, 2, None, "state", True), 2, 2),
]


def test_the_cases_are_cut(tmp_path):
    """By today's plan: a change of it that leaves these whole has to bring others."""
    got = plans(tmp_path, [c[:5] + (c[5] is not None,) for c, _, _ in CUT])
    for (c, blocks, segments), both in zip(CUT, got):
        for nblk, nseg, _, _ in both:
            assert nblk >= blocks and nseg >= segments, c


@pytest.fixture
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bidirectional_masked_linear_gb300 import build, lion
    lion.load(build.build())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ("bf16", "fp32"))
@pytest.mark.parametrize("case", [c for c, _, _ in CUT])
def test_scan_of_cut_sequences(gpu, case, dtype):
    base.test_scan(*case, dtype)


@pytest.mark.gpu
def test_conv_gradients_past_32_bits(gpu):
    """The last of the sequences against the same sequence alone, bit for bit; the weight's gradient of a loss that
    sees only the last one too."""
    B, L, D = 9, 120000, 2048
    x = torch.empty(B, L, D, dtype=torch.bfloat16, device="cuda").normal_()
    dy = torch.zeros_like(x)
    dy[-1].normal_()
    w, b = torch.randn(D, 4, device="cuda"), torch.randn(D, device="cuda")
    g, alone = ssm.conv_bwd(dy, x, w, b), ssm.conv_bwd(dy[-1:], x[-1:], w, b)
    assert torch.equal(g.dx[-1:], alone.dx) and float(g.dx[:-1].abs().max()) == 0
    # sums of L products in two orders
    xs, ds = x[-1].float().abs(), dy[-1].float().abs()
    most = 1.1 * torch.stack([(xs[:L - 3 + k] * ds[3 - k:]).sum(0) for k in range(4)], 1)
    assert bool(((g.dweight - alone.dweight).abs() <= 2 * base.E * L * most).all())
    assert bool(((g.dbias - alone.dbias).abs() <= 2.2 * base.E * L * ds.sum(0)).all())


@pytest.mark.gpu
def test_scan_gradients_past_32_bits(gpu):
    """The last sequence against the same sequence alone (cut differently)."""
    B, L, D, N = 3, 360000, 2048, 8
    big = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda").normal_()  # noqa: E731
    u, dt, Bm, Cm, dout = big(B, L, D), big(B, L, D).mul_(0.1), big(B, L, N), big(B, L, N), big(B, L, D)
    A, h0 = -(0.5 + torch.rand(D, N, device="cuda")), torch.zeros(B, D, N, device="cuda")
    g = ssm.scan_bwd(dout, u, dt, A, Bm, Cm, h0=h0)
    last = ssm.scan_bwd(dout[-1:], u[-1:], dt[-1:], A, Bm[-1:], Cm[-1:], h0=h0[-1:])
    assert float((g.dh0[-1:] - last.dh0).abs().max()) <= 1e-5 * float(last.dh0.abs().max())
    # states and their gradients of order ten that forget within some ten tokens: a cut moves the fp32 sums by a few
    # roundings (1e-5 of their terms, which for dB and dC are 2048), the results by one bfloat16 unit
    for name, most in (("du", 1e-3), ("ddt", 1e-3), ("dB", 0.1), ("dC", 0.1)):
        for lo in range(0, L, 40000):
            p, q = (getattr(r, name)[-1, lo:lo + 40000].float() for r in (g, last))
            assert bool(((p - q).abs() <= 2.0 ** -7 * q.abs() + most).all()), name
