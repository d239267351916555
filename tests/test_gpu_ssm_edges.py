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
