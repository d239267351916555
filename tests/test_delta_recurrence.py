"""The recurrence that the long GPU tests compare with gives what the 64-bit
reference of one head after the other gives."""
import numpy as np
import pytest
import torch

import delta_reference as ref
from delta_recurrence import recurrence


@pytest.mark.parametrize("reverse", (False, True))
@pytest.mark.parametrize("lengths,state", (((9, 4, 0), True), (None, False)))
def test_recurrence(lengths, state, reverse):
    rng = np.random.default_rng(2)
    B, L, Hk, Hv, dk, dv = 3, 9, 2, 4, 8, 5
    a = dict(q=rng.standard_normal((B, L, Hk, dk)), k=0.3 * rng.standard_normal((B, L, Hk, dk)),
             v=rng.standard_normal((B, L, Hv, dv)), g=-rng.random((B, L, Hv)), beta=0.3 * rng.random((B, L, Hv)))
    a["g"][0, 2, 1] = -2000.0   # of which e^g is 0
    h0, dout = rng.standard_normal((B, Hv, dk, dv)) if state else None, rng.standard_normal((B, L, Hv, dv))
    how = dict(scale=0.7, lengths=lengths, reverse=reverse)
    want = ref.delta(**a, h0=h0, dout=dout, **how)
    t = lambda x: None if x is None else torch.from_numpy(x)  # noqa: E731
    got = recurrence(**{x: t(y) for x, y in a.items()}, h0=t(h0), dout=t(dout), **how)
    for x in ("out", "h", "dq", "dk", "dv", "dg", "dbeta", "dh0"):
        assert np.abs(got[x].numpy() - want[x]).max() <= 1e-13 * max(1, np.abs(want[x]).max()), x
