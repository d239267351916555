"""Turns of the norms' outputs by frequencies above and below 0.

The bound is the norms' own: the angle, its cosine and sine and the turn are 8 e
off of the pair's two values, e = 2^-24.  Heads of length 1 and eps = 0 leave
nothing else: 1 / length is 1."""
import numpy as np
import pytest
import torch

from bidirectional_masked_linear_gb300 import delta, lion
from test_gpu_ssm import E, _check, _f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bidirectional_masked_linear_gb300 import build
    lion.load(build.build())


@pytest.mark.parametrize("sign", (1, -1))
@pytest.mark.parametrize("interleaved", (False, True))
def test_turns_from_far_positions(interleaved, sign):
    """Both signs keep 32 bits of a turn's fraction at positions of 31 bits."""
    d, L = 256, 500
    gen = torch.Generator().manual_seed(4)
    f = sign * 10.0 ** (-7 * torch.rand(d // 2, generator=gen))
    pos = 2 ** 31 - 1 - torch.arange(L)
    q = torch.zeros(1, L, 1, d)
    first = slice(0, d, 2) if interleaved else slice(0, d // 2)
    where = torch.randint(0, d // 2, (L, 4), generator=gen)
    for t in range(L):   # four values of 1/2 or, where two fell on one place, fewer: of length 1 all the same
        places = where[t].unique()
        q[0, t, 0, first][places[:4] if len(places) == 4 else places[:1]] = 0.5 if len(places) == 4 else 1.0
    y, _ = delta.qknorm_fwd(q.cuda(), q.cuda(), eps=0.0, freqs=f.cuda(), positions=pos.int()[None].cuda(),
                            interleaved=interleaved)
    a = pos.numpy()[:, None].astype(np.longdouble) * _f64(f)
    x = _f64(q)[0, :, 0, first]
    want, size = np.zeros((1, L, 1, d)), np.zeros((1, L, 1, d))
    second = slice(1, d, 2) if interleaved else slice(d // 2, d)
    want[0, :, 0, first], want[0, :, 0, second] = x * np.cos(a), x * np.sin(a)
    size[0, :, 0, first] = size[0, :, 0, second] = x
    _check("y", y, want, 8 * E * size)
