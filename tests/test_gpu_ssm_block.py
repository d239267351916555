"""The small model of examples/ssm_block.py: its ops learn together, and a
prompt followed by single tokens gives the whole sequence's logits."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bidirectional_masked_linear_gb300 import build, lion
    lion.load(build.build())
    import ssm_block
    return ssm_block


@pytest.mark.parametrize("directions", (1, 2))
def test_learns(example, directions):
    torch.manual_seed(0)
    losses = example.train(example.Model(directions=directions).cuda(), 100)
    # a uniform guess over 16 tokens costs 2.77
    assert losses[0] > 2.3 and sum(losses[-5:]) / 5 < 0.6 * losses[0]


def test_prompt_and_steps_give_the_whole(example):
    torch.manual_seed(1)
    assert example.serve_error(example.Model().cuda()) <= 1e-4   # fp32 products in another order, two blocks


def test_ragged_batch_is_its_sequences(example):
    """A padded batch of ragged sequences gives each sequence's own logits."""
    torch.manual_seed(2)
    m = example.Model(directions=2).cuda()
    t = torch.randint(0, 16, (3, 50), device="cuda")
    n = [50, 1, 23]
    with torch.no_grad():
        whole = m(t, torch.tensor(n, dtype=torch.int32, device="cuda"))
        for b, k in enumerate(n):
            alone = m(t[b:b + 1, :k].contiguous())
            assert float((whole[b:b + 1, :k] - alone).abs().max()) <= 1e-4 * float(alone.abs().max())
