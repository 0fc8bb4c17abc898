"""The update of the example of a memory block trained on rewards: every weight moves against its gradient."""
import os
import sys

import pytest
import torch

from conftest import ROOT
from gpu_util import require_gpu

sys.path.insert(0, os.path.join(ROOT, "examples"))
pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    require_gpu()


def test_every_weight_moves_against_its_gradient():
    import reward_memory as ex
    V, T, lr = 90, 150, 0.02
    block = ex.Block(V, base_rows=211, seed=2, dtype=torch.float32)
    batch = ex.batch(V, T, 3, 5)
    weights = {**block.proj, **block.norm, "table": block.table}
    before = {n: w.clone() for n, w in weights.items()}
    _, grads = block.gradients(*batch)
    rows, d = grads.pop("table")
    grads["table"] = torch.zeros_like(block.table).index_add_(0, rows.clamp_min(0).long(), d)
    block.step(*batch, lr=lr)
    for n, w in weights.items():
        g, size = grads[n].double(), float(before[n].double().norm())
        step = w.double() - before[n].double()
        want = -lr * size / float(g.norm()) * g
        # (an fp32 weight's rounding, 2^-24, and the gradient's own from one call to the next: none)
        assert float((step - want).norm()) <= 1e-5 * size, n
        assert float((step * g).sum()) < 0.0, n
