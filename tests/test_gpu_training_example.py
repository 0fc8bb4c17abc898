"""The training example: the operators together learn, and decoding agrees with prefill."""
import os
import sys

import pytest
import torch

from conftest import ROOT
from gpu_util import DEV, require_gpu

sys.path.insert(0, os.path.join(ROOT, "examples"))
pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    require_gpu()


def test_the_memory_learns_its_teacher():
    import distill_memory as ex
    losses = ex.main(steps=40)
    assert losses[-1] < 0.5 * losses[0], losses[::10]


def test_decoding_agrees_with_prefill():
    """The same positions in one scan and one at a time: equal up to the bf16 roundings of the dense products."""
    import distill_memory as ex
    memory = ex.Memory(500, seed=3)
    ids, _, _, _ = ex.batch(500, 40, 1, 4)
    cu = torch.tensor([0, 40], device=DEV)
    want = memory.forward(ids, cu)[-1].float()
    got = memory.decode(ids).float()
    # products of other shapes may add up in another order: inputs x, g and y move by a bf16 step (2^-8)
    assert (got - want).abs().max() <= 2.0 ** -6 * want.abs().max()
    assert memory.status.item() == 0
