"""The training example at image positions: decoding one at a time agrees with the scan of a prompt."""
import os
import sys

import pytest
import torch

import hashed_gram_conditional_gb300 as eg
from conftest import ROOT
from gpu_util import DEV, require_gpu

sys.path.insert(0, os.path.join(ROOT, "examples"))
pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    require_gpu()


def test_decoding_agrees_with_prefill_at_image_positions():
    """They hold the state and give no logits, and the positions after them start from the state before them."""
    import distill_memory as ex
    memory = ex.Memory(500, seed=3)
    ids, _, _, _ = ex.batch(500, 40, 1, 4)
    image = [0, 7, 8, 9, 25, 39]
    ids[image] = eg.DEAD
    want = memory.forward(ids, torch.tensor([0, 40], device=DEV))[-1].float()
    got = memory.decode(ids).float()
    assert (want[image] == 0).all() and (got[image] == 0).all()
    # products of other shapes may add up in another order: inputs x, g and y move by a bf16 step (2^-8)
    assert (got - want).abs().max() <= 2.0 ** -6 * want.abs().max()
    assert memory.status.item() == 0
