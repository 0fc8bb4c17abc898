"""The example of a memory block trained on rewards: it runs, its gradients are those of the whole model by automatic
differentiation in 64 bits, and decoding agrees with prefill."""
import os
import sys

import pytest
import torch

import hashed_gram_conditional_gb300 as eg
from conftest import ROOT
from gpu_util import DEV, require_gpu
from oracle import blocks as OB

sys.path.insert(0, os.path.join(ROOT, "examples"))
pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    require_gpu()


def test_it_runs():
    import reward_memory as ex
    losses = ex.main(steps=4, vocab=200, tokens=300)
    assert len(losses) == 4 and all(x == x for x in losses)


def test_gradients_of_the_whole_model():
    import reward_memory as ex
    V, T = 90, 150
    block = ex.Block(V, base_rows=211, seed=2, dtype=torch.float32)
    ids, cu, sampled, advantage = ex.batch(V, T, 3, 5)
    ids[40:44] = eg.DEAD  # image positions
    old = block.logp(ids, cu, sampled)
    ref = old + 0.2 * torch.randn(T, device=DEV, generator=torch.Generator(DEV).manual_seed(1))
    # the present weights are others than those that the tokens were sampled with; ratios stay off the clip's edges
    for w in block.proj.values():
        w.mul_(1.05)
    loss, grads = block.gradients(ids, cu, sampled, advantage, old_logp=old, ref_logp=ref, kl=0.1)
    assert block.status.item() == 0

    rows, mask = block.rows_of(ids, cu)
    leaf = {n: w.double().requires_grad_() for n, w in {**block.proj, **block.norm, "table": block.table}.items()}
    ok = rows >= 0
    h0 = (leaf["table"][rows.clamp_min(0).long()] * ok[..., None]).view(T, -1)
    x0 = OB.norm_add(h0, leaf["first"])[0]
    p = {n: x0 @ leaf[n] for n in ("q", "k", "v", "z", "g", "b")}
    qn, kn = (OB.norm_add(p[n], block.unit.double(), groups=ex.KEYS)[0] for n in ("q", "k"))
    y = OB.delta(qn, kn, p["v"], p["g"], p["b"], cu.tolist(), ex.KEYS, ex.DIM ** -0.5, mask.tolist())["y"]
    h1 = OB.norm_add(y, leaf["head"], p["z"], h0, leaf["scale"], ex.HEADS)[0]
    logits = OB.norm_next(h1, leaf["last"])[0] @ leaf["out"]
    weight = (mask == 0).double() / T
    want = OB.policy(logits, sampled, advantage.double(), old.double(), ref.double(), (0.2, 0.2), 0.1, 1.0, weight)[0]
    assert torch.allclose(loss.double(), want.detach(), rtol=1e-4, atol=1e-7)
    want.sum().backward()
    got = dict(grads)
    r, g = got.pop("table")
    got["table"] = torch.zeros_like(block.table).index_add_(0, r.clamp_min(0).long(), g)
    for n, w in leaf.items():
        # every gradient is a chain of fp32 products of at most a few hundred terms, and some twenty of them in a row
        off = (got[n].double() - w.grad).norm() / w.grad.norm()
        assert off < 2e-4, (n, float(off))


def test_decoding_agrees_with_prefill():
    """The same positions in one call and one at a time: equal up to the bf16 roundings of the dense products."""
    import reward_memory as ex
    block = ex.Block(300, seed=3)
    ids, _, _, _ = ex.batch(300, 80, 1, 4)
    ids[20:23] = eg.DEAD
    want = block.forward(ids, torch.tensor([0, 80], device=DEV))["logits"].float()
    got = block.decode(ids).float()
    # products of other shapes may add up in another order: a stream of bf16 values moves by a step (2^-8) at some ten places
    assert (got - want).abs().max() <= 2.0 ** -4 * want.abs().max()
    assert block.status.item() == 0
