"""Positions without a usable teacher entry, whatever normaliser comes with them: loss 0 and a zero gradient."""
import numpy as np
import pytest
import torch

import hashed_gram_conditional_gb300 as eg
from gpu_util import DEV, f32, i32, require_gpu
from oracle import training as OT

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    require_gpu()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("V", [1000, 20_003, 600_001])  # a warp's rows, a cluster's, rows read twice
def test_no_teacher_mass(V, kind):
    T, K, tau = 8, 6, 2.0
    rng = np.random.default_rng(V)
    z = torch.from_numpy(rng.normal(size=(T, V)) * 2).float().to(TYPES[kind]).to(DEV)
    ids = np.stack([rng.permutation(V)[:K] for _ in range(T)]).astype(np.int32)
    t = (rng.normal(size=(T, K)) * 2 + 3).astype(np.float32)
    lse = (np.log(np.exp(t.astype(np.float64) / tau).sum(1)) + rng.random(T)).astype(np.float32)
    empty = [1, 2, 4, 5, 7]
    ids[1], ids[2], ids[7] = -1, -1, -1  # no entry at all
    t[4], t[5] = -np.inf, -np.inf        # entries without probability
    lse[[1, 4]] = -np.inf                # the log-sum-exp of nothing
    lse[[2, 5]] = np.nan
    dz = torch.full_like(z, 5.0)
    loss = eg.engram_distill(z, i32(ids), f32(t), tau, teacher_lse=f32(lse), dlogits=dz)
    alone = eg.engram_distill(z, i32(ids), f32(t), tau, teacher_lse=f32(lse))
    assert torch.equal(loss.view(torch.int32), alone.view(torch.int32))
    assert (loss[empty] == 0).all() and (dz[empty] == 0).all()
    want, le, wd, de = OT.distill(z.double().cpu().numpy(), ids, t.astype(np.float64), tau, None, lse)
    half = 2.0 ** -8 if kind == "bf16" else 0.0  # bf16 rounds to 8 significant bits
    assert (np.abs(loss.double().cpu().numpy() - want) <= le + 1e-40).all()
    assert (np.abs(dz.double().cpu().numpy() - wd) <= de * (1 + half) + half * np.abs(wd) * (1 + 1e-6) + 1e-38).all()
