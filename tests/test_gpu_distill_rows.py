"""Many rows for each cluster of the distillation: the gradient in the logits' place, and the same bits each time."""
import numpy as np
import pytest
import torch

import hashed_gram_conditional_gb300 as eg
from gpu_util import DEV, f32, i32, require_gpu

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    require_gpu()


def inputs(T, V, K, kind, pad):
    rng = np.random.default_rng(T + V)
    z = (torch.randn((T, V + pad), device=DEV, generator=torch.Generator(DEV).manual_seed(V)) * 2).to(TYPES[kind])
    ids = rng.integers(0, V, size=(T, K)).astype(np.int32)  # some twice
    ids[rng.random((T, K)) < 0.1] = -1
    ids[5::7] = -1
    ids[3::11] = ids[3::11, :1]
    t = (rng.normal(size=(T, K)) * 2 + 3).astype(np.float32)
    w = np.where(rng.random(T) < 0.2, 0.0, rng.normal(size=T)).astype(np.float32)
    return z, i32(ids), f32(t), f32(w)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("T,V,K", [(3000, 1000, 20), (1201, 4097, 64), (1500, 8192, 1), (900, 20003, 33), (400, 77777, 100),
                                   (330, 129280, 64), (700, 50_000, 200), (600, 9000, 1024), (150, 200_001, 7),
                                   (40, 600_001, 33)])
def test_in_place(T, V, K, kind):
    """Rows behind the one whose gradient is being written are read from the same buffer meanwhile."""
    pad = 3 if V % 2 else 0  # odd row lengths also get an odd pitch
    z, ids, t, w = inputs(T, V, K, kind, pad)
    dz = torch.empty_like(z)
    loss = eg.engram_distill(z[:, :V], ids, t, 1.5, weight=w, dlogits=dz[:, :V])
    for _ in range(2):
        mine = z.clone()
        again = eg.engram_distill(mine[:, :V], ids, t, 1.5, weight=w, dlogits=mine[:, :V])
        assert torch.equal(loss.view(torch.int32), again.view(torch.int32))
        assert torch.equal(mine[:, :V], dz[:, :V]) and torch.equal(mine[:, V:], z[:, V:])


def test_past_two_giga_elements_run_to_run():
    """Every row with work, offsets beyond 2^31 elements, twice; some rows also alone."""
    T, V, K = 17_000, 129_280, 4
    z = torch.empty((T, V), dtype=torch.bfloat16, device=DEV)
    z.normal_(0.0, 2.0, generator=torch.Generator(DEV).manual_seed(1))
    ids = torch.randint(0, V, (T, K), generator=torch.Generator(DEV).manual_seed(2), device=DEV, dtype=torch.int32)
    t = torch.randn((T, K), generator=torch.Generator(DEV).manual_seed(3), device=DEV)
    dz, dz2 = torch.empty_like(z), torch.empty_like(z)
    loss = eg.engram_distill(z, ids, t, dlogits=dz)
    again = eg.engram_distill(z, ids, t, dlogits=dz2)
    assert torch.equal(loss.view(torch.int32), again.view(torch.int32)) and torch.equal(dz, dz2)
    for r in (0, 8000, 16_610, T - 2):  # the third pair straddles 2^31 elements
        few = torch.empty((2, V), dtype=torch.bfloat16, device=DEV)
        want = eg.engram_distill(z[r:r + 2], ids[r:r + 2].contiguous(), t[r:r + 2].contiguous(), dlogits=few)
        assert torch.equal(loss[r:r + 2], want) and torch.equal(dz[r:r + 2], few)
