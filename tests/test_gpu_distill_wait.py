"""The waits between the distillation's blocks run out: the status says so, every access stays in bounds, and the
context stays usable."""
import numpy as np
import pytest
import torch

import hashed_gram_conditional_gb300 as eg
from gpu_util import DEV, f32, i32, require_gpu, status

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
GUARD = 4096


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    require_gpu()


@pytest.mark.parametrize("T,V,K,kind", [(700, 9000, 20, "bf16"), (700, 50_000, 200, "bf16"), (500, 99_092, 64, "f32"),
                                        (400, 129_280, 5, "bf16"), (3000, 9001, 64, "bf16")])
@pytest.mark.parametrize("gradient", [True, False])
def test_a_row_whose_pairs_do_not_come(T, V, K, kind, gradient):
    """Clusters of 1 to 8 blocks, fewer and more rows kept, repeated ids: preparing warps are busy when it happens."""
    rng = np.random.default_rng(V)
    pad = 3 if V % 2 else 0
    z = (torch.randn((T, V + pad), device=DEV, generator=torch.Generator(DEV).manual_seed(V)) * 2).to(TYPES[kind])[:, :V]
    ids = rng.integers(0, V, size=(T, K)).astype(np.int32)
    ids[3::11] = ids[3::11, :1]
    ids, t = i32(ids), f32(rng.normal(size=(T, K)))
    want_dz = torch.empty_like(z)
    want = eg.engram_distill(z, ids, t, dlogits=want_dz)
    wide = torch.full((T * (V + pad) + 2 * GUARD,), 7.0, dtype=TYPES[kind], device=DEV)
    dz = wide[GUARD:GUARD + T * (V + pad)].view(T, V + pad)[:, :V]
    wide_l = torch.full((T + 2 * GUARD,), 7.0, device=DEV)
    loss = wide_l[GUARD:GUARD + T]
    st = status()
    eg.engram_selftest_distill_wait(z, ids, t, st, loss, dz if gradient else None)
    torch.cuda.synchronize()
    assert int(st.item()) == eg.ST_TIMEOUT
    for w in (wide, wide_l):
        assert (w[:GUARD] == 7).all() and (w[-GUARD:] == 7).all()
    if pad:
        assert (wide[GUARD:-GUARD].view(T, V + pad)[:, V:] == 7).all()
    st.zero_()
    eg.engram_distill(z, ids, t, loss=loss, dlogits=dz, status=st)  # nothing missing
    assert int(st.item()) == 0
    assert torch.equal(loss.view(torch.int32), want.view(torch.int32)) and torch.equal(dz, want_dz)


def test_short_rows_have_no_wait():
    z, ids, t = torch.zeros((3, 500), device=DEV), i32(np.zeros((3, 2))), f32(np.zeros((3, 2)))
    st, loss = status(), torch.empty(3, device=DEV)
    eg.engram_selftest_distill_wait(z, ids, t, st, loss)
    assert int(st.item()) == 0 and torch.isfinite(loss).all()
