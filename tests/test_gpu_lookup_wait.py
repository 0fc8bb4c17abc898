"""The waits of the lookup gradient's sort run out: the status says so, nothing follows the unsorted list, and the
context stays usable."""
import numpy as np
import pytest
import torch

import hashed_gram_conditional_gb300 as eg
from gpu_util import DEV, i32, require_gpu, status
from oracle import training as OT

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
GUARD = 4096


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    require_gpu()


def guarded(n, dtype, fill):
    """A buffer of n elements between two guard areas that hold the same value."""
    wide = torch.full((n + 2 * GUARD,), fill, dtype=dtype, device=DEV)
    return wide, wide[GUARD:GUARD + n]


@pytest.mark.parametrize("T,D,R,kind", [(5000, 24, 40, "bf16"), (4097, 33, 5000, "f32"),
                                        (5000, 257, 20_000, "bf16"),  # other SMs clear rows meanwhile
                                        (200_000, 8, 2_000_000, "bf16")])
@pytest.mark.parametrize("dense", [False, True])
def test_a_sort_that_gives_up_leaves_no_gradient(T, D, R, kind, dense):
    rng = np.random.default_rng(T)
    ids = rng.integers(-1, R, size=T).astype(np.int32)
    dout = torch.from_numpy(rng.normal(size=(T, D))).float().to(TYPES[kind]).to(DEV)
    ws = eg.lookup_grad_workspace(T, 1, D, DEV)
    ws.fill_(0x5A)  # entries that name no row of anything
    wide_g, grad = guarded((R if dense else T) * D, torch.float32, 7.0)
    wide_r, rows = guarded(T, torch.int32, 7)
    wide_c, count = guarded(1, torch.int32, 7)
    st = status()
    if dense:
        eg.engram_selftest_grad_wait(dout, i32(ids), R, st, grad, workspace=ws)
    else:
        eg.engram_selftest_grad_wait(dout, i32(ids), R, st, grad, rows, count, workspace=ws)
    torch.cuda.synchronize()
    assert int(st.item()) == eg.ST_TIMEOUT
    assert (grad == 0).all()
    if not dense:
        assert (rows == -1).all() and int(count.item()) == 0
    for wide, n in ((wide_g, grad.numel()), (wide_r, T), (wide_c, 1)):
        assert (wide[:GUARD] == 7).all() and (wide[GUARD + n:] == 7).all()
    # the same call, with nothing missing, in the same workspace
    st.zero_()
    if dense:
        got = eg.engram_lookup_grad(dout, i32(ids), R, grad=grad.view(R, D), workspace=ws, status=st)
    else:
        eg.engram_lookup_grad_rows(dout, i32(ids), R, rows=rows, grad=grad.view(T, D), count=count, workspace=ws, status=st)
        m = int(count.item())
        got = torch.zeros((R, D), device=DEV)
        got[rows[:m].long()] = grad.view(T, D)[:m]
    assert int(st.item()) == 0
    live = torch.from_numpy(ids >= 0).to(DEV)
    at, d = i32(ids).long()[live], dout.double()[live]
    ref = torch.zeros((R, D), dtype=torch.float64, device=DEV).index_add_(0, at, d)
    size = torch.zeros_like(ref).index_add_(0, at, d.abs())
    n = torch.zeros(R, dtype=torch.float64, device=DEV).index_add_(0, at, torch.ones_like(at, dtype=torch.float64))
    assert ((got.double() - ref).abs() <= size * (n[:, None] + 1) * OT.UNIT).all()


def test_small_sorts_have_no_wait():
    dout, ids = torch.zeros((4096, 8), device=DEV), i32(np.zeros(4096))
    with pytest.raises(eg.EngramError, match="RANGE"):
        eg.engram_selftest_grad_wait(dout, ids, 10, status(), torch.empty((10, 8), device=DEV))
