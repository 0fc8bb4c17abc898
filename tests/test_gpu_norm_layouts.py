"""Block norms and their gradients of other layouts and of rows that no ring of shared memory holds."""
import pytest
import torch

from gpu_util import DEV, require_gpu
from test_gpu_norm import run

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    require_gpu()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("T,D,groups", [(33, 512, 4), (33, 512, 1), (2600, 1000, 1), (3, 8192, 1)])
def test_the_same_bits_between_other_columns(T, D, groups, kind):
    """Columns of a wider matrix that are 16-byte aligned go through the kernel that contiguous rows go through."""
    def lay(t):
        wide = torch.full((t.shape[0], D + 24), float("nan"), dtype=t.dtype, device=DEV)
        wide[:, 8:8 + D] = t
        return wide[:, 8:8 + D]
    want, got = (run(T, D, kind, 600, groups, **how) for how in ({}, dict(lay=lay)))
    for u, w in zip((*got[:2], *got[2]), (*want[:2], *want[2])):
        assert torch.equal(u, w)


@pytest.mark.parametrize("T,D,groups,kind", [(700, 8192, 1, "bf16"), (330, 8192, 64, "bf16"), (640, 7512, 1, "bf16"), (400, 7504, 1, "bf16"),
                                             (330, 16384, 1, "bf16"), (650, 4096, 1, "f32"), (330, 5120, 1, "f32"), (330, 5120, 40, "f32"),
                                             (400, 3756, 1, "f32"), (400, 3752, 1, "f32"), (310, 8192, 8, "f32")])
def test_wide_rows_several_for_each_block(T, D, groups, kind):
    """Rows of more than 7504 bf16 or 3752 fp32 values, of which no three are on their way at once, and the last ones
    that are."""
    run(T, D, kind, 620, groups)
    run(T, D, kind, 630, groups, gate=False, res=False, scaled=False, weighted=False, nxt=False)
