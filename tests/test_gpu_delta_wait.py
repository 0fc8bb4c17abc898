"""The delta rule's waits within a block and between blocks run out: the status says so, every access stays in bounds, the
call ends, and the next one on the same buffers is right."""
import pytest
import torch

import hashed_gram_conditional_gb300 as eg
from gpu_util import DEV, i64, require_gpu, status
from test_gpu_delta import cuts, inputs, make

pytestmark = pytest.mark.gpu
GUARD = 4096


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    require_gpu()


class Guarded:
    """A contiguous matrix between two guards."""

    def __init__(self, shape, dtype):
        self.wide = torch.full((torch.Size(shape).numel() + 2 * GUARD,), 7.0, dtype=dtype, device=DEV)
        self.t = self.wide[GUARD:-GUARD].view(shape)

    def intact(self):
        return bool((self.wide[:GUARD] == 7).all() and (self.wide[-GUARD:] == 7).all())


@pytest.mark.parametrize("which,T,S,keys,H,dk,dv,kind,runs_out", [
    (0, 900, 10, 4, 8, 128, 128, "bf16", True), (0, 700, 20, 2, 8, 64, 40, "bf16", True),  # four quads a block
    (0, 300, 80, 1, 2, 33, 125, "bf16", True),  # rows that are not copied in pieces of 16 bytes
    (0, 300, 1, 1, 2, 64, 64, "bf16", False), (0, 300, 4, 2, 4, 64, 64, "f32", False),  # one quad a block: no such wait
    (1, 2000, 12, 4, 40, 16, 40, "bf16", True), (1, 2000, 12, 4, 40, 16, 40, "f32", True),
    (1, 2000, 5, 5, 10, 64, 128, "bf16", True), (1, 300, 1, 1, 2, 64, 64, "bf16", False)])
def test_what_never_comes(which, T, S, keys, H, dk, dv, kind, runs_out):
    args, dy, cu = inputs(T, keys, H, dk, dv, kind, 600), make((T, H * dv), kind, 610), i64(cuts(T, S, S))
    dtype = args[0].dtype
    y, carry = Guarded((T, H * dv), dtype), Guarded(eg.delta_carry(T, S, keys, H, dk, dv, DEV).shape, torch.float32)
    grads = [Guarded(t.shape, dtype) for t in args]
    names, st = ("dq", "dk", "dv", "dg", "db"), status()

    def ordinary():
        st.zero_()
        eg.engram_delta(*args, cu, keys, scale=1.0, y=y.t, carry=carry.t, status=st)
        eg.engram_delta_grad(dy, *args, carry.t, cu, keys, scale=1.0, status=st, **dict(zip(names, (g.t for g in grads))))
        assert int(st.item()) == 0
        return [y.t.clone(), *(g.t.clone() for g in grads)]
    want = ordinary()
    for back in (False, True):
        st.zero_()
        if back:
            eg.engram_selftest_delta_wait(which, *args, cu, keys, st, carry.t, dy=dy, grads=[g.t for g in grads])
        else:
            eg.engram_selftest_delta_wait(which, *args, cu, keys, st, carry.t, y=y.t)
        torch.cuda.synchronize()
        assert int(st.item()) == (eg.ST_TIMEOUT if runs_out else 0)
        assert y.intact() and carry.intact() and all(g.intact() for g in grads)
        if not runs_out:
            assert all(torch.equal(a, b) for a, b in zip(want, (y.t, *(g.t for g in grads))))
        for u, w in zip(ordinary(), want):
            assert torch.equal(u, w)


def test_refusals():
    T, keys, H, d = 8, 1, 2, 8
    args, cu = inputs(T, keys, H, d, d, "f32", 620), i64([0, T])
    carry, y, st = eg.delta_carry(T, 1, keys, H, d, d, DEV), torch.empty((T, H * d), device=DEV), status()
    with pytest.raises(eg.EngramError):
        eg.engram_selftest_delta_wait(2, *args, cu, keys, st, carry, y=y)
    with pytest.raises(ValueError):
        eg.engram_selftest_delta_wait(0, *args, cu, keys, st, carry[:-1], y=y)
    with pytest.raises(ValueError):
        eg.engram_selftest_delta_wait(0, *args, cu, keys, st, carry, dy=y, grads=[torch.empty_like(t) for t in args[:4]])
