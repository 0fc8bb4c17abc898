"""The training operators' C entry points refuse bad arguments before they touch a device (no GPU needed)."""
import ctypes
import os

import pytest

import hashed_gram_conditional_gb300 as eg

P = ctypes.c_void_p
OK, INVALID, SHAPE, ALIGN, RANGE = 0, -1, -3, -4, -5
BF16, F32 = 0, 1


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(eg.library_path()):
        from hashed_gram_conditional_gb300 import build
        build.build()
    return eg.lib()


def test_lookup(lib):
    def call(table=P(16), ty=BF16, R=10, D=8, ids=P(16), T=4, C=3, out=P(16), ld=24):
        return lib.engram_lookup(table, ty, R, D, ids, T, C, 1.0, out, ld, None, None)
    assert call(ty=2) == INVALID
    assert call(R=-1) == INVALID
    assert call(T=-1) == INVALID
    assert call(R=2 ** 31 - 1) == RANGE
    assert call(T=2 ** 31 // 3 + 1) == RANGE
    assert call(D=0) == SHAPE
    assert call(C=0) == SHAPE
    assert call(ld=23) == SHAPE
    assert call(ids=None) == INVALID
    assert call(table=None) == INVALID
    assert call(table=P(17)) == ALIGN
    assert call(out=P(18), ty=F32) == ALIGN
    assert call(T=0, table=None, ids=None, out=None) == OK


def test_lookup_gradients(lib):
    need = lib.engram_lookup_grad_workspace_bytes(4, 3, 8)
    assert need > 0 and lib.engram_lookup_grad_workspace_bytes(-1, 3, 8) == 0

    def dense(dout=P(16), ty=BF16, ld=24, ids=P(16), T=4, C=3, D=8, R=10, grad=P(16), ws=P(256), n=need):
        return lib.engram_lookup_grad(dout, ty, ld, ids, T, C, D, R, 1.0, grad, ws, n, None, None)

    def rows(dout=P(16), ids=P(16), rows=P(16), grad=P(16), count=P(16), ws=P(256), n=need, T=4):
        return lib.engram_lookup_grad_rows(dout, BF16, 24, ids, T, 3, 8, 10, 1.0, rows, grad, count, ws, n, None, None)
    assert dense(ty=-1) == INVALID
    assert dense(ld=20) == SHAPE
    assert dense(R=2 ** 31) == RANGE
    assert dense(dout=None) == INVALID
    assert dense(grad=None) == INVALID
    assert dense(grad=P(18)) == ALIGN
    assert dense(ws=P(128)) == ALIGN
    assert dense(ws=None) == INVALID
    assert dense(n=need - 1) == RANGE
    assert dense(R=0, grad=None) == OK
    assert rows(rows=None) == INVALID
    assert rows(count=None) == INVALID
    assert rows(n=need - 1) == RANGE


def test_recurrence(lib):
    need = lib.engram_recurrence_workspace_bytes(4, 8)
    assert lib.engram_recurrence_carry_bytes(129, 8) == 3 * 8 * 4
    assert lib.engram_recurrence_carry_bytes(0, 8) == 0

    def fwd(x=P(16), xs=8, ty=F32, T=4, D=8, cu=P(16), S=1, state=None, n_slots=0, y=P(16), ys=8, ws=P(256), n=need):
        return lib.engram_recurrence(x, xs, P(16), 8, ty, T, D, cu, S, None, None, state, state, n_slots, y, ys, None,
                                     ws, n, None, None)
    assert fwd(ty=3) == INVALID
    assert fwd(T=-1) == INVALID
    assert fwd(D=0) == SHAPE
    assert fwd(xs=7) == SHAPE
    assert fwd(ys=7) == SHAPE
    assert fwd(x=None) == INVALID
    assert fwd(x=P(18)) == ALIGN
    assert fwd(cu=None) == INVALID
    assert fwd(S=0) == SHAPE
    assert fwd(state=P(16), n_slots=0) == INVALID
    assert fwd(ws=P(8)) == ALIGN
    assert fwd(n=need - 1) == RANGE
    assert fwd(T=0, S=0) == OK

    def bwd(dy=P(16), carry=P(16), dx=P(16), dxs=8, T=4, ws=P(256)):
        return lib.engram_recurrence_grad(dy, 8, P(16), 8, P(16), 8, F32, T, 8, P(16), 1, None, None, None, carry,
                                          None, 0, dx, dxs, P(16), 8, ws, need, None, None)
    assert bwd(carry=None) == INVALID
    assert bwd(dy=None) == INVALID
    assert bwd(dxs=4) == SHAPE
    assert bwd(dx=P(17)) == ALIGN
    assert bwd(ws=None) == INVALID
    assert bwd(T=0) == OK

    def step(x=P(16), B=4, slots=P(16), state=P(16), n_slots=4):
        return lib.engram_recurrence_step(x, 8, P(16), 8, F32, B, 8, slots, state, state, n_slots, P(16), 8, None, None)
    assert step(x=None) == INVALID
    assert step(slots=None) == INVALID
    assert step(state=None) == INVALID
    assert step(n_slots=0) == INVALID
    assert step(B=-1) == INVALID
    assert step(B=0) == OK


def test_distill(lib):
    def call(z=P(16), ty=BF16, T=2, V=50, zs=50, ids=P(16), K=3, tau=1.0, loss=P(16), dz=P(16), ds=50):
        return lib.engram_distill(z, ty, T, V, zs, ids, P(16), K, tau, None, None, loss, dz, ds, None, None)
    assert call(ty=7) == INVALID
    assert call(T=-1) == INVALID
    assert call(V=0) == SHAPE
    assert call(K=1025) == SHAPE
    assert call(K=-1) == SHAPE
    assert call(tau=0.0) == INVALID
    assert call(tau=float("nan")) == INVALID
    assert call(tau=float("inf")) == INVALID
    assert call(zs=49) == SHAPE
    assert call(ds=49) == SHAPE
    assert call(z=None) == INVALID
    assert call(loss=None) == INVALID
    assert call(ids=None) == INVALID
    assert call(z=P(17)) == ALIGN
    assert call(zs=51, ds=50) == SHAPE  # in place with another stride
    assert call(T=0, z=None, loss=None) == OK


def test_binding_refuses_what_is_not_on_the_device(lib):
    import torch
    t = torch.zeros((4, 8))
    with pytest.raises(ValueError):
        eg.engram_lookup(t, torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError):
        eg.engram_recurrence(t, t, torch.tensor([0, 4]))
    with pytest.raises(ValueError):
        eg.engram_distill(t, torch.zeros((4, 2), dtype=torch.int32), torch.zeros((4, 2)))
    with pytest.raises(TypeError):
        eg.engram_lookup_grad(t.int(), torch.zeros(4, dtype=torch.int32), 5)
