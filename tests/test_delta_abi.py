"""The C entry points of the gated delta rule's backward pass and of its waits' diagnostic refuse bad arguments before they
touch a device (no GPU needed)."""
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


def test_delta_grad(lib):
    need = lib.engram_delta_workspace_bytes(70, 2, 1, 2, 8, 8, 1)
    assert need > 0 and lib.engram_delta_workspace_bytes(70, -1, 1, 2, 8, 8, 1) == 0

    def call(dy=P(16), dys=16, q=P(16), qs=8, k=P(16), ks=8, v=P(16), vs=16, g=P(16), gs=2, b=P(16), bs=2, ty=F32, T=70, keys=1,
             H=2, dk=8, dv=8, scale=1.0, cu=P(16), S=2, carry=P(16), ds=None, n_slots=0, dq=P(16), dqs=8, dk_=P(16), dks=8,
             dv_=P(16), dvs=16, dg=P(16), dgs=2, db=P(16), dbs=2, ws=P(256), n=need):
        return lib.engram_delta_grad(dy, dys, q, qs, k, ks, v, vs, g, gs, b, bs, ty, T, keys, H, dk, dv, scale, cu, S, None, None,
                                     carry, ds, n_slots, dq, dqs, dk_, dks, dv_, dvs, dg, dgs, db, dbs, ws, n, None, None)
    assert call(ty=2) == INVALID
    assert call(T=-1) == INVALID
    for bad in (dict(keys=0), dict(H=3, keys=2), dict(dk=129), dict(dv=0), dict(qs=7), dict(ks=7), dict(vs=15), dict(gs=1),
                dict(bs=1), dict(dys=15), dict(dqs=7), dict(dks=7), dict(dvs=15), dict(dgs=1), dict(dbs=1), dict(S=0)):
        assert call(**bad) == SHAPE, bad
    for name in ("dy", "q", "k", "g", "b", "cu", "carry", "dq", "dk_", "dv_", "dg", "db", "ws"):
        assert call(**{name: None}) == INVALID, name
    for name in ("dy", "q", "k", "v", "g", "b", "carry", "dq", "dk_", "dv_", "dg", "db"):
        assert call(**{name: P(18)}) == ALIGN, name
    assert call(scale=float("nan")) == INVALID
    assert call(ds=P(16)) == INVALID
    assert call(ds=P(18), n_slots=2) == ALIGN
    assert call(ws=P(16)) == ALIGN
    assert call(n=need - 1) == RANGE
    assert call(v=None, vs=0, n=need - 1) == RANGE  # the values are not needed: the next check is reached
    assert call(T=0, S=0) == OK
    assert call(T=0, dy=None, q=None, k=None, v=None, carry=None) == OK


def test_the_diagnostic_of_the_waits(lib):
    need = [lib.engram_delta_workspace_bytes(70, 2, 1, 2, 8, 8, b) for b in (0, 1)]

    def call(which=0, dy=None, q=P(16), ty=BF16, T=70, y=P(16), carry=P(16), dq=P(16), n=None):
        return lib.engram_selftest_delta_wait(which, dy, q, P(16), P(16), P(16), P(16), ty, T, 1, 2, 8, 8, P(16), 2, y, carry, dq,
                                              P(16), P(16), P(16), P(16), P(256), need[dy is not None] if n is None else n, None,
                                              None)
    for dy in (None, P(16)):
        assert call(which=-1, dy=dy) == INVALID and call(which=2, dy=dy) == INVALID
        assert call(ty=3, dy=dy) == INVALID
        assert call(q=None, dy=dy) == INVALID
        assert call(carry=P(18), dy=dy) == ALIGN
        assert call(n=16, dy=dy) == RANGE
    assert call(y=None) == INVALID
    assert call(dy=P(16), dq=None) == INVALID
    assert call(dy=P(16), carry=None) == INVALID
    # what it leaves out is left out of its own call alone
    assert lib.engram_delta(P(16), 8, P(16), 8, P(16), 16, P(16), 2, P(16), 2, BF16, 0, 1, 2, 8, 8, 1.0, P(16), 2, None, None, None,
                            None, 0, None, 16, None, None, 0, None, None) == OK
