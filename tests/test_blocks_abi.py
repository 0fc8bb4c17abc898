"""The block operators' C entry points refuse bad arguments before they touch a device (no GPU needed)."""
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


def test_norm_add(lib):
    def call(y=P(16), ys=8, gate=P(16), gs=8, h=P(16), hs=8, ty=F32, n=4, D=8, G=2, eps=1e-6, w=P(16), s=P(16),
             out=P(32), os_=8, x=P(64), xs=8):
        return lib.engram_norm_add(y, ys, gate, gs, h, hs, ty, n, D, G, eps, w, s, P(16), out, os_, x, xs, None)
    assert call(ty=2) == INVALID
    assert call(n=-1) == INVALID
    assert call(n=2 ** 31) == RANGE
    assert call(D=0) == SHAPE
    assert call(D=2 ** 24 + 8) == SHAPE
    assert call(G=3) == SHAPE
    assert call(G=0) == SHAPE
    assert call(D=4100, G=2050, ys=4100) == SHAPE
    assert call(eps=-1.0) == INVALID
    assert call(eps=float("nan")) == INVALID
    assert call(eps=float("inf")) == INVALID
    assert call(y=None) == INVALID
    assert call(out=None) == INVALID
    for name in ("ys", "gs", "hs", "os_", "xs"):
        assert call(**{name: 7}) == SHAPE
    for name in ("y", "gate", "h", "out", "x", "w", "s"):
        assert call(**{name: P(18)}) == ALIGN
    assert call(out=P(16), os_=9) == SHAPE  # in place with another stride
    assert call(n=0, y=None, out=None) == OK


def test_norm_add_grad(lib):
    need = lib.engram_norm_add_workspace_bytes(4, 8)
    assert need == 2 * 4 * 8 * 4 and lib.engram_norm_add_workspace_bytes(-1, 8) == 0
    assert lib.engram_norm_add_workspace_bytes(10 ** 9, 8) == lib.engram_norm_add_workspace_bytes(10 ** 6, 8)

    def call(dh=P(16), dx=P(16), y=P(16), gate=P(16), out=P(16), ty=F32, n=4, D=8, G=2, dy=P(16), dgate=P(16), dres=P(32),
             ds=8, dw=P(16), ws=P(256), size=need, eps=1e-6):
        return lib.engram_norm_add_grad(dh, 8, dx, 8, y, 8, gate, 8, out, 8, ty, n, D, G, eps, P(16), P(16), P(16), dy, 8,
                                        dgate, 8, dres, ds, dw, P(16), P(16), ws, size, None)
    assert call(ty=5) == INVALID
    assert call(n=-1) == INVALID
    assert call(G=16) == SHAPE
    assert call(eps=-1e-6) == INVALID
    assert call(dh=None, dx=None) == INVALID
    assert call(y=None) == INVALID
    assert call(dy=None) == INVALID
    assert call(out=None) == INVALID  # with dx
    assert call(gate=None) == INVALID  # with dgate
    assert call(ds=7) == SHAPE
    assert call(dres=P(16), ds=9) == SHAPE  # in place with another stride
    assert call(dw=P(18)) == ALIGN
    assert call(dy=P(18)) == ALIGN
    assert call(ws=None) == INVALID
    assert call(ws=P(16)) == ALIGN
    assert call(size=need - 1) == RANGE


def test_policy(lib):
    def call(z=P(16), ty=BF16, T=2, V=50, zs=50, ids=P(16), adv=P(16), ref=None, low=0.2, high=0.2, kl=0.0, tau=1.0,
             loss=P(16), dz=P(16), ds=50):
        return lib.engram_policy(z, ty, T, V, zs, ids, adv, None, ref, low, high, kl, tau, None, loss, None, dz, ds, None,
                                 None)
    assert call(ty=7) == INVALID
    assert call(T=-1) == INVALID
    assert call(T=2 ** 28) == RANGE
    assert call(V=0) == SHAPE
    assert call(tau=0.0) == INVALID
    assert call(tau=float("inf")) == INVALID
    assert call(low=-0.1) == INVALID
    assert call(high=float("nan")) == INVALID
    assert call(high=float("inf")) == INVALID
    assert call(kl=-1.0) == INVALID
    assert call(kl=0.1) == INVALID  # without a reference
    assert call(zs=49) == SHAPE
    assert call(ds=49) == SHAPE
    for name in ("z", "ids", "adv", "loss"):
        assert call(**{name: None}) == INVALID
    assert call(z=P(17)) == ALIGN
    assert call(zs=51, ds=50) == SHAPE  # in place with another stride
    assert call(T=0, z=None, ids=None, adv=None, loss=None) == OK


def test_binding_refuses_what_is_not_on_the_device(lib):
    import torch
    t = torch.zeros((4, 8))
    with pytest.raises(ValueError):
        eg.engram_norm_add(t)
    with pytest.raises(ValueError):
        eg.engram_norm_add_grad(t, t)
    with pytest.raises(ValueError):
        eg.engram_policy(t, torch.zeros(4, dtype=torch.int32), torch.zeros(4))
    with pytest.raises(TypeError):
        eg.engram_norm_add(t.int())


def test_delta(lib):
    need = lib.engram_delta_workspace_bytes(70, 2, 1, 2, 8, 8, 0)
    assert need > 0 and lib.engram_delta_workspace_bytes(-1, 2, 1, 2, 8, 8, 0) == 0
    # at most floor((70 + 63 * 2) / 64) chunks, matrices padded to 16 x 16, and the writes
    assert lib.engram_delta_carry_bytes(70, 2, 2, 8, 8) == (3 * 2 * 16 * 16 + 70 * 2 * 8) * 4 + 3 * 2 * (2 * 3 * 5120 + 1280)
    assert lib.engram_delta_carry_bytes(0, 2, 2, 8, 8) == 0

    def call(q=P(16), qs=8, k=P(16), ks=8, v=P(16), vs=16, g=P(16), gs=2, b=P(16), bs=2, ty=F32, T=70, keys=1, H=2, dk=8,
             dv=8, scale=1.0, cu=P(16), S=2, state=None, n_slots=0, y=P(16), ys=16, carry=None, ws=P(256), n=need):
        return lib.engram_delta(q, qs, k, ks, v, vs, g, gs, b, bs, ty, T, keys, H, dk, dv, scale, cu, S, None, None, state,
                                state, n_slots, y, ys, carry, ws, n, None, None)
    assert call(ty=2) == INVALID
    assert call(T=-1) == INVALID
    assert call(S=-1) == INVALID
    assert call(T=2 ** 31 - 1) == RANGE
    for bad in (dict(keys=0), dict(H=3, keys=2), dict(H=0), dict(dk=0), dict(dk=129), dict(dv=129), dict(dv=0),
                dict(H=65536), dict(qs=7), dict(ks=7), dict(vs=15), dict(gs=1), dict(bs=1), dict(ys=15), dict(S=0)):
        assert call(**bad) == SHAPE, bad
    for name in ("q", "k", "v", "g", "b", "y", "cu", "ws"):
        assert call(**{name: None}) == INVALID, name
    for name in ("q", "k", "v", "g", "b", "y", "carry"):
        assert call(**{name: P(18)}) == ALIGN, name
    assert call(scale=float("inf")) == INVALID
    assert call(state=P(16)) == INVALID
    assert call(state=P(18), n_slots=2) == ALIGN
    assert call(ws=P(16)) == ALIGN
    assert call(n=need - 1) == RANGE
    assert call(T=0, S=0) == OK
    assert call(T=0, q=None, k=None, v=None, g=None, b=None, y=None, ws=None) == OK


def test_delta_step(lib):
    def call(q=P(16), qs=8, vs=16, ty=BF16, B=3, keys=1, H=2, dk=8, dv=8, slots=P(16), state=P(16), out=P(16), n_slots=3,
             y=P(16), ys=16, scale=1.0):
        return lib.engram_delta_step(q, qs, P(16), 8, P(16), vs, P(16), 2, P(16), 2, ty, B, keys, H, dk, dv, scale, slots,
                                     state, out, n_slots, y, ys, None, None)
    assert call(ty=9) == INVALID
    assert call(B=-1) == INVALID
    for bad in (dict(keys=3), dict(dk=200), dict(qs=7), dict(vs=1), dict(ys=3)):
        assert call(**bad) == SHAPE, bad
    for bad in (dict(q=None), dict(slots=None), dict(state=None), dict(out=None), dict(y=None), dict(n_slots=0),
                dict(scale=float("nan"))):
        assert call(**bad) == INVALID, bad
    for bad in (dict(q=P(17)), dict(state=P(18)), dict(out=P(18)), dict(y=P(17))):
        assert call(**bad) == ALIGN, bad
    assert call(B=0, q=None, slots=None, state=None) == OK
