"""The distillation loss and its gradient on the GPU against the 64-bit oracle."""
import numpy as np
import pytest
import torch

import hashed_gram_conditional_gb300 as eg
from gpu_util import DEV, f32, i32, require_gpu, status
from oracle import training as OT

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    require_gpu()


def inputs(T, V, K, kind, seed, spread=2.0):
    rng = np.random.default_rng(seed)
    z = torch.from_numpy(rng.normal(size=(T, V)) * spread).float().to(TYPES[kind]).to(DEV)
    ids = np.stack([rng.permutation(V)[:K] for _ in range(T)]).astype(np.int32).reshape(T, K)
    t = (rng.normal(size=(T, K)) * 2 + 3).astype(np.float32)
    return z, ids, t, rng


def check(z, ids, t, tau, weight=None, lse=None, kind="f32", st=None):
    dz = torch.empty_like(z)
    w = None if weight is None else f32(weight)
    e = None if lse is None else f32(lse)
    loss = eg.engram_distill(z, i32(ids), f32(t), tau, weight=w, teacher_lse=e, dlogits=dz, status=st)
    alone = eg.engram_distill(z, i32(ids), f32(t), tau, weight=w, teacher_lse=e)
    assert torch.equal(loss.view(torch.int32), alone.view(torch.int32))  # the loss alone is the same loss
    want, le, wd, de = OT.distill(z.double().cpu().numpy(), ids, t.astype(np.float64), tau, weight, lse)
    got = loss.double().cpu().numpy()
    fin = np.isfinite(want)
    assert (got[~fin] == want[~fin]).all()
    assert (np.abs(got - want)[fin] <= le[fin] + 1e-40).all(), float((np.abs(got - want)[fin] / (le[fin] + 1e-40)).max())
    half = 2.0 ** -8 if kind == "bf16" else 0.0  # bf16 rounds to 8 significant bits
    g = dz.double().cpu().numpy()
    tol = de * (1 + half) + half * np.abs(wd) * (1 + 1e-6) + 1e-38
    assert (np.abs(g - wd) <= tol).all(), float((np.abs(g - wd) / tol).max())
    return loss, dz


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("T,V,K", [(1, 1, 1), (1, 1000, 1), (3, 7, 7), (5, 1300, 20), (2, 99092, 64), (3, 129280, 64),
                                   (7, 4099, 300), (40, 257, 5), (2, 20001, 1024), (1, 600_001, 33)])
def test_loss_and_gradient(T, V, K, kind):
    z, ids, t, rng = inputs(T, V, K, kind, V + K)
    check(z, ids, t, 1.0, kind=kind)
    check(z, ids, t, 2.5, weight=rng.random(T).astype(np.float32), kind=kind)
    lse = np.log(np.exp(t.astype(np.float64) / 2.0).sum(1)) + rng.random(T)
    check(z, ids, t, 2.0, lse=lse.astype(np.float32), kind=kind)


def distill_all(z, ids, t, tau, weight):
    """OT.distill for many rows at once, in torch's 64 bits: the same values and the same bounds."""
    T, V = z.shape
    K, U = ids.shape[1], OT.UNIT
    ok = (ids >= 0) & (ids < V)
    at = torch.where(ok, ids, 0).long()
    a = torch.where(ok, t / tau, -torch.inf)
    top = a.max(1, keepdim=True).values
    live = (weight != 0) & (top[:, 0] > -torch.inf)
    top = torch.where(top > -torch.inf, top, 0.0)
    norm = top + torch.log(torch.exp(a - top).sum(1, keepdim=True))
    norm = torch.where(live[:, None], norm, 0.0)
    lnp = a - norm
    p = torch.exp(lnp)
    some = p > 0
    fa = torch.where(some, a.abs(), 0.0)
    pe = p * (8 + 2 * torch.where(some, lnp.abs(), 0.0) + 2 * K + 2 * norm.abs() + 2 * fa) * U
    zz = z / tau
    arg = zz - zz.max(1, keepdim=True).values
    e = torch.exp(arg)
    total = e.sum(1, keepdim=True)
    q = e / total
    fin = arg.abs()
    se = (28 + 2 * (q * fin).sum(1, keepdim=True) + V / 256) * U
    gap = torch.where(some, lnp - (arg.gather(1, at) - total.log()), 0.0)
    size = fa + norm.abs() + fin.gather(1, at) + total.log().abs()
    loss = (p * gap).sum(1)
    le = (pe * gap.abs() + p * (se + 4 * size * U) + 4 * U * p * gap.abs()).sum(1)
    le = le * (1 + K * U) + (K + 4) * U * loss.abs()
    pv, pve = torch.zeros_like(zz), torch.zeros_like(zz)
    pv.scatter_add_(1, at, p * ok)
    pve.scatter_add_(1, at, pe * ok)
    w = torch.where(live, weight, 0.0)[:, None]
    mass = p.sum(1, keepdim=True)
    dz = w * tau * (mass * q - pv)
    de = w.abs() * tau * (mass * q * (se + (12 + 2 * fin) * U) + q * pe.sum(1, keepdim=True) + pve + (K + 3) * U * pv)
    f = w[:, 0] * tau * tau
    return loss * f, le * f.abs(), dz, de


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("T,V,K", [(3000, 1000, 20), (1201, 4097, 64), (1500, 8192, 1), (900, 20003, 33), (500, 40000, 64),
                                   (400, 77777, 100), (330, 129280, 64), (700, 50_000, 200), (600, 9000, 1024), (5000, 4088, 300),
                                   (2500, 31, 31), (200, 200_001, 7)])
def test_many_rows_for_each_cluster(T, V, K, kind):
    """Each block works through several rows, with rows among them that have nothing to do or an odd teacher."""
    rng = np.random.default_rng(T)
    pad = 3 if V % 2 else 0  # odd row lengths also get an odd pitch
    z = (torch.randn((T, V + pad), device=DEV, generator=torch.Generator(DEV).manual_seed(V)) * 2).to(TYPES[kind])[:, :V]
    ids = rng.integers(0, V, size=(T, K)).astype(np.int32)  # some twice
    ids[rng.random((T, K)) < 0.1] = -1
    t = (rng.normal(size=(T, K)) * 2 + 3).astype(np.float32)
    t[rng.random((T, K)) < 0.05] = -np.inf
    ids[5::7] = -1
    ids[3::11] = ids[3::11, :1]
    w = np.where(rng.random(T) < 0.3, 0.0, rng.normal(size=T)).astype(np.float32)
    w[40:90] = 0.0  # a stretch of them
    dz = torch.full((T, V + pad), float("nan"), dtype=TYPES[kind], device=DEV)
    loss = eg.engram_distill(z, i32(ids), f32(t), 1.5, weight=f32(w), dlogits=dz[:, :V])
    alone = eg.engram_distill(z, i32(ids), f32(t), 1.5, weight=f32(w))
    assert torch.equal(loss.view(torch.int32), alone.view(torch.int32))
    again = torch.empty_like(dz)
    eg.engram_distill(z, i32(ids), f32(t), 1.5, weight=f32(w), dlogits=again[:, :V])
    assert torch.equal(dz[:, :V], again[:, :V])
    if pad:
        assert torch.isnan(dz[:, V:].float()).all()
    half = 2.0 ** -8 if kind == "bf16" else 0.0
    for lo in range(0, T, 100):
        c = slice(lo, min(lo + 100, T))
        want, le, wd, de = distill_all(z[c].double(), i32(ids[c]), f32(t[c]).double(), 1.5, f32(w[c]).double())
        assert ((loss[c].double() - want).abs() <= le + 1e-40).all()
        assert ((dz[c, :V].double() - wd).abs() <= de * (1 + half) + half * wd.abs() * (1 + 1e-6) + 1e-38).all()
        if lo == 0:  # the two 64-bit forms agree
            few = slice(0, 12)
            o = OT.distill(z[few].double().cpu().numpy(), ids[few], t[few].astype(np.float64), 1.5, w[few].astype(np.float64))
            for mine, other in zip((want, le, wd, de), o):
                np.testing.assert_allclose(mine[few].cpu().numpy(), other, rtol=1e-9, atol=1e-15)


def test_unused_repeated_and_bad_entries():
    T, V, K = 9, 500, 12
    z, ids, t, _ = inputs(T, V, K, "f32", 1)
    ids[0, 3:] = -1            # a short list
    ids[1] = -1                # an empty one
    ids[2, 5] = ids[2, 4]      # an id twice
    ids[3] = 77                # one id for every entry
    t[4, 2:] = -np.inf         # entries without probability
    t[5] = -np.inf
    st = status()
    loss, dz = check(z, ids, t, 1.5, st=st)
    assert int(st.item()) == 0
    for r in (1, 5):
        assert loss[r] == 0 and (dz[r] == 0).all()
    ids[6, 0], ids[7, 1], ids[8, 2] = V, 2 ** 31 - 1, -2 ** 31
    check(z, ids, t, 1.5, st=st)
    assert int(st.item()) == eg.ST_BAD_TOKEN


def test_no_entries_at_all():
    z, _, _, _ = inputs(3, 50, 1, "f32", 2)
    dz = torch.full_like(z, 5.0)
    none = torch.empty((3, 0), device=DEV)
    loss = eg.engram_distill(z, none.int(), none, dlogits=dz)
    assert (loss == 0).all() and (dz == 0).all()
    assert eg.engram_distill(z[:0], none[:0].int(), none[:0]).shape == (0,)


def test_positions_without_weight_may_hold_anything():
    z, ids, t, _ = inputs(6, 3001, 8, "bf16", 3)
    z[1], z[4] = float("nan"), float("inf")
    w = np.array([1, 0, 0.5, 1, 0, 2], dtype=np.float32)
    dz = torch.empty_like(z)
    loss = eg.engram_distill(z, i32(ids), f32(t), weight=f32(w), dlogits=dz)
    assert (loss[[1, 2, 4]][[0, 2]] == 0).all() and (dz[[1, 4]] == 0).all()
    keep = [0, 2, 3, 5]
    check(z[keep].contiguous(), ids[keep], t[keep], 1.0, weight=w[keep], kind="bf16")
    assert torch.isfinite(loss).all() and torch.isfinite(dz.float()).all()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_masked_logits(kind):
    """-inf and the type's lowest value in masked places of the vocabulary."""
    low = torch.finfo(TYPES[kind]).min
    for fill in (float("-inf"), low):
        z, ids, t, rng = inputs(4, 2000, 10, kind, 4)
        ids[:] = ids % 700
        for r in range(4):
            ids[r] = rng.permutation(700)[:10]
        z[:, 700:] = fill
        _, dz = check(z, ids, t, 1.0, kind=kind)
        assert (dz[:, 700:] == 0).all()
    z, ids, t, _ = inputs(2, 64, 3, kind, 5)
    z[0] = low  # nothing but the lowest value: the uniform distribution
    check(z, ids, t, 2.0, kind=kind)
    z[1, int(ids[1, 0])] = float("-inf")  # the student excludes what the teacher gives
    dz = torch.empty_like(z)
    loss = eg.engram_distill(z, i32(ids), f32(t), 2.0, dlogits=dz)
    assert loss[1] == float("inf") and torch.isfinite(dz[1].float()).all() and dz[1, int(ids[1, 0])] < 0


def test_large_logits_do_not_overflow():
    z, ids, t, _ = inputs(3, 5000, 6, "f32", 6, spread=200.0)
    check(z, ids, t * 50, 1.0)
    check(z, ids, t, 0.25)


def test_nan_gives_nan_in_its_position_only():
    z, ids, t, _ = inputs(3, 4000, 6, "f32", 7)
    z[1, 3999] = float("nan")
    dz = torch.empty_like(z)
    loss = eg.engram_distill(z, i32(ids), f32(t), dlogits=dz)
    assert torch.isnan(loss).tolist() == [False, True, False]
    assert torch.isnan(dz[1]).all() and torch.isfinite(dz[[0, 2]]).all()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("V", [999, 1000, 70001, 140000])
def test_strides_alignment_and_in_place(kind, V):
    T, K = 5, 9
    z, ids, t, _ = inputs(T, V + 11, K, kind, 8)
    ids %= V
    part = z[:, 3:3 + V]  # rows on odd addresses
    want_dz = torch.empty((T, V), dtype=TYPES[kind], device=DEV)
    want = eg.engram_distill(part.contiguous(), i32(ids), f32(t), 1.5, dlogits=want_dz)
    wide = torch.full((T, V + 6), 4.0, dtype=TYPES[kind], device=DEV)
    loss = eg.engram_distill(part, i32(ids), f32(t), 1.5, dlogits=wide[:, 2:2 + V])
    # another alignment may add the vocabulary in another order: one fp32 error bound apart
    _, le, wd, de = OT.distill(part.double().cpu().numpy(), ids, t.astype(np.float64), 1.5)
    assert (np.abs((loss - want).double().cpu().numpy()) <= 2 * le).all()
    half = 2.0 ** -7 if kind == "bf16" else 0.0  # two roundings
    gap = np.abs((wide[:, 2:2 + V].double() - want_dz.double()).cpu().numpy())
    assert (gap <= 2 * de + half * np.abs(wd) * 1.01 + 1e-38).all()
    assert (wide[:, :2] == 4).all() and (wide[:, 2 + V:] == 4).all()
    mine = z.clone()
    loss2 = eg.engram_distill(mine[:, 3:3 + V], i32(ids), f32(t), 1.5, dlogits=mine[:, 3:3 + V])
    assert torch.equal(loss, loss2)
    assert (mine[:, :3] == z[:, :3]).all() and (mine[:, 3 + V:] == z[:, 3 + V:]).all()
    gap = np.abs((mine[:, 3:3 + V].double() - want_dz.double()).cpu().numpy())
    assert (gap <= 2 * de + half * np.abs(wd) * 1.01 + 1e-38).all()


def test_gradient_against_differences():
    T, V, K, tau = 4, 300, 7, 1.7
    z, ids, t, rng = inputs(T, V, K, "f32", 9)
    dz = torch.empty_like(z)
    eg.engram_distill(z, i32(ids), f32(t), tau, dlogits=dz)
    z64, t64, h = z.double().cpu().numpy(), t.astype(np.float64), 1e-5
    _, _, _, de = OT.distill(z64, ids, t64, tau)
    for _ in range(3):
        v = rng.normal(size=z64.shape)
        up, down = (OT.distill(z64 + s * h * v, ids, t64, tau)[0].sum() for s in (1, -1))
        got = (dz.double().cpu().numpy() * v).sum()
        # the gradient's fp32 bound in this direction, and the differences' own error
        assert abs(got - (up - down) / (2 * h)) <= (de * np.abs(v)).sum() + 2.0 ** -24 * T * V + 1e-7


def test_rows_past_two_giga_elements_and_run_to_run():
    """Row offsets beyond 2^31 elements; the same bits each time."""
    T, V, K = 17_000, 129_280, 4
    z = torch.zeros((T, V), dtype=torch.bfloat16, device=DEV)
    last, ids, t, _ = inputs(2, V, K, "bf16", 10)
    z[T - 2:] = last
    w = torch.zeros(T, device=DEV)
    w[T - 2:] = 1.0
    full_ids = torch.zeros((T, K), dtype=torch.int32, device=DEV)
    full_t = torch.zeros((T, K), device=DEV)
    full_ids[T - 2:], full_t[T - 2:] = i32(ids), f32(t)
    dz = torch.empty_like(z)
    loss = eg.engram_distill(z, full_ids, full_t, weight=w, dlogits=dz)
    small = torch.empty_like(last)
    want = eg.engram_distill(last, i32(ids), f32(t), dlogits=small)
    assert torch.equal(loss[T - 2:], want) and torch.equal(dz[T - 2:], small) and (loss[:T - 2] == 0).all()


def test_refusals():
    z, ids, t, _ = inputs(2, 50, 3, "f32", 11)
    with pytest.raises(TypeError):
        eg.engram_distill(z.double(), i32(ids), f32(t))
    with pytest.raises(TypeError):
        eg.engram_distill(z, i32(ids).long(), f32(t))
    with pytest.raises(ValueError):
        eg.engram_distill(z, i32(ids)[:1], f32(t))
    with pytest.raises(ValueError):
        eg.engram_distill(z, i32(ids), f32(t.T.copy()))
    with pytest.raises(ValueError):
        eg.engram_distill(z, i32(ids), f32(t), status=torch.zeros(1, dtype=torch.int32))
    with pytest.raises(TypeError):
        eg.engram_distill(z, i32(ids), f32(t), status=torch.zeros(1, device=DEV))
    with pytest.raises(ValueError):
        eg.engram_distill(z, i32(ids), f32(t), dlogits=torch.empty((2, 49), device=DEV))
    with pytest.raises(eg.EngramError, match="INVALID"):
        eg.engram_distill(z, i32(ids), f32(t), temperature=0.0)
    with pytest.raises(eg.EngramError, match="INVALID"):
        eg.engram_distill(z, i32(ids), f32(t), temperature=float("nan"))
    big = torch.zeros((2, 1025), device=DEV)
    with pytest.raises(eg.EngramError, match="SHAPE"):
        eg.engram_distill(z, big.int(), big)
