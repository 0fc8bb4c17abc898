"""The clipped policy loss and its gradient on the GPU against the 64-bit oracle."""
import math

import pytest
import torch

import hashed_gram_conditional_gb300 as eg
from gpu_util import DEV, require_gpu, status
from oracle import blocks as OB

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    require_gpu()


def inputs(T, V, kind, seed, tau, clip=(0.2, 0.28), pitch=0):
    gen = torch.Generator(DEV).manual_seed(seed)
    z = (torch.randn((T, V + pitch), generator=gen, device=DEV) * 2).to(TYPES[kind])[:, :V]
    ids = torch.randint(0, V, (T,), generator=gen, device=DEV, dtype=torch.int32)
    adv = torch.randn(T, generator=gen, device=DEV)
    l = torch.log_softmax(z.double() / tau, 1).gather(1, ids[:, None].long())[:, 0]
    d = torch.randn(T, generator=gen, device=DEV) * 0.3
    for edge in (math.log(1 - clip[0]), math.log(1 + clip[1])):  # the gradient jumps at the clip's edges
        d = torch.where((d - edge).abs() < 1e-2, edge + 1e-2, d)
    old = (l - d).float()
    ref = (l + torch.randn(T, generator=gen, device=DEV) * 0.5).float()
    w = torch.rand(T, generator=gen, device=DEV)
    return z, ids, adv, old, ref, w


def close(got, want, err, kind="f32"):
    half = 2.0 ** -8 if kind == "bf16" else 0.0  # bf16 rounds to 8 significant bits
    fine = torch.isfinite(want)
    assert torch.equal(got.double()[~fine], want[~fine])
    off = (got.double() - want)[fine].abs()
    tol = (err * (1 + half) + half * want.abs() * (1 + 1e-6) + 1e-38)[fine]
    assert (off <= tol).all(), (int((off > tol).sum()), float((off / tol).max()))


def check(z, ids, adv, old=None, ref=None, clip=(0.2, 0.28), kl=0.0, tau=1.0, weight=None, kind="f32", st=None):
    dz = torch.empty_like(z)
    args = dict(old_logp=old, ref_logp=ref, clip=clip, kl=kl, temperature=tau, weight=weight)
    loss, logp = eg.engram_policy(z, ids, adv, dlogits=dz, status=st, **args)
    alone = eg.engram_policy(z, ids, adv, **args)
    assert torch.equal(loss, alone[0]) and torch.equal(logp, alone[1])  # the loss alone is the same loss
    d = lambda t: None if t is None else t.double()  # noqa: E731
    want = OB.policy(z.double(), ids, d(adv), d(old), d(ref), clip, kl, tau, d(weight))
    close(loss, want[0], want[1])
    close(logp, want[2], want[3])
    close(dz, want[4], want[5], kind)
    return loss, logp, dz


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("T,V", [(1, 1), (1, 1000), (3, 7), (5, 1300), (40, 257), (9, 4099), (3, 20001), (2, 99092),
                                 (3, 129280), (1, 600_001)])
def test_loss_and_gradient(T, V, kind):
    z, ids, adv, old, ref, w = inputs(T, V, kind, V, 1.0)
    check(z, ids, adv, kind=kind)
    check(z, ids, adv, old, kind=kind)
    check(z, ids, adv, old, ref, kl=0.1, weight=w, kind=kind)
    z, ids, adv, old, ref, w = inputs(T, V, kind, V, 0.7)
    check(z, ids, adv, None, ref, kl=0.5, tau=0.7, weight=w, kind=kind)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("T,V,pitch", [(3000, 1000, 0), (1201, 4097, 3), (900, 20003, 5), (500, 40000, 0), (400, 77777, 3),
                                       (330, 129280, 0), (5000, 4088, 0), (2500, 31, 1), (200, 200_001, 7)])
def test_many_rows_for_each_cluster(T, V, pitch, kind):
    """Each block works through several rows, with rows among them that have no token, no weight or nothing to learn."""
    z, ids, adv, old, ref, w = inputs(T, V, kind, T, 1.0, pitch=pitch)
    ids[5::7] = -1
    w[3::11] = 0.0
    adv[2::13] = 0.0
    z[4::17] = float("nan")  # rows that are not read may hold anything
    ids[4::17] = -7
    st = status()
    check(z, ids, adv, old, weight=w, kind=kind, st=st)
    assert int(st.item()) == 0
    ids[8::19] = V
    check(z, ids, adv, old, ref, kl=0.05, weight=w, kind=kind, st=st)
    assert int(st.item()) == eg.ST_BAD_TOKEN


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("V", [1000, 30001, 129280])
def test_the_gradient_takes_the_logits_place(V, kind):
    z, ids, adv, old, ref, w = inputs(300, V, kind, 5, 1.0)
    ids[::9] = -1
    dz = torch.empty_like(z)
    args = dict(old_logp=old, ref_logp=ref, kl=0.1, weight=w)
    want = eg.engram_policy(z, ids, adv, dlogits=dz, **args)
    got = eg.engram_policy(z, ids, adv, dlogits=z, **args)
    assert torch.equal(z, dz) and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_clipped_positions_have_no_gradient():
    """By the formula, on both sides of both edges and for advantages of both signs."""
    z, ids, adv, _, _, _ = inputs(8, 500, "f32", 9, 1.0)
    logp = eg.engram_policy(z, ids, adv)[1]
    ratio = torch.tensor([0.5, 0.5, 0.9, 0.9, 1.1, 1.1, 2.0, 2.0], device=DEV)
    adv = torch.tensor([1.0, -1.0] * 4, device=DEV)
    dz = torch.empty_like(z)
    loss, _ = eg.engram_policy(z, ids, adv, old_logp=logp - ratio.log(), clip=(0.2, 0.2), dlogits=dz)
    want = -torch.minimum(ratio * adv, ratio.clamp(0.8, 1.2) * adv)
    assert torch.allclose(loss, want, rtol=1e-5)
    none = (dz == 0).all(1).tolist()
    assert none == [False, True, False, False, False, False, True, False]


def test_gradient_by_differences():
    z, ids, adv, old, ref, w = inputs(6, 40, "f32", 12, 0.7)
    dz = torch.empty_like(z)
    args = dict(old_logp=old, ref_logp=ref, kl=0.2, temperature=0.7, weight=w)
    eg.engram_policy(z, ids, adv, dlogits=dz, **args)
    d64 = lambda t: t.double()  # noqa: E731
    d = torch.randn(z.shape, dtype=torch.float64, device=DEV, generator=torch.Generator(DEV).manual_seed(3))
    loss = lambda x: OB.policy(x, ids, d64(adv), d64(old), d64(ref), (0.2, 0.2), 0.2, 0.7, d64(w))[0].sum()  # noqa: E731
    want = (loss(z.double() + 1e-6 * d) - loss(z.double() - 1e-6 * d)) / 2e-6
    assert abs(float((dz.double() * d).sum() - want)) < 1e-4 * (1 + abs(float(want)))


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("V", [600, 40000])
def test_logits_of_minus_infinity(V, kind):
    """Masked logits have no probability and no gradient; a token among them has probability 0."""
    z, ids, adv, _, _, _ = inputs(20, V, kind, 15, 1.0)
    cut = torch.rand(z.shape, device=DEV, generator=torch.Generator(DEV).manual_seed(4)) < 0.5
    cut.scatter_(1, ids[:, None].long(), False)
    z[cut] = float("-inf")
    _, logp, dz = check(z, ids, adv, kind=kind)
    assert (dz[cut] == 0).all() and torch.isfinite(logp).all()
    z[0, ids[0].long()] = float("-inf")
    loss, logp = eg.engram_policy(z, ids, adv, old_logp=torch.full_like(adv, -5.0))
    assert logp[0] == -math.inf and torch.isfinite(loss[1:]).all()


@pytest.mark.parametrize("V", [600, 40000])
def test_a_token_without_probability_is_infinitely_far(V):
    z, ids, adv, old, ref, _ = inputs(20, V, "f32", 16, 1.0)
    clean = eg.engram_policy(z, ids, adv, old_logp=old, ref_logp=ref, kl=0.1)
    z[3, ids[3].long()] = float("-inf")
    ref[5] = float("-inf")
    loss, logp = eg.engram_policy(z, ids, adv, old_logp=old, ref_logp=ref, kl=0.1)
    assert logp[3] == -math.inf and loss[3] == math.inf and loss[5] == math.inf
    rest = [t for t in range(20) if t not in (3, 5)]
    assert torch.equal(loss[rest], clean[0][rest]) and torch.equal(logp[rest], clean[1][rest])


@pytest.mark.parametrize("V", [600, 40000])
def test_two_calls_at_once(V):
    """Calls on two streams share nothing."""
    sets = [inputs(200, V, "bf16", 50 + k, 1.0) for k in range(2)]
    want = [eg.engram_policy(z, ids, adv, old_logp=old, ref_logp=ref, kl=0.1, weight=w) for z, ids, adv, old, ref, w in sets]
    sides = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for side, (z, ids, adv, old, ref, w) in zip(sides, sets):
            with torch.cuda.stream(side):
                got.append(eg.engram_policy(z, ids, adv, old_logp=old, ref_logp=ref, kl=0.1, weight=w,
                                            dlogits=torch.empty_like(z)))
        torch.cuda.synchronize()
        for u, x in zip(got, want):
            assert torch.equal(u[0], x[0]) and torch.equal(u[1], x[1])


def test_small_kl_keeps_its_digits():
    """e^d - 1 - d at d of 1e-3 is 5e-7: the difference of its terms would have no digits left."""
    z, ids, adv, _, _, _ = inputs(50, 300, "f32", 21, 1.0)
    logp = eg.engram_policy(z, ids, adv)[1]
    for d in (1e-3, -1e-2, 0.1, 0.2, -0.2):
        ref = logp + d
        gap = (ref - logp).double()
        loss, again = eg.engram_policy(z, ids, torch.zeros_like(adv), ref_logp=ref, kl=1.0)
        assert torch.equal(again, logp)
        want = torch.expm1(gap) - gap
        assert torch.allclose(loss.double(), want, rtol=2.0 ** -19, atol=0.0)


def test_another_stream_and_a_captured_graph():
    z, ids, adv, old, ref, w = inputs(100, 30000, "bf16", 30, 1.0)
    dz = torch.empty_like(z)
    args = dict(old_logp=old, ref_logp=ref, kl=0.1, weight=w)
    want = eg.engram_policy(z, ids, adv, dlogits=dz, **args)
    grad = dz.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = eg.engram_policy(z, ids, adv, dlogits=dz, **args)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got[0], want[0]) and torch.equal(dz, grad)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = eg.engram_policy(z, ids, adv, dlogits=dz, **args)
    dz.zero_()
    graph.replay()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(dz, grad)


def test_the_binding_refuses():
    z, ids, adv, old, ref, w = inputs(4, 50, "f32", 40, 1.0)
    with pytest.raises(TypeError):
        eg.engram_policy(z, ids.long(), adv)
    with pytest.raises(ValueError):
        eg.engram_policy(z, ids[:3], adv)
    with pytest.raises(TypeError):
        eg.engram_policy(z, ids, adv.double())
    with pytest.raises(ValueError):
        eg.engram_policy(z, ids, adv, weight=w[:2])
    for bad in (dict(temperature=0.0), dict(kl=-0.1, ref_logp=ref), dict(kl=0.1), dict(clip=(-0.1, 0.2)),
                dict(clip=(0.2, float("nan")))):
        with pytest.raises(eg.EngramError):
            eg.engram_policy(z, ids, adv, **bad)
