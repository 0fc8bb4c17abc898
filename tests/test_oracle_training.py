"""The training oracle against central differences and identities of its definitions (CPU)."""
import numpy as np
import pytest

from oracle import training as OT


def central(f, x, v, h=1e-5):
    return (f(x + h * v) - f(x - h * v)) / (2 * h)


def test_lookup_gradient_is_its_transpose():
    rng = np.random.default_rng(1)
    table = rng.normal(size=(11, 5))
    ids = rng.integers(-1, 11, size=(9, 3))
    d = rng.normal(size=(9, 15))
    grad, _, rows = OT.lookup_grad(d, ids, 11, 1.7)
    # the lookup is linear: <d, lookup(v)> = <grad, v>
    v = rng.normal(size=table.shape)
    assert abs((d * OT.lookup(v, ids, 1.7)).sum() - (grad * v).sum()) < 1e-12 * np.abs(grad * v).sum() * 100
    assert (rows == np.unique(ids[ids >= 0])).all()


@pytest.mark.parametrize("masked", [False, True])
def test_recurrence_gradients_against_differences(masked):
    rng = np.random.default_rng(2)
    T, D = 23, 4
    x, g, dy = (rng.normal(size=(T, D)) for _ in range(3))
    cu = [0, 5, 5, 22, 23]
    mask = (rng.random(T) < 0.3).astype(np.uint8) if masked else None
    slots = [2, 0, 3, 5]
    state, dstate = rng.normal(size=(6, D)), rng.normal(size=(6, D))

    def value(x_, g_, s_):
        r = OT.recurrence(x_, g_, cu, mask, s_, slots)
        return (r["y"] * dy).sum() + (r["state"] * dstate).sum()

    got = OT.recurrence_grad(dy, x, g, cu, mask, state, slots, dstate)
    for name, at, f in (("dx", x, lambda a: value(a, g, state)), ("dg", g, lambda a: value(x, a, state)),
                        ("dstate", state, lambda a: value(x, g, a))):
        for _ in range(3):
            v = rng.normal(size=at.shape)
            want = central(f, at, v)
            # the differences' own error: h^2 times third derivatives of order one, and rounding / h
            assert abs((got[name] * v).sum() - want) < 1e-7 * (1 + np.abs(got[name] * v).sum())


def test_recurrence_of_one_position_and_of_masked_sequences():
    x, g = np.array([[2.0]]), np.array([[0.0]])
    assert OT.recurrence(x, g, [0, 1])["y"][0, 0] == 1.0
    r = OT.recurrence(x, g, [0, 1], np.array([1]), np.array([[3.0]]))
    assert r["y"][0, 0] == 0.0 and r["state"][0, 0] == 3.0


@pytest.mark.parametrize("with_lse", [False, True])
def test_distillation_gradient_against_differences(with_lse):
    rng = np.random.default_rng(3)
    T, V, K, tau = 5, 17, 4, 2.5
    z = rng.normal(size=(T, V)) * 2
    ids = np.stack([rng.permutation(V)[:K] for _ in range(T)])
    ids[1, 2] = -1
    ids[2] = -1
    ids[3, 1] = ids[3, 0]
    t = rng.normal(size=(T, K)) * 2
    w = np.array([1.0, 0.5, 2.0, 1.5, 0.0])
    lse = np.log(np.exp(t / tau).sum(1)) + 0.4 if with_lse else None
    _, _, dz, _ = OT.distill(z, ids, t, tau, w, lse)
    assert (dz[2] == 0).all() and (dz[4] == 0).all()
    for _ in range(4):
        v = rng.normal(size=z.shape)
        want = central(lambda a: OT.distill(a, ids, t, tau, w, lse)[0].sum(), z, v)
        assert abs((dz * v).sum() - want) < 1e-7 * (1 + np.abs(dz * v).sum())
    # the gradient of a position sums to w tau (P - P) = 0
    assert np.abs(dz.sum(1)).max() < 1e-12


def test_distillation_is_zero_where_the_student_is_the_teacher():
    z = np.array([[1.0, 2.0, 0.5]])
    loss, _, dz, _ = OT.distill(z, np.array([[0, 1, 2]]), z.copy(), 1.3)
    assert abs(loss[0]) < 1e-15 and np.abs(dz).max() < 1e-15
