"""The oracle of the block operators against automatic differentiation and differences, on the CPU."""
import pytest
import torch

from oracle import blocks as OB


def rand(*shape, seed=0, scale=1.0, shift=0.0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64) * scale + shift


@pytest.mark.parametrize("groups,gate,res,next_", [(1, True, True, True), (4, True, False, True), (3, False, True, False)])
def test_norm_gradient(groups, gate, res, next_):
    T, D = 5, 24
    y, z, h = rand(T, D, seed=1), rand(T, D, seed=2), rand(T, D, seed=3)
    w, s, wn = rand(D // groups, seed=4), rand(D, seed=5), rand(D, seed=6)
    dh, dx = rand(T, D, seed=7), rand(T, D, seed=8)
    leaves = [t.requires_grad_() for t in (y, z, h, w, s, wn)]
    out, _ = OB.norm_add(y, w, z if gate else None, h if res else None, s, groups, 1e-3)
    total = (out * dh).sum()
    if next_:
        total = total + (OB.norm_next(out, wn, 1e-3)[0] * dx).sum()
    total.backward()
    got = OB.norm_add_grad(dh, y.detach(), w.detach(), z.detach() if gate else None, s.detach(), out.detach(),
                           dx if next_ else None, wn.detach(), groups, 1e-3)
    for name, t in zip(("dy", "dgate", "dres", "dw", "dscale", "dw_next"), leaves):
        if t.grad is not None:
            assert torch.allclose(got[name][0], t.grad, rtol=1e-10, atol=1e-12), name


@pytest.mark.parametrize("kl,old", [(0.0, True), (0.3, True), (0.3, False)])
def test_policy_gradient(kl, old):
    T, V = 7, 30
    z = rand(T, V, seed=10, scale=2.0).requires_grad_()
    ids = torch.tensor([0, 5, 29, -1, 7, 30, 3], dtype=torch.int32)
    adv, w = rand(T, seed=11), torch.rand(T, dtype=torch.float64, generator=torch.Generator().manual_seed(12))
    w[4] = 0.0
    logp = torch.log_softmax(z.detach() / 0.8, 1)[torch.arange(T), ids.clamp(0, V - 1).long()]
    prev = logp - rand(T, seed=13, scale=0.4) if old else None
    ref = logp + rand(T, seed=14, scale=0.4) if kl else None
    loss, _, lp, _, dz, _ = OB.policy(z, ids, adv, prev, ref, (0.2, 0.3), kl, 0.8, w)
    assert (lp[[3, 4, 5]] == 0).all() and (loss[[3, 4, 5]] == 0).all() and (dz[[3, 4, 5]] == 0).all()
    live = [0, 1, 2, 6]
    assert torch.allclose(lp[live], logp[live], rtol=1e-12)
    if not old:  # the ratio is 1, and its gradient that of l
        now = torch.log_softmax(z / 0.8, 1)[torch.arange(T), ids.clamp(0, V - 1).long()]
        loss = w * (torch.where((ids >= 0) & (ids < V), 1.0, 0.0)) * (-adv * torch.exp(now - now.detach()))
        loss = loss + w * torch.where((ids >= 0) & (ids < V), kl * (torch.expm1(ref - now) - (ref - now)), 0.0)
    loss.sum().backward()
    assert torch.allclose(dz.detach(), z.grad, rtol=1e-9, atol=1e-13)


def test_delta_gradient_by_differences():
    T, keys, H, dk, dv = 9, 2, 4, 3, 5
    q, k, v = rand(T, keys * dk, seed=20), rand(T, keys * dk, seed=21, scale=0.5), rand(T, H * dv, seed=22)
    g, b = rand(T, H, seed=23, shift=1.0), rand(T, H, seed=24)
    cu, mask, slots = [0, 4, 4, 9], [0, 0, 1, 0, 0, 0, 0, 1, 0], [2, 0, 1]
    state, dy, dstate = rand(3, H, dk, dv, seed=25), rand(T, H * dv, seed=26), rand(3, H, dk, dv, seed=27)

    def total(q, k, v, g, b, state):
        r = OB.delta(q, k, v, g, b, cu, keys, 0.7, mask, state, slots)
        return (r["y"] * dy).sum() + (r["state"] * dstate).sum()

    args = [q, k, v, g, b, state]
    got = OB.delta_grad(dy, q, k, v, g, b, cu, keys, 0.7, mask, state, slots, dstate)
    for i, name in enumerate(("dq", "dk", "dv", "dg", "db", "dstate")):
        d = rand(*args[i].shape, seed=30 + i)
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + 1e-5 * d, args[i] - 1e-5 * d
        want = (total(*up) - total(*down)) / 2e-5
        assert abs(float((got[name] * d).sum() - want)) <= 1e-7 * (1 + abs(float(want))), name
