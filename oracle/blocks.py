"""Block norm, policy loss and gated delta rule with their gradients (oracle; test infrastructure only).

The definitions in 64 bits, in torch on whichever device the inputs are:

* norm: n = y r(y) w silu(gate) over groups, h' = h + scale n, x = h' r(h') w_next.
* policy: loss = w (-min(r A, clip(r) A) + kl (e^d - 1 - d)) with r = exp(l - old), d = ref - l.
* delta: S <- f S, u = beta (v - S^T k), S <- S + k u^T, y = scale S^T q, with f = sigmoid(g), beta = sigmoid(b); a
  masked position holds the state, gives y = 0 and takes no gradient.

Each function of the norm and the loss also returns bounds on the error of a
computation in fp32 (``UNIT`` = 2^-24), from which the tests take their tolerances.
"""
from __future__ import annotations

from typing import List, Optional

import torch

UNIT = 2.0 ** -24


def _groups(x: torch.Tensor, groups: int) -> torch.Tensor:
    return x.view(x.shape[0], groups, -1)


def _spread(x: torch.Tensor, width: int) -> torch.Tensor:
    return x.repeat_interleave(width, 1)


# --------------------------------------------------------------------------- block norm


def _norm_parts(y, w, gate, groups, eps):
    """n and the pieces of it.  Errors in units: the mean's sum of at most width / 32 + 40 roundings a term gives half of
    that to r, rsqrt and the products a few more; sigmoid(z) carries its argument's rounding (|z|) and a few."""
    T, D = y.shape
    width = D // groups
    r = _spread((_groups(y, groups).pow(2).mean(2) + eps).rsqrt(), width)
    w = torch.ones(D, dtype=torch.float64, device=y.device) if w is None else w.repeat(groups)
    sig = torch.ones_like(y) if gate is None else torch.sigmoid(gate)
    act = torch.ones_like(y) if gate is None else gate * sig
    far = torch.zeros_like(y) if gate is None else gate.abs()
    units = width / 64 + 40 + 4 * far
    return r, w, sig, act, y * r * w * act, units


def norm_add(y, w=None, gate=None, h=None, scale=None, groups=1, eps=1e-6):
    """(h', its error bound)."""
    n, units = _norm_parts(y, w, gate, groups, eps)[4:]
    s = n if scale is None else n * scale
    out = s if h is None else h + s
    return out, UNIT * (s.abs() * units + 2 * out.abs())


def norm_next(h, w_next=None, eps=1e-6):
    """(x, its error bound) of the h' that was kept."""
    x = h * (h.pow(2).mean(1, keepdim=True) + eps).rsqrt()
    x = x if w_next is None else x * w_next
    return x, UNIT * x.abs() * (h.shape[1] / 64 + 40)


def norm_add_grad(dh, y, w=None, gate=None, scale=None, h_out=None, dx=None, w_next=None, groups=1, eps=1e-6):
    """dict of name -> (gradient, error bound): dy, dgate, dres, dw, dscale, dw_next."""
    T, D = y.shape
    width = D // groups
    r, wf, sig, act, n, units = _norm_parts(y, w, gate, groups, eps)
    units = units + D / 32 + 40
    l = torch.zeros_like(y) if dh is None else dh
    size = l.abs()
    out = {}
    if dx is not None:
        r2 = (h_out.pow(2).mean(1, keepdim=True) + eps).rsqrt()
        a = dx if w_next is None else dx * w_next
        l = l + a * r2 - h_out * r2 ** 3 * (a * h_out).mean(1, keepdim=True)
        size = size + (a * r2).abs() + h_out.abs() * r2 ** 3 * (a * h_out).abs().mean(1, keepdim=True)
        t = dx * h_out * r2
        out["dw_next"] = (t.sum(0), UNIT * (units.max() + T) * t.abs().sum(0))
    out["dres"] = (l, UNIT * units * size)
    s = 1.0 if scale is None else scale
    g, gs = l * s, size * abs(s)
    t, ts = l * n, size * n.abs()
    out["dscale"] = (t.sum(0), UNIT * (units.max() + T) * ts.sum(0))
    hat = y * r
    t, ts = g * act * hat, gs * (act * hat).abs()
    out["dw"] = (t.view(T, groups, width).sum((0, 1)),
                 UNIT * (units.max() + T + groups) * ts.view(T, groups, width).sum((0, 1)))
    if gate is not None:
        out["dgate"] = (g * hat * wf * sig * (1.0 + gate * (1.0 - sig)),
                        UNIT * units * gs * (hat * wf).abs() * sig * (1.0 + gate.abs()))
    p, ps = g * act * wf, gs * (act * wf).abs()
    mean = lambda x: _spread(_groups(x, groups).mean(2), width)  # noqa: E731
    out["dy"] = (p * r - y * r ** 3 * mean(p * y), UNIT * units * (ps * r + y.abs() * r ** 3 * mean(ps * y.abs())))
    return out


# --------------------------------------------------------------------------- policy loss


def policy(z, ids, adv, old=None, ref=None, clip=(0.2, 0.2), kl=0.0, tau=1.0, weight=None):
    """(loss [T], error bound, logp [T], error bound, dz [T][V], error bound).

    The fp32 error of exp(a) is taken as (8 + 2 |a|) units, that of a sum over
    the vocabulary as V / 256 + 20 more (at least 256 partial sums, then a tree)."""
    T, V = z.shape
    w = torch.ones(T, dtype=torch.float64, device=z.device) if weight is None else weight
    ok = (ids >= 0) & (ids < V) & (w != 0)
    at = torch.where(ok, ids, 0).long()[:, None]
    arg = (z - z.max(1, keepdim=True).values) / tau
    total = torch.exp(arg).sum(1, keepdim=True)
    q = torch.exp(arg) / total
    far = torch.where(torch.isfinite(arg), arg.abs(), 0.0)
    se = (28 + 2 * (q * far).sum(1) + V / 256) * UNIT  # relative error of the vocabulary's sum
    l = arg.gather(1, at)[:, 0] - total[:, 0].log()
    le = se + 4 * UNIT * (far.gather(1, at)[:, 0] + total[:, 0].log().abs() + l.abs())
    r = torch.ones_like(l) if old is None else torch.exp(l - old)
    re = r * (le + UNIT * (8 + 4 * (l if old is None else (l - old)).abs())) * (0.0 if old is None else 1.0)
    cut = r.clamp(1.0 - clip[0], 1.0 + clip[1])
    kept = r * adv <= cut * adv
    loss = -torch.minimum(r * adv, cut * adv)
    lerr = (re + 4 * UNIT * (r + cut)) * adv.abs()
    d = torch.where(kept, -r * adv, 0.0)
    de = torch.where(kept, lerr, 0.0)
    if kl:
        gap = ref - l
        ge = le + UNIT * gap.abs()
        slope = torch.expm1(gap)
        loss = loss + kl * (slope - gap)
        lerr = lerr + kl * (slope.abs() * ge + 16 * UNIT * (slope - gap).abs() + 8 * UNIT * slope.abs() * (gap.abs() >= 0.125))
        d = d - kl * slope
        de = de + kl * ((1 + slope.abs()) * ge + 8 * UNIT * slope.abs())
    w = torch.where(ok, w, 0.0)
    # a row that is not read gives zeros, whatever its numbers are
    zero = lambda x: torch.where(w != 0, x, 0.0)  # noqa: E731
    lerr = zero(lerr + 4 * UNIT * loss.abs())
    dd, dde = zero(w * d) / tau, zero(w.abs() * (de + 6 * UNIT * d.abs())) / tau
    q, far, se = (torch.where((w != 0).view(-1, *[1] * (x.dim() - 1)), x, 0.0) for x in (q, far, se))
    dz = -dd[:, None] * q
    dz.scatter_add_(1, at, dd[:, None])
    dze = dde[:, None] * q + dd.abs()[:, None] * q * (se[:, None] + (12 + 2 * far) * UNIT)
    dze.scatter_add_(1, at, (dde + 2 * UNIT * dd.abs())[:, None])
    return zero(w * loss), w.abs() * lerr, torch.where(ok, l, 0.0), torch.where(ok, le, 0.0), dz, dze


# --------------------------------------------------------------------------- gated delta rule


def _heads(x, heads, group):
    return x.view(x.shape[0], heads, -1).repeat_interleave(group, 1)


def delta(q, k, v, g, b, cu: List[int], keys: int, scale: float, mask: Optional[List[int]] = None,
          state: Optional[torch.Tensor] = None, slots: Optional[List[int]] = None):
    """dict of y [T][H*dv], the states before every position and the last states [n_slots][H][dk][dv]."""
    T, H = g.shape
    q, k, v = _heads(q, keys, H // keys), _heads(k, keys, H // keys), v.view(T, H, -1)
    f, beta = torch.sigmoid(g), torch.sigmoid(b)
    dk, dv = q.shape[2], v.shape[2]
    y, us = torch.zeros_like(v), torch.zeros_like(v)
    before = torch.zeros((T, H, dk, dv), dtype=torch.float64, device=q.device)
    out = None if state is None else state.clone()
    for n in range(len(cu) - 1):
        slot = n if slots is None else slots[n]
        if slot < 0:
            continue
        S = torch.zeros_like(before[0]) if T and state is None else None
        S = S if state is None else state[slot].clone()
        for t in range(cu[n], cu[n + 1]):
            if mask is not None and mask[t]:
                continue
            before[t] = S
            S = S * f[t][:, None, None]
            u = beta[t][:, None] * (v[t] - (S * k[t][:, :, None]).sum(1))
            S = S + k[t][:, :, None] * u[:, None]
            us[t] = u
            y[t] = scale * (S * q[t][:, :, None]).sum(1)
        if out is not None:
            out[slot] = S
    return dict(y=y.reshape(T, -1), before=before, us=us, state=out)


def delta_grad(dy, q, k, v, g, b, cu: List[int], keys: int, scale: float, mask: Optional[List[int]] = None,
               state: Optional[torch.Tensor] = None, slots: Optional[List[int]] = None,
               dstate: Optional[torch.Tensor] = None):
    """dict of dq, dk, dv, dg, db and the first states' gradient dstate; `reach`, the largest value of any position's
    state's gradient, and `held`, that of any state, for the tests' tolerances."""
    fwd = delta(q, k, v, g, b, cu, keys, scale, mask, state, slots)
    T, H = g.shape
    Q, K, V = _heads(q, keys, H // keys), _heads(k, keys, H // keys), v.view(T, H, -1)
    f, beta = torch.sigmoid(g), torch.sigmoid(b)
    do = dy.view(T, H, -1) * scale
    dq, dk, dv = torch.zeros_like(Q), torch.zeros_like(K), torch.zeros_like(V)
    dg, db = torch.zeros_like(f), torch.zeros_like(f)
    out = None if dstate is None else dstate.clone()
    reach = 0.0
    for n in range(len(cu) - 1):
        slot = n if slots is None else slots[n]
        if slot < 0:
            continue
        dS = torch.zeros((H, Q.shape[2], V.shape[2]), dtype=torch.float64, device=q.device)
        dS = dS if dstate is None else dstate[slot].clone()
        for t in range(cu[n + 1] - 1, cu[n] - 1, -1):
            if mask is not None and mask[t]:
                continue
            S = fwd["before"][t] * f[t][:, None, None]
            u = fwd["us"][t]
            after = S + K[t][:, :, None] * u[:, None]
            dq[t] = (after * do[t][:, None]).sum(2)
            dS = dS + Q[t][:, :, None] * do[t][:, None]
            reach = max(reach, float(dS.abs().max()))
            du = (dS * K[t][:, :, None]).sum(1)
            dv[t] = beta[t][:, None] * du
            seen = (S * K[t][:, :, None]).sum(1)
            db[t] = (du * (V[t] - seen)).sum(1) * beta[t] * (1 - beta[t])
            dk[t] = (dS * u[:, None]).sum(2) - (S * dv[t][:, None]).sum(2)
            dS = dS - K[t][:, :, None] * dv[t][:, None]
            dg[t] = (dS * S).sum((1, 2)) * (1 - f[t])
            dS = dS * f[t][:, None, None]
        if out is not None:
            out[slot] = dS
    shared = lambda x: x.view(T, keys, H // keys, -1).sum(2).reshape(T, -1)  # noqa: E731
    held = max(float(fwd["before"].abs().max()), float(fwd["us"].abs().max())) if T else 0.0
    return dict(dq=shared(dq), dk=shared(dk), dv=dv.reshape(T, -1), dg=dg, db=db, dstate=out, reach=reach, held=held)
