"""Row lookup, gated linear recurrence and distillation loss with their gradients (oracle; test infrastructure only).

The definitions in 64 bits, position by position:

* lookup: out[t, j*D + c] = scale * table[ids[t, j], c], ids outside the
  table give zeros; the gradient of row r sums the entries that name it.
* recurrence: s_t = f_t s_{t-1} + (1 - f_t) x_t with f_t = sigmoid(g_t), y_t =
  s_t; a masked position holds the state, gives y = 0 and takes no gradient.
* distillation: loss = w tau^2 sum_k p_k (ln p_k - ln q_{id_k}) with q the
  softmax of the student's logits / tau and p the teacher's probabilities.

Each function also returns, where the GPU result is rounded on the way, a
bound on the error of a computation in fp32 (``unit`` = 2^-24), from which the
tests take their tolerances.
"""
from __future__ import annotations

from typing import List, Optional

import numpy as np

UNIT = 2.0 ** -24


def sigmoid(g: np.ndarray) -> np.ndarray:
    e = np.exp(-np.abs(g))
    return np.where(g >= 0, 1.0, e) / (1.0 + e)


# --------------------------------------------------------------------------- lookup


def lookup(table: np.ndarray, ids: np.ndarray, scale: float) -> np.ndarray:
    """table [R][D], ids [T][C] -> [T][C*D]."""
    T, C = ids.shape
    R, D = table.shape
    out = np.zeros((T, C, D))
    for t in range(T):
        for j in range(C):
            if 0 <= ids[t, j] < R:
                out[t, j] = scale * table[ids[t, j]]
    return out.reshape(T, C * D)


def lookup_grad(dout: np.ndarray, ids: np.ndarray, rows: int, scale: float):
    """(gradient [rows][D], error bound [rows][D], sorted distinct row ids).

    A row's n entries are added in fp32 in some order and multiplied by the
    scale: the error is at most (n + 1) unit times the sum of their sizes."""
    T, C = ids.shape
    D = dout.shape[1] // C
    d = dout.reshape(T * C, D)
    grad, size, n = np.zeros((rows, D)), np.zeros((rows, D)), np.zeros((rows, 1))
    for i, r in enumerate(ids.reshape(-1)):
        if 0 <= r < rows:
            grad[r] += d[i]
            size[r] += np.abs(d[i])
            n[r] += 1
    return scale * grad, abs(scale) * size * (n + 1) * UNIT, np.flatnonzero(n[:, 0] > 0)


# --------------------------------------------------------------------------- recurrence


# Errors of the fp32 gates in units: e = exp(-|g|) carries its argument's
# rounding (|g| units) and the exponential's own few; f = 1 / (1 + e) and 1 - f
# = e / (1 + e) then add the sum's, the reciprocal's and the product's.
def _gate_err(g):
    return 8.0 * UNIT, (12.0 + 2.0 * np.abs(g)) * UNIT


def recurrence(x: np.ndarray, g: np.ndarray, cu: List[int], mask: Optional[np.ndarray] = None,
               state: Optional[np.ndarray] = None, slots: Optional[List[int]] = None):
    """dict of y, its error bound, the states before every position (with their bounds) and the last states
    [n_slots][D] (with theirs)."""
    T, D = x.shape
    f = sigmoid(g)
    u = sigmoid(-g)
    fe, ue = _gate_err(g)
    y, ye = np.zeros((T, D)), np.zeros((T, D))
    before, be = np.zeros((T, D)), np.zeros((T, D))
    out = None if state is None else state.copy()
    oe = None if state is None else np.zeros_like(state)
    n_slots = 0 if state is None else state.shape[0]
    for q in range(len(cu) - 1):
        slot = q if slots is None else slots[q]
        pad = slot < 0 or (state is not None and slot >= n_slots)
        s = np.zeros(D) if state is None or pad else state[slot].copy()
        err = np.zeros(D)
        for t in range(cu[q], cu[q + 1]):
            before[t], be[t] = s, err
            if pad or (mask is not None and mask[t]):
                continue
            new = f[t] * s + u[t] * x[t]
            err = f[t] * err + fe * f[t] * np.abs(s) + ue[t] * u[t] * np.abs(x[t]) + 2 * UNIT * np.abs(new)
            s = new
            y[t], ye[t] = s, err
        if state is not None and not pad:
            out[slot], oe[slot] = s, err
    return dict(y=y, y_err=ye, before=before, before_err=be, state=out, state_err=oe)


def recurrence_grad(dy: np.ndarray, x: np.ndarray, g: np.ndarray, cu: List[int], mask: Optional[np.ndarray] = None,
                    state: Optional[np.ndarray] = None, slots: Optional[List[int]] = None,
                    dstate: Optional[np.ndarray] = None):
    """dict of dx, dg and the first states' gradients, with error bounds."""
    T, D = x.shape
    f, u = sigmoid(g), sigmoid(-g)
    fe, ue = _gate_err(g)
    fwd = recurrence(x, g, cu, mask, state, slots)
    dx, dxe, dg, dge = (np.zeros((T, D)) for _ in range(4))
    out = None if dstate is None else dstate.copy()
    oe = None if dstate is None else np.zeros_like(dstate)
    held = state if state is not None else dstate
    n_slots = 0 if held is None else held.shape[0]
    for q in range(len(cu) - 1):
        slot = q if slots is None else slots[q]
        if slot < 0 or (held is not None and slot >= n_slots):
            continue
        l = np.zeros(D) if dstate is None else dstate[slot].copy()
        err = np.zeros(D)
        for t in range(cu[q + 1] - 1, cu[q] - 1, -1):
            if mask is not None and mask[t]:
                continue
            l = l + dy[t]
            err = err + UNIT * np.abs(l)
            gap = fwd["before"][t] - x[t]
            ge = fwd["before_err"][t] + UNIT * np.abs(gap)
            dx[t] = l * u[t]
            dxe[t] = err * u[t] + np.abs(dx[t]) * (ue[t] + UNIT)
            dg[t] = dx[t] * f[t] * gap
            dge[t] = dxe[t] * f[t] * np.abs(gap) + np.abs(dx[t]) * f[t] * ge + np.abs(dg[t]) * (fe + 3 * UNIT)
            err = f[t] * (err + np.abs(l) * (fe + UNIT))
            l = l * f[t]
        if dstate is not None:
            out[slot], oe[slot] = l, err
    return dict(dx=dx, dx_err=dxe, dg=dg, dg_err=dge, dstate=out, dstate_err=oe)


# --------------------------------------------------------------------------- distillation


def distill(z: np.ndarray, ids: np.ndarray, t: np.ndarray, tau: float, weight: Optional[np.ndarray] = None,
            lse: Optional[np.ndarray] = None):
    """(loss [T], error bound, dz [T][V], error bound).

    The fp32 error of exp(a) is taken as (8 + 2 |a|) units, that of a sum over
    the vocabulary as V / 256 + 20 more (at least 256 partial sums, then a tree)."""
    T, V = z.shape
    K = ids.shape[1]
    loss, le, dz, de = np.zeros(T), np.zeros(T), np.zeros((T, V)), np.zeros((T, V))
    for r in range(T):
        w = 1.0 if weight is None else float(weight[r])
        ok = (ids[r] >= 0) & (ids[r] < V)
        a = np.where(ok, t[r] / tau, -np.inf)
        top = a.max() if K else -np.inf
        if w == 0.0 or top == -np.inf:
            continue
        norm = top + np.log(np.exp(a - top).sum()) if lse is None else float(lse[r])
        lnp = a - norm
        p = np.exp(lnp)
        some = p > 0
        pe = p * (8 + 2 * np.abs(np.where(some, lnp, 0.0)) + 2 * K + 2 * abs(norm)
                  + 2 * np.abs(np.where(some, a, 0.0))) * UNIT
        mass = p.sum()
        if mass == 0.0:
            continue
        zz = z[r] / tau
        m = zz.max()
        arg = zz - m
        e = np.exp(arg)
        total = e.sum()
        q = e / total
        fin = np.where(np.isfinite(arg), np.abs(arg), 0.0)
        se = (28 + 2 * (q * fin).sum() + V / 256) * UNIT  # relative error of the vocabulary sum
        lnq = arg - np.log(total)
        for k in range(K):
            if not ok[k] or p[k] == 0.0:
                continue
            gap = lnp[k] - lnq[ids[r, k]]
            loss[r] += p[k] * gap
            if np.isfinite(gap):
                size = np.abs(a[k]) + abs(norm) + fin[ids[r, k]] + abs(np.log(total))
                le[r] += pe[k] * abs(gap) + p[k] * (se + 4 * size * UNIT) + 4 * UNIT * p[k] * abs(gap)
        le[r] += K * UNIT * le[r] + (K + 4) * UNIT * abs(loss[r]) if np.isfinite(loss[r]) else 0.0
        pv, pve = np.zeros(V), np.zeros(V)
        np.add.at(pv, ids[r][ok], p[ok])
        np.add.at(pve, ids[r][ok], pe[ok])
        scale = w * tau
        dz[r] = scale * (mass * q - pv)
        de[r] = abs(scale) * (mass * q * (se + (12 + 2 * fin) * UNIT) + q * pe.sum() + pve + (K + 3) * UNIT * pv)
        loss[r] *= w * tau * tau
        le[r] *= abs(w) * tau * tau
    return loss, le, dz, de
