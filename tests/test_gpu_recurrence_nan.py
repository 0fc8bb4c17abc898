"""A NaN in the recurrence stays in its channel, in both types, wherever it enters: scan, backward pass and step."""
import numpy as np
import pytest
import torch

import hashed_gram_conditional_gb300 as eg
from gpu_util import DEV, i32, i64, require_gpu
from oracle import training as OT

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
NAN = float("nan")


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    require_gpu()


def make(shape, kind, seed, shift=0.0):
    rng = np.random.default_rng(seed)
    return torch.from_numpy(rng.normal(size=shape) + shift).float().to(TYPES[kind]).to(DEV)


def f64(t):
    return t.double().cpu().numpy()


def same_but_nan(got, want, clean):
    """NaN exactly where the definition has it; every other value as in the run without NaN, bit for bit."""
    nan = torch.isnan(got)
    assert torch.equal(nan.cpu(), torch.from_numpy(np.isnan(want)))
    assert torch.equal(got[~nan], clean[~nan])


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("T,D,cu", [(100, 32, [0, 40, 100]), (100, 33, [0, 100]), (700, 40, [0, 130, 590, 700]),
                                    (2300, 264, [0, 2300])])
@pytest.mark.parametrize("where", ["g", "x", "dy"])
def test_scan_and_gradients(T, D, cu, where, kind):
    """One tile and many; a NaN at even and odd channels, the second of them late in its sequence."""
    x, g, dy = make((T, D), kind, 1), make((T, D), kind, 2, 1.0), make((T, D), kind, 3)

    def run(x, g, dy):
        carry = eg.recurrence_carry(T, D, DEV)
        ds = torch.zeros((len(cu) - 1, D), device=DEV)
        y = eg.engram_recurrence(x, g, i64(cu), carry=carry)
        dx, dg = eg.engram_recurrence_grad(dy, x, g, carry, i64(cu), dstate=ds)
        return y, dx, dg, ds

    clean = run(x, g, dy)
    bad = dict(x=x.clone(), g=g.clone(), dy=dy.clone())
    for t, c in ((T // 2, 5), (T - 3, D - 2), (T // 3, 16)):
        bad[where][t, c] = NAN
    got = run(bad["x"], bad["g"], bad["dy"])
    a = (f64(bad["x"]), f64(bad["g"]), cu)
    w = OT.recurrence_grad(f64(bad["dy"]), *a, dstate=np.zeros((len(cu) - 1, D)))
    for mine, want, other in zip(got, (OT.recurrence(*a)["y"], w["dx"], w["dg"], w["dstate"]), clean):
        same_but_nan(mine, want, other)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("D", [8, 9, 600])
@pytest.mark.parametrize("where", ["g", "x", "state"])
def test_step(D, where, kind):
    """Decoding: the other channels' states stay what they are."""
    B = 5
    at = dict(x=make((B, D), kind, 4), g=make((B, D), kind, 5), state=make((B + 1, D), "f32", 6))
    slots = i32([3, 0, 5, 1, 2])

    def run(v):
        out = v["state"].clone()
        return eg.engram_recurrence_step(v["x"], v["g"], slots, v["state"], state_out=out), out

    clean = run(at)
    bad = {k: v.clone() for k, v in at.items()}
    bad[where][1, 2] = bad[where][2, 7] = NAN
    y, out = run(bad)
    ny, no = torch.zeros_like(y, dtype=torch.bool), torch.zeros_like(out, dtype=torch.bool)
    rows = {0: 3, 1: 0, 2: 5, 3: 1, 4: 2}
    for b, s in rows.items():
        for r, c in ((1, 2), (2, 7)):
            if (s if where == "state" else b) == r:
                ny[b, c] = no[s, c] = True
    if where == "state":  # a slot that no entry names keeps what it holds
        no |= torch.isnan(bad["state"])
    assert torch.equal(torch.isnan(y), ny) and torch.equal(torch.isnan(out), no)
    assert torch.equal(y[~ny], clean[0][~ny]) and torch.equal(out[~no], clean[1][~no])
