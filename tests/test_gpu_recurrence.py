"""The gated linear recurrence, its gradients and its one-position step on the GPU against the 64-bit oracle."""
import numpy as np
import pytest
import torch

import hashed_gram_conditional_gb300 as eg
from gpu_util import DEV, i32, i64, require_gpu, status
from oracle import training as OT

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
TILE = 128


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    require_gpu()


def make(shape, kind, seed, scale=1.0, shift=0.0):
    rng = np.random.default_rng(seed)
    return torch.from_numpy(rng.normal(size=shape) * scale + shift).to(torch.float32).to(TYPES[kind]).to(DEV)


def f64(t):
    return t.double().cpu().numpy()


def close(got, want, err, kind):
    """Within the fp32 error bound, and for bf16 (8 significant bits) the final rounding's 2^-8."""
    half = 2.0 ** -8 if kind == "bf16" else 0.0
    g = f64(got)
    tol = err * (1 + half) + half * np.abs(want) * (1 + 1e-6) + 1e-40
    bad = ~(np.abs(g - want) <= tol)
    assert not bad.any(), (int(bad.sum()), float(np.abs(g - want)[bad].max()), float(tol[bad].min()))


def cuts(T, S, seed):
    rng = np.random.default_rng(seed)
    return [0] + sorted(rng.integers(0, T + 1, S - 1).tolist()) + [T]


def run_both(T, D, cu, kind, seed, masked=0.0, state=False, grad_state=False, shift=1.0, spread=1.5):
    x, g, dy = make((T, D), kind, seed), make((T, D), kind, seed + 1, spread, shift), make((T, D), kind, seed + 2)
    S = len(cu) - 1
    rng = np.random.default_rng(seed + 3)
    mask = (rng.random(T) < masked).astype(np.uint8) if masked else None
    slots = rng.permutation(S + 2)[:S] if state or grad_state else None
    s0 = make((S + 2, D), "f32", seed + 4) if state else None
    ds = make((S + 2, D), "f32", seed + 5) if grad_state else None
    m = None if mask is None else torch.from_numpy(mask).to(DEV)
    sl = None if slots is None else i32(slots)
    carry = eg.recurrence_carry(T, D, DEV)
    out = None if s0 is None else s0.clone()
    st = status()
    y = eg.engram_recurrence(x, g, i64(cu), mask=m, state=s0, slots=sl, state_out=out, carry=carry, status=st)
    back = None if ds is None else ds.clone()
    dx, dg = eg.engram_recurrence_grad(dy, x, g, carry, i64(cu), mask=m, state=s0, slots=sl, dstate=back, status=st)
    assert int(st.item()) == 0
    a = dict(mask=mask, state=None if s0 is None else f64(s0), slots=None if slots is None else slots.tolist())
    want = OT.recurrence(f64(x), f64(g), cu, **a)
    close(y, want["y"], want["y_err"], kind)
    if s0 is not None:
        close(out, want["state"], want["state_err"], "f32")
    gw = OT.recurrence_grad(f64(dy), f64(x), f64(g), cu, dstate=None if ds is None else f64(ds), **a)
    close(dx, gw["dx"], gw["dx_err"], kind)
    close(dg, gw["dg"], gw["dg_err"], kind)
    if ds is not None:
        close(back, gw["dstate"], gw["dstate_err"], "f32")
    return y, dx, dg


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("T,D", [(1, 1), (1, 256), (2, 7), (TILE - 1, 64), (TILE, 130), (TILE + 1, 80), (3 * TILE, 8),
                                 (1000, 33), (2500, 264)])
def test_one_sequence(T, D, kind):
    run_both(T, D, [0, T], kind, 10)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("T,D,S,masked,state,grad_state",
                         [(700, 72, 9, 0.0, True, True), (700, 40, 60, 0.3, True, True), (513, 257, 4, 0.1, False, False),
                          (300, 16, 300, 0.0, True, False), (40, 8, 90, 0.2, True, True), (1, 16, 5, 0.0, True, True),
                          (600, 24, 3, 0.95, False, True), (1500, 520, 2, 0.05, True, True)])
def test_packed_sequences(T, D, S, masked, state, grad_state, kind):
    """Ragged and empty sequences (several in a tile, one over many), masks, states and their gradients."""
    run_both(T, D, cuts(T, S, 20 + S), kind, 30, masked, state, grad_state)


def test_sequence_edges_at_tile_edges():
    run_both(4 * TILE, 24, [0, TILE - 1, TILE, TILE, TILE + 1, 2 * TILE, 3 * TILE + 1, 4 * TILE], "f32", 40, 0.0, True,
             True)


def test_long_memory_and_closed_gates():
    """Gates that round to one (the state lasts through many tiles) and to zero."""
    run_both(3000, 16, [0, 3000], "f32", 50, shift=14.0, spread=0.5)
    run_both(3000, 16, [0, 1400, 3000], "bf16", 51, state=True, shift=9.0, spread=1.0)
    run_both(400, 16, [0, 400], "f32", 52, shift=-30.0, spread=20.0)
    run_both(400, 16, [0, 400], "f32", 53, shift=0.0, spread=60.0)


def test_everything_masked():
    T, D = 300, 40
    x, g = make((T, D), "bf16", 60), make((T, D), "bf16", 61)
    s0 = make((1, D), "f32", 62)
    m = torch.ones(T, dtype=torch.uint8, device=DEV)
    out, carry = torch.zeros_like(s0), eg.recurrence_carry(T, D, DEV)
    y = eg.engram_recurrence(x, g, i64([0, T]), mask=m, state=s0, state_out=out, carry=carry)
    assert (y == 0).all() and torch.equal(out, s0)
    ds = make((1, D), "f32", 63)
    want = ds.clone()
    dx, dg = eg.engram_recurrence_grad(make((T, D), "bf16", 64), x, g, carry, i64([0, T]), mask=m, state=s0, dstate=ds)
    assert (dx == 0).all() and (dg == 0).all() and torch.equal(ds, want)


def test_masked_and_padding_positions_may_hold_anything():
    """NaN and infinities in masked positions and padding sequences reach nothing."""
    T, D = 260, 24
    cu = [0, 100, 130, 260]
    x, g, dy = (make((T, D), "f32", 70 + k) for k in range(3))
    mask = np.zeros(T, np.uint8)
    mask[[0, 50, 99, 200, 259]] = 1
    slots = [1, -1, 0]
    junk = [t.clone() for t in (x, g, dy)]
    for t, v in zip(junk, (float("nan"), float("inf"), float("nan"))):
        t[torch.from_numpy(mask).to(DEV).bool()] = v
        t[100:130] = float("nan")
    s0 = make((2, D), "f32", 74)
    res = []
    for a, b, c in ((x, g, dy), tuple(junk)):
        carry, out, ds = eg.recurrence_carry(T, D, DEV), s0.clone(), s0.clone()
        m = torch.from_numpy(mask).to(DEV)
        y = eg.engram_recurrence(a, b, i64(cu), mask=m, state=s0, slots=i32(slots), state_out=out, carry=carry)
        dx, dg = eg.engram_recurrence_grad(c, a, b, carry, i64(cu), mask=m, state=s0, slots=i32(slots), dstate=ds)
        res.append((y, out, dx, dg, ds))
    for u, v in zip(*res):
        assert torch.equal(u, v)
    assert (res[0][0][100:130] == 0).all() and (res[0][2][100:130] == 0).all()


def test_nan_stays_in_its_sequence_and_channel():
    T, D = 300, 32
    x, g = make((T, D), "f32", 80), make((T, D), "f32", 81)
    x[140, 5] = float("nan")
    y = eg.engram_recurrence(x, g, i64([0, 130, 290, 300]))
    nan = torch.isnan(y)
    want = torch.zeros_like(nan)
    want[140:290, 5] = True
    assert torch.equal(nan, want)


def test_strides_and_alignment():
    """x and g as column ranges of one matrix, outputs inside wider ones, odd offsets."""
    T, D = 333, 50
    for kind in ("bf16", "f32"):
        both = make((T, 2 * D + 3), kind, 90)
        x, g = both[:, 1:1 + D], both[:, 1 + D:1 + 2 * D]
        dyw = make((T, D + 5), kind, 91)
        cu = i64([0, 150, T])
        outs = [torch.full((T, D + 7), 9.0, dtype=TYPES[kind], device=DEV) for _ in range(3)]
        y, dx, dg = (o[:, 3:3 + D] for o in outs)
        carry = eg.recurrence_carry(T, D, DEV)
        eg.engram_recurrence(x, g, cu, y=y, carry=carry)
        eg.engram_recurrence_grad(dyw[:, 2:2 + D], x, g, carry, cu, dx=dx, dg=dg)
        c2 = eg.recurrence_carry(T, D, DEV)
        wy = eg.engram_recurrence(x.contiguous(), g.contiguous(), cu, carry=c2)
        wdx, wdg = eg.engram_recurrence_grad(dyw[:, 2:2 + D].contiguous(), x.contiguous(), g.contiguous(), c2, cu)
        assert torch.equal(y, wy) and torch.equal(dx, wdx) and torch.equal(dg, wdg)
        for o in outs:
            assert (o[:, :3] == 9).all() and (o[:, 3 + D:] == 9).all()


def test_chunks_continue_one_another():
    """Two chunks with the state carried against one pass, and the same once more by single positions."""
    T, D, cut = 400, 48, 211
    x, g = make((T, D), "f32", 100), make((T, D), "f32", 101, 1.5, 1.0)
    want = OT.recurrence(f64(x), f64(g), [0, T])
    state = torch.zeros((1, D), device=DEV)
    a = eg.engram_recurrence(x[:cut], g[:cut], i64([0, cut]), state=state)
    b = eg.engram_recurrence(x[cut:], g[cut:], i64([0, T - cut]), state=state)
    close(torch.cat([a, b]), want["y"], want["y_err"], "f32")
    state.zero_()
    slot = i32([0])
    ys = torch.cat([eg.engram_recurrence_step(x[t:t + 1], g[t:t + 1], slot, state) for t in range(T)])
    close(ys, want["y"], want["y_err"], "f32")


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("B,D", [(1, 1), (1, 1280), (3, 77), (256, 512), (1000, 8), (70000, 3)])
def test_step(B, D, kind):
    x, g = make((B, D), kind, 110), make((B, D), kind, 111, 2.0)
    state = make((B + 3, D), "f32", 112)
    rng = np.random.default_rng(113)
    slots = rng.permutation(B + 3)[:B]
    slots[rng.random(B) < 0.1] = -1
    want_state = f64(state)
    f, u = OT.sigmoid(f64(g)), OT.sigmoid(-f64(g))
    live = slots >= 0
    s0 = np.where(live[:, None], want_state[np.maximum(slots, 0)], 0.0)
    want = np.where(live[:, None], f * s0 + u * f64(x), 0.0)
    fe, ue = OT._gate_err(f64(g))
    err = np.where(live[:, None], fe * f * np.abs(s0) + ue * u * np.abs(f64(x)) + 2 * OT.UNIT * np.abs(want), 0.0)
    want_state[slots[live]] = want[live]
    serr = np.zeros_like(want_state)
    serr[slots[live]] = err[live]
    keep = state.clone()
    out = state.clone()
    y = eg.engram_recurrence_step(x, g, i32(slots), state, state_out=out)
    assert torch.equal(state, keep)  # the old states stay
    close(y, want, err, kind)
    close(out, want_state, serr, "f32")
    y2 = eg.engram_recurrence_step(x, g, i32(slots), state)
    assert torch.equal(y, y2) and torch.equal(state, out)


def test_bad_slots():
    T, D = 50, 16
    x, g = make((T, D), "f32", 120), make((T, D), "f32", 121)
    state = make((2, D), "f32", 122)
    keep = state.clone()
    st = status()
    y = eg.engram_recurrence(x, g, i64([0, 20, T]), state=state, slots=i32([2, 1]), status=st)
    assert int(st.item()) == eg.ST_BAD_SLOT and (y[:20] == 0).all() and torch.equal(state[0], keep[0])
    assert not torch.equal(state[1], keep[1])
    st.zero_()
    y = eg.engram_recurrence_step(x[:2], g[:2], i32([5, 0]), state, status=st)
    assert int(st.item()) == eg.ST_BAD_SLOT and (y[0] == 0).all() and (y[1] != 0).any()


def test_no_positions():
    D = 8
    e = torch.empty((0, D), device=DEV)
    s0, out = make((2, D), "f32", 130), torch.zeros((2, D), device=DEV)
    assert eg.engram_recurrence(e, e, i64([0])).shape == (0, D)
    assert eg.engram_recurrence(e, e, i64([0, 0, 0]), state=s0, state_out=out).shape == (0, D)
    assert torch.equal(out, s0)
    ds = s0.clone()
    carry = eg.recurrence_carry(0, D, DEV)
    dx, dg = eg.engram_recurrence_grad(e, e, e, carry, i64([0, 0, 0]), dstate=ds)
    assert dx.shape == (0, D) and torch.equal(ds, s0)
    assert eg.engram_recurrence_step(e, e, i32([]), s0).shape == (0, D)


def test_gradients_against_differences():
    """Directional derivatives of the 64-bit forward pass, by central differences."""
    T, D, cu = 200, 6, [0, 70, 70, 200]
    x, g, dy = make((T, D), "f32", 140), make((T, D), "f32", 141, 1.0, 1.0), make((T, D), "f32", 142)
    s0, ds = make((3, D), "f32", 143), make((3, D), "f32", 144)
    carry = eg.recurrence_carry(T, D, DEV)
    eg.engram_recurrence(x, g, i64(cu), state=s0, state_out=torch.zeros_like(s0), carry=carry)
    back = ds.clone()
    dx, dg = eg.engram_recurrence_grad(dy, x, g, carry, i64(cu), state=s0, dstate=back)
    rng = np.random.default_rng(145)
    at = [f64(x), f64(g), f64(s0)]

    def value(a):
        r = OT.recurrence(a[0], a[1], cu, None, a[2])
        return (r["y"] * f64(dy)).sum() + (r["state"] * f64(ds)).sum()

    for k, grad in enumerate((dx, dg, back)):
        v = rng.normal(size=at[k].shape)
        h = 1e-5
        up, down = list(at), list(at)
        up[k], down[k] = at[k] + h * v, at[k] - h * v
        want = (value(up) - value(down)) / (2 * h)
        size = np.abs(f64(grad) * v).sum()
        # fp32 rounding of the gradients (a few hundred units at most) and the differences' own error
        assert abs((f64(grad) * v).sum() - want) <= 300 * OT.UNIT * size + 1e-7 * (1 + size)


def test_long_sequence_against_single_positions_and_run_to_run():
    """Many tiles in flight: the scan repeats bit for bit, and agrees with the recurrence walked in 64 bits."""
    T, D = 40_000, 96
    x, g = make((T, D), "bf16", 150), make((T, D), "bf16", 151, 1.5, 3.0)
    carry = eg.recurrence_carry(T, D, DEV)
    y = eg.engram_recurrence(x, g, i64([0, T]), carry=carry).clone()
    c0 = carry.clone()
    for _ in range(5):
        assert torch.equal(y, eg.engram_recurrence(x, g, i64([0, T]), carry=carry)) and torch.equal(c0, carry)
    want = OT.recurrence(f64(x), f64(g), [0, T])
    close(y, want["y"], want["y_err"], "bf16")
    dy = make((T, D), "bf16", 152)
    first = [t.clone() for t in eg.engram_recurrence_grad(dy, x, g, carry, i64([0, T]))]
    for _ in range(5):
        for a, b in zip(first, eg.engram_recurrence_grad(dy, x, g, carry, i64([0, T]))):
            assert torch.equal(a, b)


def test_on_another_stream_and_in_a_graph():
    T, D = 1000, 64
    x, g = make((T, D), "bf16", 160), make((T, D), "bf16", 161)
    cu = i64([0, 400, T])
    want = eg.engram_recurrence(x, g, cu)
    y, ws = torch.empty_like(want), eg.recurrence_workspace(T, D, DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        eg.engram_recurrence(x, g, cu, y=y, workspace=ws)
    s.synchronize()
    assert torch.equal(y, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        eg.engram_recurrence(x, g, cu, y=y, workspace=ws)
    for _ in range(3):
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)


def test_rows_past_four_giga_elements():
    """Row offsets beyond 2^32 elements: columns of a very wide matrix, against the same values packed."""
    T, D, wide = 66_000, 8, 66_000
    big = torch.empty((T, wide), dtype=torch.bfloat16, device=DEV)
    x, g, dy = make((T, D), "bf16", 180), make((T, D), "bf16", 181, 1.0, 2.0), make((T, D), "bf16", 182)
    parts = [big[:, k * 64:k * 64 + D] for k in range(6)]
    for p, t in zip(parts, (x, g, dy)):
        p.copy_(t)
    cu = i64([0, 30_000, T])
    c1, c2 = eg.recurrence_carry(T, D, DEV), eg.recurrence_carry(T, D, DEV)
    y = eg.engram_recurrence(x, g, cu, carry=c1)
    dx, dg = eg.engram_recurrence_grad(dy, x, g, c1, cu)
    eg.engram_recurrence(parts[0], parts[1], cu, y=parts[3], carry=c2)
    assert torch.equal(parts[3], y)
    eg.engram_recurrence_grad(parts[2], parts[0], parts[1], c2, cu, dx=parts[4], dg=parts[5])
    assert torch.equal(parts[4], dx) and torch.equal(parts[5], dg)


def test_refusals():
    x = make((4, 8), "bf16", 170)
    cu = i64([0, 4])
    with pytest.raises(TypeError):
        eg.engram_recurrence(x, x.float(), cu)
    with pytest.raises(TypeError):
        eg.engram_recurrence(x, x, cu.int())
    with pytest.raises(ValueError):
        eg.engram_recurrence(x, x[:3], cu)
    with pytest.raises(ValueError):
        eg.engram_recurrence(x, x, cu, state=torch.zeros((1, 9), device=DEV))
    with pytest.raises(ValueError):
        eg.engram_recurrence(x, x, i64([0, 2, 4]), state=torch.zeros((1, 8), device=DEV))  # two sequences, one state
    with pytest.raises(ValueError):
        eg.engram_recurrence(x, x, cu, y=torch.empty((8, 4), dtype=torch.bfloat16, device=DEV).t())
    with pytest.raises(ValueError):
        eg.engram_recurrence_grad(x, x, x, torch.empty(4, device=DEV), cu)
    with pytest.raises(eg.EngramError, match="RANGE"):
        eg.engram_recurrence(x, x, cu, workspace=torch.empty(256, dtype=torch.uint8, device=DEV)[:8])
    with pytest.raises(ValueError):
        eg.engram_recurrence_step(x, x, i32([0, 1, 2, 3]), torch.zeros((4, 9), device=DEV))
