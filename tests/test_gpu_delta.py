"""The gated delta rule on the GPU, whole sequences and token by token, against the 64-bit oracle."""
import pytest
import torch

import hashed_gram_conditional_gb300 as eg
from gpu_util import DEV, i32, i64, require_gpu, status
from oracle import blocks as OB

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
C = 64


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    require_gpu()


def make(shape, kind, seed, scale=1.0, shift=0.0):
    gen = torch.Generator(DEV).manual_seed(seed)
    return (torch.randn(shape, generator=gen, device=DEV) * scale + shift).to(TYPES[kind])


def unit(T, heads, d, kind, seed):
    x = make((T, heads, d), "f32", seed)
    return (x / x.norm(dim=2, keepdim=True)).to(TYPES[kind]).view(T, heads * d)


def inputs(T, keys, H, dk, dv, kind, seed, shift=3.0):
    return (unit(T, keys, dk, kind, seed), unit(T, keys, dk, kind, seed + 1), make((T, H * dv), kind, seed + 2),
            make((T, H), kind, seed + 3, 1.5, shift), make((T, H), kind, seed + 4))


def close(got, want, size, kind):
    """The states are sums of at most a few hundred fp32 terms of `size` (their largest value): 2^-15 of that is far
    above fp32's error of such sums and far below what a lost term, or one of bf16's 8 bits (2^-8), would show.  Outputs
    of type bf16 are then rounded, by at most 2^-8 of their value."""
    half = 2.0 ** -8 if kind == "bf16" else 0.0
    off = (got.double() - want).abs()
    tol = 2.0 ** -15 * size + half * want.abs() * (1 + 1e-6) + 1e-30
    assert (off <= tol).all(), (int((off > tol).sum()), float((off / tol).max()))


def d64(*ts):
    return [t.double() for t in ts]


def cuts(T, S, seed):
    gen = torch.Generator().manual_seed(seed)
    return [0] + sorted(torch.randint(0, T + 1, (S - 1,), generator=gen).tolist()) + [T]


def run(T, keys, H, dk, dv, cu, kind, seed, masked=0.0, state=False, scale=None, shift=3.0, given=None):
    q, k, v, g, b = given or inputs(T, keys, H, dk, dv, kind, seed, shift)
    S = len(cu) - 1
    gen = torch.Generator().manual_seed(seed)
    mask = (torch.rand(T, generator=gen) < masked).to(torch.uint8) if masked else None
    s0 = make((S + 2, H, dk, dv), "f32", seed + 5, 0.3) if state else None
    slots = torch.randperm(S + 2, generator=gen)[:S].tolist() if state else None
    st, out = status(), None if s0 is None else s0.clone()
    y = eg.engram_delta(q, k, v, g, b, i64(cu), keys, scale=scale, mask=None if mask is None else mask.to(DEV), state=s0,
                        slots=None if slots is None else i32(slots), state_out=out, status=st)
    assert int(st.item()) == 0
    want = OB.delta(*d64(q, k, v, g, b), cu, keys, dk ** -0.5 if scale is None else scale,
                    None if mask is None else mask.tolist(), None if s0 is None else s0.double(), slots)
    size = float(torch.maximum(v.double().abs().max(), want["before"].abs().max())) if T else 1.0
    close(y, want["y"], size * (dk ** -0.5 if scale is None else abs(scale)), kind)
    if s0 is not None:
        close(out, want["state"], max(size, 1.0), "f32")
    return y, out


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("T,keys,H,dk,dv", [(1, 1, 1, 1, 1), (2, 1, 1, 8, 8), (1, 2, 4, 128, 128), (17, 1, 2, 16, 24),
                                            (C - 1, 1, 1, 64, 64), (C, 2, 2, 64, 32), (C + 1, 1, 3, 128, 33), (200, 2, 4, 40, 72),
                                            (130, 1, 1, 127, 125), (3 * C, 1, 2, 65, 128), (500, 3, 3, 128, 128)])
def test_one_sequence(T, keys, H, dk, dv, kind):
    run(T, keys, H, dk, dv, [0, T], kind, 10)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("T,S,masked,state", [(300, 5, 0.0, True), (300, 40, 0.3, True), (257, 4, 0.1, False), (90, 90, 0.0, True),
                                              (40, 120, 0.2, True), (1, 5, 0.0, True), (400, 2, 0.95, True)])
def test_packed_sequences(T, S, masked, state, kind):
    """Ragged and empty sequences, masks and carried states."""
    run(T, 2, 4, 48, 40, cuts(T, S, S), kind, 30, masked, state)


@pytest.mark.parametrize("T,S,keys,H,dk,dv,masked,state", [(900, 10, 4, 8, 128, 128, 0.1, True), (700, 20, 2, 8, 64, 40, 0.0, True),
                                                           (300, 80, 1, 2, 33, 125, 0.3, True), (500, 1, 38, 76, 128, 24, 0.0, False),
                                                           (400, 2, 20, 40, 65, 128, 0.0, False), (130, 40, 2, 2, 8, 1, 0.0, True)])
def test_many_sequences_and_heads(T, S, keys, H, dk, dv, masked, state):
    """Where a block has four quads."""
    run(T, keys, H, dk, dv, cuts(T, S, S), "bf16", 35, masked, state)


def test_sequence_edges_at_chunk_edges():
    run(4 * C, 1, 2, 64, 64, [0, C - 1, C, C, C + 1, 2 * C, 3 * C + 1, 4 * C], "f32", 40, state=True)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_gates_at_their_ends(kind):
    """States that last and that are lost at once, and corrections of no and of full strength."""
    T, shape = 150, (1, 2, 32, 32)
    q, k, v, g, b = inputs(T, *shape, kind, 50)
    for shift_g, shift_b in ((14.0, 0.0), (-12.0, 3.0), (0.0, -14.0), (60.0, 60.0), (-60.0, -30.0)):
        run(T, *shape, [0, T], kind, 51, state=True, given=(q, k, v, g * 8 + shift_g, b + shift_b))


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_the_same_key_again(kind):
    """Each write overwrites the last one: (I + A) is as full as it gets."""
    T, shape = 200, (1, 1, 64, 64)
    q, k, v, g, b = inputs(T, *shape, kind, 60)
    k = k[:1].expand(T, -1).contiguous()
    run(T, *shape, [0, T], kind, 61, given=(k, k, v, g + 4.0, b + 4.0))


def test_columns_of_one_matrix_and_odd_alignment():
    T, keys, H, dk, dv = 100, 2, 4, 32, 24
    q, k, v, g, b = inputs(T, keys, H, dk, dv, "bf16", 70)
    want = eg.engram_delta(q, k, v, g, b, i64([0, 30, T]), keys)
    for gap in (8, 3):
        wide = torch.full((T, 3 * 96 + 6 * gap + 16), float("nan"), dtype=torch.bfloat16, device=DEV)
        at, cols = gap, []
        for t in (q, k, v, g, b):
            wide[:, at:at + t.shape[1]] = t
            cols.append(wide[:, at:at + t.shape[1]])
            at += t.shape[1] + gap
        out = torch.full((T, H * dv + 7), 5.0, dtype=torch.bfloat16, device=DEV)
        y = eg.engram_delta(*cols, i64([0, 30, T]), keys, y=out[:, 3:3 + H * dv])
        assert torch.equal(y, want)
        assert (out[:, :3] == 5).all() and (out[:, 3 + H * dv:] == 5).all()


def test_masked_and_padding_positions_may_hold_anything():
    T, keys, H, dk, dv = 200, 1, 2, 32, 32
    cu, slots = [0, 80, 110, 200], [1, -1, 0]
    clean = inputs(T, keys, H, dk, dv, "f32", 80)
    mask = torch.zeros(T, dtype=torch.uint8)
    mask[[0, 50, 79, 150, 199]] = 1
    junk = [t.clone() for t in clean]
    for t, x in zip(junk, (float("nan"), float("inf"), float("nan"), float("-inf"), float("nan"))):
        t[mask.bool().to(DEV)] = x
        t[80:110] = float("nan")
    s0 = make((2, H, dk, dv), "f32", 85)
    res = []
    for args in (clean, junk):
        out = s0.clone()
        y = eg.engram_delta(*args, i64(cu), keys, mask=mask.to(DEV), state=s0, slots=i32(slots), state_out=out)
        res.append((y, out))
    for u, w in zip(*res):
        assert torch.equal(u, w)
    assert (res[0][0][80:110] == 0).all() and (res[0][0][mask.bool().to(DEV)] == 0).all()


def test_nan_stays_in_its_sequence_and_head_from_its_chunk_on():
    T, keys, H, dk, dv = 300, 2, 2, 32, 32
    q, k, v, g, b = inputs(T, keys, H, dk, dv, "bf16", 90)
    cu = [0, 200, 300]
    want = eg.engram_delta(q, k, v, g, b, i64(cu), keys)
    v[100, 3] = float("nan")
    y = eg.engram_delta(q, k, v, g, b, i64(cu), keys)
    assert torch.equal(y[:C], want[:C]) and torch.equal(y[200:], want[200:])
    assert torch.equal(y[:, dv:], want[:, dv:])
    assert torch.isnan(y[100:200, 3]).all()


def test_slots_out_of_range_and_positions_outside():
    T, H, d = 60, 2, 16
    args = inputs(T, 1, H, d, d, "f32", 95)
    s0, st = make((2, H, d, d), "f32", 96), status()
    kept = s0.clone()
    y = torch.full((T, H * d), 9.0, device=DEV)
    eg.engram_delta(*args, i64([5, 20, 50]), 1, state=s0, slots=i32([2, 1]), y=y, status=st)
    assert int(st.item()) == eg.ST_BAD_SLOT
    assert (y[:5] == 9).all() and (y[50:] == 9).all() and (y[5:20] == 0).all()
    assert torch.equal(s0[0], kept[0]) and not torch.equal(s0[1], kept[1])


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("B,keys,H,dk,dv", [(1, 1, 1, 1, 1), (3, 2, 4, 128, 128), (5, 1, 3, 33, 40), (4, 2, 2, 64, 130 - 5),
                                            (70, 1, 2, 96, 32)])
def test_steps(B, keys, H, dk, dv, kind):
    """Three tokens one at a time, with padding, and the states of the slots that are not named."""
    S = B + 3
    s0 = make((S, H, dk, dv), "f32", 100, 0.3)
    gen = torch.Generator().manual_seed(B)
    slots = torch.randperm(S, generator=gen)[:B].tolist()
    if B > 2:
        slots[1] = -1
    ref, st = s0.double(), status()
    for n in range(3):
        args = inputs(B, keys, H, dk, dv, kind, 110 + n)
        before = ref.clone()
        y = eg.engram_delta_step(*args, i32(slots), s0, keys, status=st)
        want = OB.delta(*d64(*args), list(range(B + 1)), keys, dk ** -0.5, None, before, slots)
        ref = want["state"]
        size = max(1.0, float(args[2].double().abs().max()), float(before.abs().max()))
        close(y, want["y"], size * dk ** -0.5, kind)
        close(s0, ref, size, "f32")
    assert int(st.item()) == 0
    if B > 2:
        assert (y[1] == 0).all()
    out = torch.zeros_like(s0)
    kept = s0.clone()
    slots[0] = S
    args = inputs(B, keys, H, dk, dv, kind, 120)
    y = eg.engram_delta_step(*args, i32(slots), s0, keys, state_out=out, status=st)
    assert torch.equal(s0, kept) and int(st.item()) == eg.ST_BAD_SLOT and (y[0] == 0).all()
    named = [s for s in slots if 0 <= s < S]
    rest = [s for s in range(S) if s not in named]
    assert (out[rest] == 0).all()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_steps_follow_a_sequence(kind):
    """A prefill of the first positions, then token by token: the states are the whole sequence's."""
    T, n, keys, H, dk, dv = 90, 70, 1, 2, 64, 48
    args = inputs(T, keys, H, dk, dv, kind, 130)
    whole, parts = torch.zeros((1, H, dk, dv), device=DEV), torch.zeros((1, H, dk, dv), device=DEV)
    want = eg.engram_delta(*args, i64([0, T]), keys, state=whole)
    eg.engram_delta(*[t[:n] for t in args], i64([0, n]), keys, state=parts)
    for t in range(n, T):
        y = eg.engram_delta_step(*[x[t:t + 1] for x in args], i32([0]), parts, keys)
        size = float(args[2].float().abs().max()) * dk ** -0.5
        half = 2.0 ** -7 if kind == "bf16" else 0.0  # each side rounds
        assert ((y[0].float() - want[t].float()).abs() <= 2.0 ** -15 * size + half * want[t].float().abs()).all()
    assert (whole - parts).abs().max() <= 2.0 ** -15 * max(1.0, float(args[2].float().abs().max()))


def test_many_short_sequences():
    """More sequences than one block numbers at a time."""
    S = 2500
    lens = torch.randint(0, 4, (S,), generator=torch.Generator().manual_seed(1)).tolist()
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    run(cu[-1], 1, 1, 8, 8, cu, "f32", 140, state=True)


def test_many_short_sequences_of_several_heads():
    """The same where a block has four quads."""
    S = 1300
    lens = torch.randint(0, 3, (S,), generator=torch.Generator().manual_seed(2)).tolist()
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    run(cu[-1], 1, 2, 16, 24, cu, "bf16", 145, masked=0.1, state=True)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("T,S,H,masked", [(2000, 12, 40, 0.0), (1900, 5, 48, 0.1), (700, 60, 20, 0.0)])
def test_more_than_the_blocks_hold(T, S, H, masked, kind):
    """Sequences that go over from one block to the next, some of them after a few of their chunks; with the longest one
    much longer than the others, and with empty ones among them."""
    cu = cuts(T, S, 200 + S)
    run(T, 4, H, 16, 40, cu, kind, 200, masked=masked, state=True)
    cu = [0, T // 2] + [T // 2] * 3 + [T // 2 + k * (T // 2) // (S - 1) for k in range(1, S)]
    run(T, 4, H, 16, 40, cu, kind, 210, masked=masked)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_padding_among_more_than_the_blocks_hold(kind):
    """Sequences without a slot change where the others are cut, and none of their results; the backward pass likewise."""
    T, S, keys, H, dk, dv = 2500, 21, 4, 40, 16, 40
    args, cu = inputs(T, keys, H, dk, dv, kind, 220), [0] + list(range(61, T, 120))[:S - 1] + [T]
    dy, s0 = make((T, H * dv), kind, 229), make((S, H, dk, dv), "f32", 230, 0.3)
    slots = list(range(S))
    res = []
    for gone in ((), (0, 3, 4, 5, 11, S - 1)):
        sl = i32([-1 if s in gone else s for s in slots])
        out, ds, carry = s0.clone(), s0.clone(), eg.delta_carry(T, S, keys, H, dk, dv, DEV)
        y = eg.engram_delta(*args, i64(cu), keys, state=out, slots=sl, carry=carry)
        res.append((y, out, *eg.engram_delta_grad(dy, *args, carry, i64(cu), keys, slots=sl, dstate=ds), ds))
    kept = torch.ones(T, dtype=torch.bool)
    for s in gone:
        kept[cu[s]:cu[s + 1]] = False
    kept = kept.to(DEV)
    rest = [s for s in slots if s not in gone]
    for u, w in zip(*res):
        if u.dim() == 4:
            assert torch.equal(u[rest], w[rest]) and torch.equal(w[list(gone)], s0[list(gone)])
        else:
            assert torch.equal(u[kept], w[kept]) and (w[~kept] == 0).all()


def test_sequences_that_lie_over_one_another_stay_in_bounds():
    """They are no valid call: what they give is not defined, but nothing else is touched."""
    T, H, d = 300, 2, 16
    for S, kind in ((8, "bf16"), (200, "bf16"), (1500, "f32")):
        args = inputs(T, 1, H, d, d, kind, 99)
        cu = [0, T] * (S // 2) + [0]
        out = torch.full((T + 8, H * d), 9.0, dtype=TYPES[kind], device=DEV)
        states = torch.full((S + 2, H, d, d), 9.0, device=DEV)
        room, more = eg.delta_carry(T, S, 1, H, d, d, DEV).numel(), 1000
        carry = torch.full((room + more,), 9.0, device=DEV)
        size = eg.delta_workspace(T, S, 1, H, d, d, DEV).numel()
        space = torch.full((size + 4096,), 9, dtype=torch.uint8, device=DEV)
        eg.engram_delta(*args, i64(cu), 1, state=states[1:-1], y=out[4:-4], carry=carry[:room], workspace=space[:size])
        assert (out[:4] == 9).all() and (out[-4:] == 9).all() and (states[0] == 9).all() and (states[-1] == 9).all()
        assert (carry[room:] == 9).all() and (space[size:] == 9).all()


def test_two_calls_at_once():
    """Calls on two streams with workspaces of their own."""
    T, keys, H, dk, dv = 700, 2, 8, 128, 64
    sets, cu = [inputs(T, keys, H, dk, dv, "bf16", 155 + 9 * k) for k in range(2)], i64([0, 200, 700])
    want = [eg.engram_delta(*args, cu, keys) for args in sets]
    sides = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for side, args in zip(sides, sets):
            with torch.cuda.stream(side):
                got.append(eg.engram_delta(*args, cu, keys))
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_no_positions():
    H, d = 2, 8
    e = [torch.empty((0, n), device=DEV) for n in (d, d, H * d, H, H)]
    s0, out = make((2, H, d, d), "f32", 1), torch.zeros((2, H, d, d), device=DEV)
    y = eg.engram_delta(*e, i64([0, 0, 0]), 1, state=s0, state_out=out)
    assert y.shape == (0, H * d) and torch.equal(out, s0)
    assert eg.engram_delta(*e, i64([0]), 1).shape == (0, H * d)
    assert eg.engram_delta_step(*e, i32([]), s0, 1).shape == (0, H * d)


def test_runs_are_the_same_on_any_stream_and_in_a_graph():
    T, keys, H, dk, dv = 500, 2, 4, 128, 64
    args, cu = inputs(T, keys, H, dk, dv, "bf16", 150), i64([0, 200, 500])
    s0 = make((2, H, dk, dv), "f32", 151)
    want, out = [], s0.clone()
    want.append(eg.engram_delta(*args, cu, keys, state=out))
    want.append(out)
    side, got = torch.cuda.Stream(), s0.clone()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y = eg.engram_delta(*args, cu, keys, state=got)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, want[0]) and torch.equal(got, want[1])
    graph, got = torch.cuda.CUDAGraph(), s0.clone()
    step, slots = inputs(2, keys, H, dk, dv, "bf16", 160), i32([1, 0])
    with torch.cuda.graph(graph):
        y = eg.engram_delta(*args, cu, keys, state=got)
        z = eg.engram_delta_step(*step, slots, got, keys)
    graph.replay()
    assert torch.equal(y, want[0])
    assert torch.equal(z, eg.engram_delta_step(*step, slots, want[1], keys)) and torch.equal(got, want[1])


def test_the_binding_refuses():
    T, keys, H, dk, dv = 8, 2, 4, 16, 16
    q, k, v, g, b = inputs(T, keys, H, dk, dv, "bf16", 170)
    cu, s0 = i64([0, T]), make((1, H, dk, dv), "f32", 171)
    for bad in ((q, k, v, g, b, cu, 3), (q, k, v[:, :62], g, b, cu, 2), (q, k, v, g[:, :3], b, cu, 2), (q, k[:4], v, g, b, cu, 2)):
        with pytest.raises(ValueError):
            eg.engram_delta(*bad)
    with pytest.raises(TypeError):
        eg.engram_delta(q, k.float(), v, g, b, cu, keys)
    with pytest.raises(ValueError):
        eg.engram_delta(q, k, v, g, b, cu, keys, state=s0[:, :, :8].contiguous())
    with pytest.raises(ValueError):
        eg.engram_delta(q, k, v, g, b, i64([0, 4, T]), keys, state=s0)
    with pytest.raises(eg.EngramError):
        eg.engram_delta(q, k, v, g, b, cu, keys, scale=float("nan"))
    with pytest.raises(eg.EngramError):
        eg.engram_delta(q, k, v, g, b, i64([0]), keys)
    with pytest.raises(eg.EngramError):
        eg.engram_delta(q, k, v, g, b, cu, keys, workspace=torch.empty(256, dtype=torch.uint8, device=DEV))
    wide = make((T, 129 * 2), "bf16", 1)
    with pytest.raises(eg.EngramError):
        eg.engram_delta(wide, wide, v, g, b, cu, 2)
