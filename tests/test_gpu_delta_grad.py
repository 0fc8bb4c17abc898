"""The gated delta rule's gradients on the GPU against the 64-bit oracle and against differences."""
import pytest
import torch

import hashed_gram_conditional_gb300 as eg
from gpu_util import DEV, i32, i64, require_gpu, status
from oracle import blocks as OB
from test_gpu_delta import C, cuts, d64, inputs, make

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    require_gpu()


def close(got, want, size, kind):
    """`size` is what the sum behind a gradient comes to if its terms' signs are independent, from the largest values of its
    factors.  Products on the way keep 16 bits at least (2^-17 a factor, and a few such products follow one another): 2^-14
    of the size, with half of a bf16 step for the output."""
    half = 2.0 ** -8 if kind == "bf16" else 0.0
    off = (got.double() - want).abs()
    tol = 2.0 ** -14 * size + half * want.abs() * (1 + 1e-6) + 1e-30
    assert (off <= tol).all(), (int((off > tol).sum()), float((off / tol).max()))


def run(T, keys, H, dk, dv, cu, kind, seed, masked=0.0, state=False, scale=None, shift=3.0, given=None, slots=None):
    args = given or inputs(T, keys, H, dk, dv, kind, seed, shift)
    dy = make((T, H * dv), kind, seed + 9)
    S = len(cu) - 1
    gen = torch.Generator().manual_seed(seed)
    mask = (torch.rand(T, generator=gen) < masked).to(torch.uint8) if masked else None
    s0 = make((S + 2, H, dk, dv), "f32", seed + 5, 0.3) if state else None
    ds = make((S + 2, H, dk, dv), "f32", seed + 6, 0.3) if state else None
    slots = torch.randperm(S + 2, generator=gen)[:S].tolist() if state and slots is None else slots
    m, sl = None if mask is None else mask.to(DEV), None if slots is None else i32(slots)
    carry, st = eg.delta_carry(T, S, keys, H, dk, dv, DEV), status()
    out = None if s0 is None else s0.clone()
    y = eg.engram_delta(*args, i64(cu), keys, scale=scale, mask=m, state=s0, slots=sl, state_out=out, carry=carry, status=st)
    back = None if ds is None else ds.clone()
    got = eg.engram_delta_grad(dy, *args, carry, i64(cu), keys, scale=scale, mask=m, slots=sl, dstate=back, status=st)
    assert int(st.item()) == 0
    f = dk ** -0.5 if scale is None else scale
    want = OB.delta_grad(*d64(dy, *args), cu, keys, f, None if mask is None else mask.tolist(),
                         None if s0 is None else s0.double(), slots, None if ds is None else ds.double())
    Y, G, R = abs(f) * float(dy.double().abs().max()), want["reach"], max(want["held"], 1.0)
    share = (H // keys) ** 0.5
    sizes = dict(dq=share * dv ** 0.5 * Y * R, dk=share * dv ** 0.5 * G * R, dv=G, dg=(dk * dv) ** 0.5 * G * R,
                 db=dv ** 0.5 * G * R)
    for (name, size), t in zip(sizes.items(), got):
        close(t, want[name], size, kind)
    if ds is not None:
        close(back, want["dstate"], max(G, 1.0), "f32")
    return y, got, back


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("T,keys,H,dk,dv", [(1, 1, 1, 1, 1), (2, 1, 1, 8, 8), (1, 2, 4, 128, 128), (17, 1, 2, 16, 24),
                                            (C - 1, 1, 1, 64, 64), (C, 2, 2, 64, 32), (C + 1, 1, 3, 128, 33), (200, 2, 4, 40, 72),
                                            (130, 1, 1, 127, 125), (3 * C, 1, 2, 65, 128), (300, 2, 6, 128, 128)])
def test_one_sequence(T, keys, H, dk, dv, kind):
    run(T, keys, H, dk, dv, [0, T], kind, 10)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("T,S,masked,state", [(300, 5, 0.0, True), (300, 40, 0.3, True), (257, 4, 0.1, False), (90, 90, 0.0, True),
                                              (40, 120, 0.2, True), (1, 5, 0.0, True), (400, 2, 0.95, True)])
def test_packed_sequences(T, S, masked, state, kind):
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
    T, shape = 150, (1, 2, 32, 32)
    q, k, v, g, b = inputs(T, *shape, kind, 50)
    for shift_g, shift_b in ((14.0, 0.0), (-12.0, 3.0), (0.0, -14.0), (60.0, 60.0), (-60.0, -30.0)):
        run(T, *shape, [0, T], kind, 51, state=True, given=(q, k, v, g * 8 + shift_g, b + shift_b))


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_the_same_key_again(kind):
    T, shape = 200, (1, 1, 64, 64)
    q, k, v, g, b = inputs(T, *shape, kind, 60)
    k = k[:1].expand(T, -1).contiguous()
    run(T, *shape, [0, T], kind, 61, given=(k, k, v, g + 4.0, b + 4.0))


def test_gradients_by_differences():
    T, keys, H, dk, dv, cu = 150, 1, 2, 16, 24, [0, 70, 150]
    args = inputs(T, keys, H, dk, dv, "f32", 70)
    s0, dy, ds = make((2, H, dk, dv), "f32", 71, 0.3), make((T, H * dv), "f32", 72), make((2, H, dk, dv), "f32", 73, 0.3)
    carry = eg.delta_carry(T, 2, keys, H, dk, dv, DEV)
    eg.engram_delta(*args, i64(cu), keys, state=s0, state_out=torch.empty_like(s0), carry=carry)
    back = ds.clone()
    got = eg.engram_delta_grad(dy, *args, carry, i64(cu), keys, dstate=back)

    def total(*a):
        r = OB.delta(*a[:5], cu, keys, dk ** -0.5, None, a[5])
        return (r["y"] * dy.double()).sum() + (r["state"] * ds.double()).sum()
    full = d64(*args, s0)
    for i, grad in enumerate((*got, back)):
        d = torch.randn(full[i].shape, dtype=torch.float64, device=DEV, generator=torch.Generator(DEV).manual_seed(i))
        up, down = list(full), list(full)
        up[i], down[i] = full[i] + 1e-5 * d, full[i] - 1e-5 * d
        want = float(total(*up) - total(*down)) / 2e-5
        size = float((grad.double() * d).abs().sum())
        assert abs(float((grad.double() * d).sum()) - want) <= 1e-5 * size + 1e-6, i


def test_masked_and_padding_positions_may_hold_anything():
    T, keys, H, dk, dv = 200, 1, 2, 32, 32
    cu, slots = [0, 80, 110, 200], [1, -1, 0]
    clean = [*inputs(T, keys, H, dk, dv, "f32", 80), make((T, H * dv), "f32", 86)]
    mask = torch.zeros(T, dtype=torch.uint8)
    mask[[0, 50, 79, 150, 199]] = 1
    junk = [t.clone() for t in clean]
    for t, x in zip(junk, (float("nan"), float("inf"), float("nan"), float("-inf"), float("nan"), float("inf"))):
        t[mask.bool().to(DEV)] = x
        t[80:110] = float("nan")
    s0, res, m = make((2, H, dk, dv), "f32", 85), [], mask.to(DEV)
    for *args, dy in (clean, junk):
        carry, ds = eg.delta_carry(T, 3, keys, H, dk, dv, DEV), s0.clone()
        eg.engram_delta(*args, i64(cu), keys, mask=m, state=s0, slots=i32(slots), state_out=s0.clone(), carry=carry)
        grads = eg.engram_delta_grad(dy, *args, carry, i64(cu), keys, mask=m, slots=i32(slots), dstate=ds)
        res.append((*grads, ds))
    for u, w in zip(*res):
        assert torch.equal(u, w)
    for t in res[0][:5]:
        assert (t[80:110] == 0).all() and (t[m.bool()] == 0).all()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_everything_masked(kind):
    T, keys, H, dk, dv, cu = 150, 1, 2, 32, 24, i64([0, 90, 150])
    args, dy = inputs(T, keys, H, dk, dv, kind, 87), make((T, H * dv), kind, 88)
    s0, ds = make((2, H, dk, dv), "f32", 89), make((2, H, dk, dv), "f32", 90)
    m, out, carry = torch.ones(T, dtype=torch.uint8, device=DEV), torch.zeros_like(s0), eg.delta_carry(T, 2, keys, H, dk, dv, DEV)
    y = eg.engram_delta(*args, cu, keys, mask=m, state=s0, state_out=out, carry=carry)
    assert (y == 0).all() and torch.equal(out, s0)
    back = ds.clone()
    grads = eg.engram_delta_grad(dy, *args, carry, cu, keys, mask=m, dstate=back)
    assert all((g == 0).all() for g in grads) and torch.equal(back, ds)


def test_arrays_past_two_to_the_31_elements():
    """The last sequence of arrays of 2^31 values and more gives what it gives alone."""
    H, d, n = 64, 128, 300
    T = 2 ** 31 // (H * d) + 1000
    if torch.cuda.mem_get_info()[0] < 90 << 30:
        pytest.skip("needs 90 GB of device memory")
    gen = torch.Generator(DEV).manual_seed(7)
    q, k = (torch.randn((T, 16), generator=gen, device=DEV).mul_(0.25).bfloat16() for _ in range(2))
    g, b = (torch.randn((T, H), generator=gen, device=DEV).bfloat16() for _ in range(2))
    v, dy = (torch.empty((T, H * d), dtype=torch.bfloat16, device=DEV).normal_(generator=gen) for _ in range(2))
    args, cu = (q, k, v, g, b), i64([0, 1000, T - n, T])
    carry = eg.delta_carry(T, 3, 1, H, 16, d, DEV)
    y = eg.engram_delta(*args, cu, 1, carry=carry)
    got = eg.engram_delta_grad(dy, *args, carry, cu, 1)
    last = [t[T - n:].contiguous() for t in args]
    carry = eg.delta_carry(n, 2, 1, H, 16, d, DEV)
    cu = i64([0, 0, n])
    assert torch.equal(y[T - n:], eg.engram_delta(*last, cu, 1, carry=carry))
    for u, w in zip(got, eg.engram_delta_grad(dy[T - n:].contiguous(), *last, carry, cu, 1)):
        assert torch.equal(u[T - n:], w)


def test_outputs_between_other_columns_and_positions_outside():
    T, keys, H, dk, dv, cu = 100, 2, 4, 32, 24, [10, 40, 90]
    args, dy = inputs(T, keys, H, dk, dv, "bf16", 90), make((T, H * dv), "bf16", 95)
    carry = eg.delta_carry(T, 2, keys, H, dk, dv, DEV)
    eg.engram_delta(*args, i64(cu), keys, carry=carry)
    outs = [torch.full((T, t.shape[1] + 5), 3.0, dtype=torch.bfloat16, device=DEV) for t in args]
    views = [o[:, 2:2 + t.shape[1]] for o, t in zip(outs, args)]
    got = eg.engram_delta_grad(dy, *args, carry, i64(cu), keys, **dict(zip(("dq", "dk", "dv", "dg", "db"), views)))
    want = eg.engram_delta_grad(dy, *args, carry, i64(cu), keys)
    for u, w, o in zip(got, want, outs):
        assert torch.equal(u[10:90], w[10:90])
        assert (u[:10] == 3).all() and (u[90:] == 3).all() and (o[:, :2] == 3).all() and (o[:, -3:] == 3).all()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("T,S,H,masked", [(2000, 12, 40, 0.0), (1900, 5, 48, 0.1), (700, 60, 20, 0.0)])
def test_more_than_the_blocks_hold(T, S, H, masked, kind):
    run(T, 4, H, 16, 40, cuts(T, S, 200 + S), kind, 200, masked=masked, state=True)


@pytest.mark.parametrize("S,keys,H,dk,dv,kind", [(1300, 1, 2, 16, 24, "bf16"), (1100, 1, 1, 8, 8, "f32")])
def test_many_short_sequences(S, keys, H, dk, dv, kind):
    """More sequences than one block numbers at a time."""
    cu = [0]
    for n in torch.randint(0, 3, (S,), generator=torch.Generator().manual_seed(3)).tolist():
        cu.append(cu[-1] + n)
    run(cu[-1], keys, H, dk, dv, cu, kind, 97, masked=0.1, state=True)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("T,keys,H,dk,dv", [(130, 1, 2, 32, 40), (90, 2, 2, 128, 64)])
def test_a_carry_within_a_larger_one(T, keys, H, dk, dv, kind):
    """What is kept may lie at any multiple of 16 bytes; the last sequence ends inside a chunk."""
    args, dy, cu = inputs(T, keys, H, dk, dv, kind, 98), make((T, H * dv), kind, 99), i64([0, 70, T])
    room, want = eg.delta_carry(T, 2, keys, H, dk, dv, DEV).numel(), None
    for shift in (0, 4, 8):
        carry = torch.full((room + 12,), 7.0, device=DEV)
        part = carry[shift:shift + room]
        eg.engram_delta(*args, cu, keys, carry=part)
        got = eg.engram_delta_grad(dy, *args, part, cu, keys)
        want = got if want is None else want
        for u, w in zip(got, want):
            assert torch.equal(u, w)
        assert (carry[:shift] == 7).all() and (carry[shift + room:] == 7).all()
    for call in (lambda c: eg.engram_delta(*args, cu, keys, carry=c), lambda c: eg.engram_delta_grad(dy, *args, c, cu, keys)):
        with pytest.raises(eg.EngramError):
            call(carry[1:1 + room])


def test_captured_beside_an_eager_backward_pass():
    """Forward and backward in a graph, replayed on other inputs; results are the same from run to run."""
    T, keys, H, dk, dv, cu = 300, 2, 4, 128, 64, i64([0, 130, 300])
    args, dy = inputs(T, keys, H, dk, dv, "bf16", 100), make((T, H * dv), "bf16", 105)

    def both():
        carry = eg.delta_carry(T, 2, keys, H, dk, dv, DEV)
        y = eg.engram_delta(*args, cu, keys, carry=carry)
        return (y, *eg.engram_delta_grad(dy, *args, carry, cu, keys))
    both()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    for t, new in zip((*args, dy), (*inputs(T, keys, H, dk, dv, "bf16", 110), make((T, H * dv), "bf16", 115))):
        t.copy_(new)
    want = both()
    graph.replay()
    for u, w in zip(got, want):
        assert torch.equal(u, w)


def test_no_positions_and_refusals():
    H, d = 2, 8
    e = [torch.empty((0, n), device=DEV) for n in (d, d, H * d, H, H)]
    ds = make((2, H, d, d), "f32", 1)
    kept = ds.clone()
    got = eg.engram_delta_grad(torch.empty((0, H * d), device=DEV), *e, torch.empty(1, device=DEV), i64([0, 0, 0]), 1, dstate=ds)
    assert [t.shape[0] for t in got] == [0] * 5 and torch.equal(ds, kept)
    T = 8
    args, dy = inputs(T, 1, H, d, d, "bf16", 120), make((T, H * d), "bf16", 125)
    carry = eg.delta_carry(T, 1, 1, H, d, d, DEV)
    with pytest.raises(ValueError):
        eg.engram_delta_grad(dy[:4], *args, carry, i64([0, T]), 1)
    with pytest.raises(ValueError):
        eg.engram_delta_grad(dy, *args, carry[:-1], i64([0, T]), 1)
    with pytest.raises(TypeError):
        eg.engram_delta_grad(dy.float(), *args, carry, i64([0, T]), 1)
    with pytest.raises(ValueError):
        eg.engram_delta_grad(dy, *args, carry, i64([0, T]), 1, dg=torch.empty((T, H + 1), device=DEV, dtype=dy.dtype))
    with pytest.raises(eg.EngramError):
        eg.engram_delta_grad(dy, *args, carry, i64([0, T]), 1, workspace=torch.empty(256, dtype=torch.uint8, device=DEV))
