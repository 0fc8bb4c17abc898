"""Row lookup and its gradient on the GPU against the 64-bit oracle."""
import numpy as np
import pytest
import torch

import hashed_gram_conditional_gb300 as eg
from gpu_util import DEV, i32, require_gpu, status
from oracle import training as OT

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    require_gpu()


def make(shape, kind, seed, scale=1.0):
    rng = np.random.default_rng(seed)
    return torch.from_numpy(rng.normal(size=shape) * scale).to(torch.float32).to(TYPES[kind]).to(DEV)


def ids_of(T, C, R, seed, pad=0.1):
    """Row ids with a few that repeat often, and some DEAD."""
    rng = np.random.default_rng(seed)
    ids = rng.integers(0, R, size=(T, C))
    ids = np.where(rng.random((T, C)) < 0.3, rng.integers(0, min(R, 3), size=(T, C)), ids)
    return np.where(rng.random((T, C)) < pad, -1, ids).astype(np.int32)


SHAPES = [(1, 1, 1, 1), (1, 24, 256, 5000), (7, 3, 80, 100), (33, 16, 80, 4099), (64, 1, 5120, 50), (129, 2, 7, 11),
          (300, 5, 33, 20), (1000, 1, 8, 3)]


@pytest.mark.parametrize("T,C,D,R", SHAPES)
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_lookup_is_exact(T, C, D, R, kind):
    table, ids = make((R, D), kind, 1), ids_of(T, C, R, 2)
    st = status()
    got = eg.engram_lookup(table, i32(ids), 1.25, status=st)
    # one fp32 product and one rounding of it: the same bits as torch's
    ok = torch.from_numpy((ids >= 0) & (ids < R)).to(DEV)
    want = (table[torch.from_numpy(np.maximum(ids, 0)).long().to(DEV)].float() * 1.25 * ok[..., None]).to(TYPES[kind])
    assert torch.equal(got, want.view(T, C * D))
    ref = OT.lookup(table.double().cpu().numpy(), ids, 1.25)
    unit = 2.0 ** -8 if kind == "bf16" else 0.0
    assert (np.abs(got.double().cpu().numpy() - ref) <= 1.01 * (unit + 2.0 ** -24) * np.abs(ref)).all()
    assert int(st.item()) == 0


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_lookup_strides_alignment_and_bad_ids(kind):
    T, C, D, R = 37, 3, 40, 60
    table = make((R * D + 1,), kind, 3)[1:].view(R, D)  # element-aligned only
    ids = ids_of(T, C, R, 4)
    ids[5, 1], ids[6, 0], ids[7, 2] = R, -2, 2 ** 31 - 1
    out = torch.full((T, C * D + 13), 7.0, dtype=TYPES[kind], device=DEV)
    st = status()
    eg.engram_lookup(table, i32(ids), 0.5, out=out[:, 5:5 + C * D], status=st)
    ref = OT.lookup(table.double().cpu().numpy(), ids, 0.5)  # halving is exact
    assert (out[:, 5:5 + C * D].double().cpu().numpy() == ref).all()
    assert (out[:, :5] == 7).all() and (out[:, 5 + C * D:] == 7).all()
    assert int(st.item()) == eg.ST_BAD_ROW


def test_lookup_special_values_and_no_positions():
    table = torch.tensor([[float("inf"), float("-inf"), float("nan"), -0.0, 3e38, 1e-40, 1.0, 2.0]], device=DEV)
    got = eg.engram_lookup(table, i32([0, -1]), 2.0)
    want = torch.stack([table[0] * 2.0, torch.zeros(8, device=DEV)])
    assert torch.equal(got.view(torch.int32), want.view(torch.int32))
    assert eg.engram_lookup(table, torch.empty((0, 3), dtype=torch.int32, device=DEV)).shape == (0, 24)


def test_lookup_past_four_giga_elements():
    """Row offsets beyond 2^32 elements."""
    R, D = 4_400_000, 1024
    table = torch.empty((R, D), dtype=torch.bfloat16, device=DEV)
    table[R - 1] = make((D,), "bf16", 5)
    table[0] = make((D,), "bf16", 6)
    got = eg.engram_lookup(table, i32([R - 1, 0]), 1.0)
    assert torch.equal(got[0], table[R - 1]) and torch.equal(got[1], table[0])


def check_grad(dout, ids, R, scale, C):
    d = dout.double().cpu().numpy()
    ref, err, uniq = OT.lookup_grad(d, ids, R, scale)
    st = status()
    dense = eg.engram_lookup_grad(dout, i32(ids), R, scale, status=st)
    got = dense.double().cpu().numpy()
    assert got.shape == ref.shape and (np.abs(got - ref) <= err).all()
    rows, grad, count = eg.engram_lookup_grad_rows(dout, i32(ids), R, scale, status=st)
    m = int(count.item())
    r = rows.cpu().numpy()
    assert m == len(uniq) and (r[:m] == uniq).all() and (r[m:] == -1).all()
    gr = grad.double().cpu().numpy()
    assert (np.abs(gr[:m] - ref[uniq]) <= err[uniq]).all() and (gr[m:] == 0).all()
    return st, dense, (rows, grad, count)


@pytest.mark.parametrize("T,C,D,R", SHAPES)
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_gradients(T, C, D, R, kind):
    ids = ids_of(T, C, R, 7)
    st, dense, rows = check_grad(make((T, C * D), kind, 8), ids, R, 1.5, C)
    assert int(st.item()) == 0


@pytest.mark.parametrize("T,R,how", [(20000, 70000, "one"), (20000, 70000, "runs"), (9000, 2_000_000_000, "wide"),
                                     (4096, 300, "few"), (4097, 300, "distinct"), (70000, 40, "few")])
def test_gradient_of_long_and_short_segments(T, R, how):
    """One row for every entry, long runs, ids of 31 bits, every id once; sizes around the sort's blocks."""
    rng = np.random.default_rng(9)
    if how == "one":
        ids = np.full(T, 69999)
    elif how == "runs":
        ids = np.sort(rng.integers(0, 7, T)) * 9973
    elif how == "wide":
        ids = rng.integers(0, R, T)
        ids[::5] = ids[0]
        ids[-1] = R - 1
    elif how == "distinct":
        ids, R = rng.permutation(T), T
    else:
        ids = rng.integers(0, R, T)
    ids = ids.astype(np.int32)
    D = 24
    dout = make((T, D), "bf16", 10)
    d = dout.double().cpu().numpy()
    uniq, inv, n = np.unique(ids, return_inverse=True, return_counts=True)
    ref, size = np.zeros((len(uniq), D)), np.zeros((len(uniq), D))
    np.add.at(ref, inv, d)
    np.add.at(size, inv, np.abs(d))
    rows, grad, count = eg.engram_lookup_grad_rows(dout, i32(ids), R, 1.0)
    m = int(count.item())
    assert m == len(uniq) and (rows[:m].cpu().numpy() == uniq).all() and (rows[m:] == -1).all()
    assert (np.abs(grad[:m].double().cpu().numpy() - ref) <= size * (n[:, None] + 1) * OT.UNIT).all()
    assert (grad[m:] == 0).all()
    if R < 100000:
        dense = eg.engram_lookup_grad(dout, i32(ids), R, 1.0).double().cpu().numpy()
        want = np.zeros((R, D))
        want[uniq] = ref
        bound = np.zeros((R, D))
        bound[uniq] = size * (n[:, None] + 1) * OT.UNIT
        assert (np.abs(dense - want) <= bound).all()


@pytest.mark.parametrize("T,D,R", [(3, 5120, 500), (40, 4299, 700), (700, 257, 5000), (2000, 8, 90000), (9000, 1000, 4000),
                                   (1, 1, 3), (5000, 6, 6),
                                   # large enough for rows to be cleared during the sort, and the last number of them
                                   (513, 257, 20_000), (300, 40, 7), (9000, 1000, 6001), (100_000, 24, 180_000), (2000, 17, 262_144),
                                   (6000, 17, 262_145)])
def test_every_row_of_the_outputs_is_written(T, D, R):
    """Outputs that hold something else before: rows that no entry names become zeros, with none left out."""
    rng = np.random.default_rng(31)
    ids = rng.integers(-1, R, size=T).astype(np.int32)
    ids[rng.random(T) < 0.3] = ids[0]
    dout = make((T, D), "bf16", 32)
    ref, err, uniq = OT.lookup_grad(dout.double().cpu().numpy(), ids[:, None], R, 1.0)
    grad = torch.full((R, D), float("nan"), device=DEV)
    eg.engram_lookup_grad(dout, i32(ids), R, 1.0, grad=grad)
    assert (np.abs(grad.double().cpu().numpy() - ref) <= err).all()
    rows = torch.full((T,), 12345, dtype=torch.int32, device=DEV)
    grad = torch.full((T, D), float("nan"), device=DEV)
    count = torch.full((1,), -5, dtype=torch.int32, device=DEV)
    eg.engram_lookup_grad_rows(dout, i32(ids), R, 1.0, rows=rows, grad=grad, count=count)
    m = len(uniq)
    assert int(count.item()) == m and (rows[:m].cpu().numpy() == uniq).all() and (rows[m:] == -1).all()
    g = grad.double().cpu().numpy()
    assert (np.abs(g[:m] - ref[uniq]) <= err[uniq]).all() and (g[m:] == 0).all()


@pytest.mark.parametrize("T,R", [(319, 90), (320, 90), (321, 90), (320, 2), (512, 90), (4095, 4000), (4097, 5000), (622_592, 200_000),
                                 (622_593, 200_000), (700_001, 2_000_000_000), (1_300_000, 300)])
def test_gradient_where_the_sort_changes_its_way(T, R):
    """Sizes beside each of the sort's limits, and ones that need several rounds; ids outside the table among them."""
    rng = np.random.default_rng(T)
    ids = rng.integers(0, R, size=T)
    ids[rng.random(T) < 0.2] = rng.integers(0, R)
    ids[rng.random(T) < 0.05] = -1
    ids[T // 2], ids[T - 1] = -7, R if R < 2 ** 31 else -1
    ids = ids.astype(np.int32)
    D = 8
    dout = make((T, D), "f32", 33)
    live = (ids >= 0) & (ids < R)
    uniq, inv, n = np.unique(ids[live], return_inverse=True, return_counts=True)
    at, d = torch.from_numpy(inv).to(DEV), dout.double()[torch.from_numpy(live).to(DEV)]
    ref = torch.zeros((len(uniq), D), dtype=torch.float64, device=DEV).index_add_(0, at, d)
    err = torch.zeros_like(ref).index_add_(0, at, d.abs()) * torch.from_numpy(n + 1).to(DEV)[:, None] * OT.UNIT
    st = status()
    rows, grad, count = eg.engram_lookup_grad_rows(dout, i32(ids), R, 1.0, status=st)
    m = int(count.item())
    assert m == len(uniq) and (rows[:m].cpu().numpy() == uniq).all() and (rows[m:] == -1).all()
    assert ((grad[:m].double() - ref).abs() <= err).all() and (grad[m:] == 0).all()
    assert int(st.item()) == eg.ST_BAD_ROW
    again = eg.engram_lookup_grad_rows(dout, i32(ids), R, 1.0)
    assert torch.equal(grad, again[1]) and torch.equal(rows, again[0])
    if R <= 300_000:
        dense = torch.full((R, D), float("nan"), device=DEV)
        eg.engram_lookup_grad(dout, i32(ids), R, 1.0, grad=dense)
        want, bound = torch.zeros((2, R, D), dtype=torch.float64, device=DEV)
        want[torch.from_numpy(uniq).long().to(DEV)] = ref
        bound[torch.from_numpy(uniq).long().to(DEV)] = err
        assert ((dense.double() - want).abs() <= bound).all()


def test_gradient_is_the_same_from_run_to_run():
    ids = i32(ids_of(5000, 4, 300, 11))
    dout = make((5000, 4 * 48), "bf16", 12)
    first = [t.clone() for t in eg.engram_lookup_grad_rows(dout, ids, 300)]
    dense = eg.engram_lookup_grad(dout, ids, 300).clone()
    for _ in range(3):
        for a, b in zip(first, eg.engram_lookup_grad_rows(dout, ids, 300)):
            assert torch.equal(a, b)
        assert torch.equal(dense, eg.engram_lookup_grad(dout, ids, 300))


def test_gradient_strides_bad_ids_and_empty_batches():
    T, C, D, R = 41, 2, 20, 30
    wide = make((T, C * D + 9), "f32", 13)
    dout = wide[:, 3:3 + C * D]
    ids = ids_of(T, C, R, 14)
    ids[0, 0], ids[3, 1] = R, -7
    st, _, _ = check_grad(dout, ids, R, 1.0, C)
    assert int(st.item()) == eg.ST_BAD_ROW
    none = torch.full((T, C), -1, dtype=torch.int32, device=DEV)
    assert (eg.engram_lookup_grad(dout, none, R) == 0).all()
    rows, grad, count = eg.engram_lookup_grad_rows(dout, none, R)
    assert int(count.item()) == 0 and (rows == -1).all() and (grad == 0).all()
    empty = torch.empty((0, C), dtype=torch.int32, device=DEV)
    assert (eg.engram_lookup_grad(dout[:0], empty, R) == 0).all()
    rows, grad, count = eg.engram_lookup_grad_rows(dout[:0], empty, R)
    assert int(count.item()) == 0 and rows.numel() == 0 and grad.shape == (0, D)


def test_gradient_against_differences():
    """<grad, v> is the change of <dout, lookup(table + v)>: the lookup is linear in the table."""
    T, C, D, R = 50, 3, 16, 40
    table, v = make((R, D), "f32", 15), make((R, D), "f32", 16)
    dout, ids = make((T, C * D), "f32", 17), i32(ids_of(T, C, R, 18))
    grad = eg.engram_lookup_grad(dout, ids, R, 0.75).double()
    up = eg.engram_lookup(table + v, ids, 0.75).double()
    down = eg.engram_lookup(table - v, ids, 0.75).double()
    change = (dout.double() * (up - down)).sum().item() / 2
    # each looked-up value is off by three fp32 roundings (sum, product, the gradient's own) of sizes of a few
    bound = 8 * OT.UNIT * (dout.abs().double() * (up.abs() + down.abs() + 1)).sum().item()
    assert abs((grad * v.double()).sum().item() - change) <= bound


def test_gradient_on_another_stream():
    T, C, D, R = 3000, 4, 64, 500
    ids, dout = i32(ids_of(T, C, R, 19)), make((T, C * D), "bf16", 20)
    want = eg.engram_lookup_grad(dout, ids, R)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = eg.engram_lookup_grad(dout, ids, R)
    s.synchronize()
    assert torch.equal(got, want)


def test_refusals():
    table, ids = make((4, 8), "bf16", 21), i32([[0, 1]])
    with pytest.raises(TypeError):
        eg.engram_lookup(table.half(), ids)
    with pytest.raises(TypeError):
        eg.engram_lookup(table, ids.long())
    with pytest.raises(ValueError):
        eg.engram_lookup(table, ids, out=torch.empty((1, 8), dtype=torch.bfloat16, device=DEV))
    with pytest.raises(ValueError):
        eg.engram_lookup(table.t(), ids)
    with pytest.raises(ValueError):
        eg.engram_lookup_grad(make((1, 15), "f32", 22), ids, 4)  # 15 is not n_cols * row_dim
    with pytest.raises(eg.EngramError, match="RANGE"):
        eg.engram_lookup_grad(make((1, 16), "f32", 22), ids, 4, workspace=torch.empty(256, dtype=torch.uint8,
                                                                                    device=DEV)[:1])
    with pytest.raises(eg.EngramError, match="RANGE"):
        eg.engram_lookup_grad_rows(make((1, 16), "f32", 22), ids, 2 ** 31)
