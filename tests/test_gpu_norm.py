"""The norm behind a block, its gate and residual scale, the next block's norm, and their gradients on the GPU against
the 64-bit oracle."""
import pytest
import torch

import hashed_gram_conditional_gb300 as eg
from gpu_util import DEV, require_gpu
from oracle import blocks as OB

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    require_gpu()


def make(shape, kind, seed, scale=1.0, shift=0.0):
    gen = torch.Generator(DEV).manual_seed(seed)
    return (torch.randn(shape, generator=gen, device=DEV) * scale + shift).to(TYPES[kind])


def close(got, want, err, kind):
    """Within the fp32 error bound, and for bf16 (8 significant bits) the final rounding's 2^-8."""
    half = 2.0 ** -8 if kind == "bf16" else 0.0
    off = (got.double() - want).abs()
    tol = err * (1 + half) + half * want.abs() * (1 + 1e-6) + 1e-38
    assert (off <= tol).all(), (int((off > tol).sum()), float((off / tol).max()))


def d64(t):
    return None if t is None else t.double()


def run(T, D, kind, seed, groups=1, gate=True, res=True, scaled=True, weighted=True, nxt=True, dh=True, eps=1e-6,
        lay=lambda t: t):
    """One forward and one backward call; `lay` puts the matrices elsewhere in memory."""
    m = lambda k, s=1.0: lay(make((T, D), kind, seed + k, s))  # noqa: E731
    y, z, h = m(1, 2.0), m(2) if gate else None, m(3, 3.0) if res else None
    w = make((D // groups,), "f32", seed + 4, 0.3, 1.0) if weighted else None
    s = make((D,), "f32", seed + 5, 0.3, 0.5) if scaled else None
    wn = make((D,), "f32", seed + 6, 0.3, 1.0) if nxt else None
    out, x = eg.engram_norm_add(y, w, gate=z, h=h, scale=s, w_next=wn, groups=groups, eps=eps)
    want, err = OB.norm_add(d64(y), d64(w), d64(z), d64(h), d64(s), groups, eps)
    close(out, want, err, kind)
    if nxt:
        close(x, *OB.norm_next(d64(out), d64(wn), eps), kind)
    else:
        assert x is None
    g = m(7, 0.2) if dh or not nxt else None
    dx = m(8, 0.2) if nxt else None
    got = eg.engram_norm_add_grad(g, y, w, gate=z, scale=s, h_out=out if nxt else None, dx=dx, w_next=wn, groups=groups,
                                  eps=eps, residual=res)
    want = OB.norm_add_grad(d64(g), d64(y), d64(w), d64(z), d64(s), d64(out), d64(dx), d64(wn), groups, eps)
    have = dict(dy=True, dgate=gate, dres=res, dw=weighted, dscale=scaled, dw_next=nxt)
    for (name, there), t in zip(have.items(), got):
        assert (t is not None) == there, name
        if there:
            close(t, *want[name], "f32" if name in ("dw", "dscale", "dw_next") else kind)
    return out, x, got


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("T,D,groups", [(1, 1, 1), (3, 8, 1), (5, 7, 7), (4, 80, 1), (9, 80, 4), (3, 257, 1), (700, 64, 1),
                                        (17, 1280, 10), (300, 1280, 1), (6, 5120, 40), (330, 5120, 1), (2, 5128, 1),
                                        (5, 4096, 1024), (4, 960, 4), (3, 8200, 5), (7, 8192, 1), (2, 16384, 2),
                                        (2, 16392, 1), (1, 40001, 1), (2, 2400, 50), (3, 4001, 1), (2, 8191, 1),
                                        (9, 6003, 3), (4, 2047, 23), (3, 40005, 9)])
def test_forward_and_gradient(T, D, groups, kind):
    run(T, D, kind, 100, groups)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("T,D,groups", [(1300, 2560, 1), (1301, 2560, 20), (1400, 2400, 50), (2700, 1280, 10), (6000, 8, 1),
                                        (5100, 264, 3), (700, 5120, 1), (640, 5120, 40), (1300, 2000, 5)])
def test_many_rows_for_each_block(T, D, groups, kind):
    run(T, D, kind, 400, groups)
    run(T, D, kind, 410, groups, gate=False, res=False, scaled=False, weighted=groups > 1, nxt=groups == 1)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("D", [40, 1000, 2560, 5120])
@pytest.mark.parametrize("gate,nxt,dh", [(True, False, True), (False, False, True), (False, True, False)])
def test_parts_left_out_of_many_rows(D, gate, nxt, dh, kind):
    T = 1400 if D > 2000 else 5000
    run(T, D, kind, 440, 1, gate=gate, nxt=nxt, dh=dh)


def test_many_rows_with_nan_and_zeros():
    """They stay in their row, in the rows of a block before and after it too."""
    T, D = 2600, 2000
    y, z, h, wn = make((T, D), "bf16", 450), make((T, D), "bf16", 451), make((T, D), "bf16", 452), make((D,), "f32", 453)
    clean, cx = eg.engram_norm_add(y, gate=z, h=h, w_next=wn)
    y[1000, 5], h[1700, 9] = float("nan"), float("inf")
    y[1300] = 0.0
    out, x = eg.engram_norm_add(y, gate=z, h=h, w_next=wn)
    rest = torch.ones(T, dtype=torch.bool, device=DEV)
    rest[[1000, 1300, 1700]] = False
    assert torch.equal(out[rest], clean[rest]) and torch.equal(x[rest], cx[rest])
    assert torch.isnan(out[1000]).all() and torch.equal(out[1300], h[1300])
    g = torch.ones_like(y)
    got = eg.engram_norm_add_grad(g, y, gate=z, h_out=out, dx=g, w_next=wn)
    assert all(torch.isfinite(t[rest]).all() for t in got[:3])


def test_many_rows_in_place():
    T, D = 1300, 2000
    y, z, h = (make((T, D), "bf16", 420 + k) for k in range(3))
    w, s, wn = (make((D,), "f32", 430 + k) for k in range(3))
    out, x = eg.engram_norm_add(y, w, gate=z, h=h, scale=s, w_next=wn)
    kept, again = eg.engram_norm_add(y, w, gate=z, h=h, scale=s, w_next=wn, h_out=h)
    assert kept is h and torch.equal(h, out) and torch.equal(again, x)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("gate,res,scaled,weighted,nxt,dh", [(False, False, False, False, False, True),
                                                             (False, False, False, True, True, False),
                                                             (True, False, False, True, False, True),
                                                             (False, True, True, False, True, True),
                                                             (True, True, False, True, True, False)])
@pytest.mark.parametrize("D", [264, 97])
def test_parts_left_out(D, gate, res, scaled, weighted, nxt, dh, kind):
    run(40, D, kind, 200, 1, gate, res, scaled, weighted, nxt, dh)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("pitch,shift", [(600, 0), (521, 0), (600, 1), (520, 8)])
def test_strides_and_alignment(pitch, shift, kind):
    """Matrices that are columns of wider ones, some of them not 16-byte aligned: the same values to the last bit where the
    aligned kernel runs, and within the bounds elsewhere."""
    def lay(t):
        wide = torch.full((t.shape[0], pitch + shift), float("nan"), dtype=t.dtype, device=DEV)
        wide[:, shift:shift + t.shape[1]] = t
        return wide[:, shift:shift + t.shape[1]]
    run(33, 512, kind, 300, 4, lay=lay)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("D", [512, 77])
def test_in_place_and_between_other_columns(D, kind):
    """h_out over h and dres over dh; outputs into columns of wider matrices, whose other columns stay."""
    T = 50
    y, z, h = make((T, D), kind, 1), make((T, D), kind, 2), make((T, D), kind, 3)
    w, s, wn = make((D,), "f32", 4), make((D,), "f32", 5), make((D,), "f32", 6)
    out, x = eg.engram_norm_add(y, w, gate=z, h=h, scale=s, w_next=wn)
    wide = torch.full((T, D + 16), 7.0, dtype=h.dtype, device=DEV)
    kept = h.clone()
    out2, x2 = eg.engram_norm_add(y, w, gate=z, h=kept, scale=s, w_next=wn, h_out=kept, x=wide[:, 8:8 + D])
    assert out2 is kept and torch.equal(out, kept) and torch.equal(x, x2)
    assert (wide[:, :8] == 7).all() and (wide[:, 8 + D:] == 7).all()
    dh, dx = make((T, D), kind, 7), make((T, D), kind, 8)
    a = eg.engram_norm_add_grad(dh, y, w, gate=z, scale=s, h_out=out, dx=dx, w_next=wn)
    b = eg.engram_norm_add_grad(dh, y, w, gate=z, scale=s, h_out=out, dx=dx, w_next=wn, dres=dh)
    assert b[2] is dh
    for u, v in zip(a, b):
        assert torch.equal(u, v)


def test_no_rows():
    w = torch.ones(8, device=DEV)
    e = torch.empty((0, 8), device=DEV)
    out, x = eg.engram_norm_add(e, w, w_next=w)
    assert out.shape == (0, 8) and x.shape == (0, 8)
    got = eg.engram_norm_add_grad(e, e, w, scale=w, h_out=e, dx=e, w_next=w)
    assert all((g == 0).all() for g in got[3:])


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_rows_of_zeros_and_nan_stay_in_their_row(kind):
    T, D = 20, 264
    y, z, h = make((T, D), kind, 11), make((T, D), kind, 12), make((T, D), kind, 13)
    y[3] = 0.0
    clean, cx = eg.engram_norm_add(y, gate=z, h=h, w_next=torch.ones(D, device=DEV))
    assert torch.isfinite(clean).all() and torch.equal(clean[3], h[3])
    y[7, 5] = float("nan")
    h[9, 0] = float("inf")
    out, x = eg.engram_norm_add(y, gate=z, h=h, w_next=torch.ones(D, device=DEV))
    rest = [t for t in range(T) if t not in (7, 9)]
    assert torch.equal(out[rest], clean[rest]) and torch.equal(x[rest], cx[rest])
    assert torch.isnan(out[7]).all()
    got = eg.engram_norm_add_grad(h, y, gate=z)
    assert torch.isfinite(got[0][rest]).all() and torch.isfinite(got[1][rest]).all()


def test_another_stream_and_a_captured_graph():
    T, D = 64, 520
    y, z, h = (make((T, D), "bf16", 20 + k) for k in range(3))
    w, s, wn = (make((D,), "f32", 30 + k) for k in range(3))
    dh, dx = make((T, D), "bf16", 40), make((T, D), "bf16", 41)

    def both():
        out, x = eg.engram_norm_add(y, w, gate=z, h=h, scale=s, w_next=wn)
        return (out, x) + eg.engram_norm_add_grad(dh, y, w, gate=z, scale=s, h_out=out, dx=dx, w_next=wn)
    want = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = both()
    torch.cuda.current_stream().wait_stream(side)
    for u, v in zip(want, got):
        assert torch.equal(u, v)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    y.copy_(make((T, D), "bf16", 50))
    graph.replay()
    want = both()
    for u, v in zip(want, got):
        assert torch.equal(u, v)


def test_the_binding_refuses():
    y = make((4, 24), "bf16", 1)
    w = torch.ones(24, device=DEV)
    with pytest.raises(ValueError):
        eg.engram_norm_add(y, w, groups=5)
    with pytest.raises(ValueError):
        eg.engram_norm_add(y, w, groups=2)
    with pytest.raises(TypeError):
        eg.engram_norm_add(y, w.bfloat16())
    with pytest.raises(ValueError):
        eg.engram_norm_add(y, w, h=y[:, :16])
    with pytest.raises(TypeError):
        eg.engram_norm_add(y, w, gate=y.float())
    with pytest.raises(eg.EngramError):
        eg.engram_norm_add(y, w, eps=-1.0)
    with pytest.raises(eg.EngramError):
        eg.engram_norm_add_grad(None, y, w)
    with pytest.raises(eg.EngramError):
        eg.engram_norm_add_grad(y, y, w, dx=y)
    with pytest.raises(eg.EngramError):
        eg.engram_norm_add_grad(y, y, w, dgate=torch.empty_like(y))
