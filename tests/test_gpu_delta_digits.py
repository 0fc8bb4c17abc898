"""Gradients of the gated delta rule that are small differences of large terms."""
import pytest
import torch

import hashed_gram_conditional_gb300 as eg
from gpu_util import DEV, i64, require_gpu
from oracle import blocks as OB
from test_gpu_delta import d64, inputs, make

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    require_gpu()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("T,keys,H,d,shift", [(300, 2, 4, 64, 5.0), (300, 2, 4, 64, 8.0), (200, 64, 128, 64, 8.0), (190, 1, 2, 128, 8.0),
                                              (130, 60, 60, 128, 8.0)])
def test_a_decay_that_hardly_matters(T, keys, H, d, shift, kind):
    """One key again and again, written with beta near 1 and read by itself: what decays is overwritten before it is read, and
    dg_t = (1 - f_t) sum over s >= t of (y_s . dy_s - v_s . dv_s) is thousands of times smaller than its terms.

    Tolerance, with A the sum of the terms' sizes: the tensor cores cut an accumulator off at its last bit, 2^-23 of a dot
    product for each of the at most 5 d / 16 + 2 d / 16 instructions behind two dots that cancel, 2^-24 on average and all
    in one direction; a dot of d terms of independent signs is d^-1/2 of their sizes' sum.  That is 2^-24 7 d^1/2 / 16 A,
    2^-21.6 A for d = 128; operands of 24 bits and sums in fp32 are below that: 2^-21 A, and half of a bf16 step."""
    q, k, v, g, b = inputs(T, keys, H, d, d, kind, 300, 4.0)
    k = k[:1].expand(T, -1).contiguous()
    b = (b.float() + shift).to(b.dtype)
    args, dy, cu, scale = (k, k, v, g, b), make((T, H * d), kind, 310, 0.1), [0, T], d ** -0.5
    carry = eg.delta_carry(T, 1, keys, H, d, d, DEV)
    eg.engram_delta(*args, i64(cu), keys, carry=carry)
    got = eg.engram_delta_grad(dy, *args, carry, i64(cu), keys)[3].double()
    y = OB.delta(*d64(*args), cu, keys, scale)["y"]
    want = OB.delta_grad(dy.double(), *d64(*args), cu, keys, scale)

    def later(x):
        return x.view(T, H, d).sum(2).flip(0).cumsum(0).flip(0) * torch.sigmoid(-g.double())
    parts = y * dy.double(), v.double() * want["dv"]
    assert torch.allclose(later(parts[0] - parts[1]), want["dg"], rtol=1e-6, atol=1e-12)  # the sum that the tolerance is of
    half = 2.0 ** -8 if kind == "bf16" else 0.0
    tol = 2.0 ** -21 * later(parts[0].abs() + parts[1].abs()) + half * want["dg"].abs() * (1 + 1e-6)
    off = (got - want["dg"]).abs()
    assert (off <= tol).all(), (int((off > tol).sum()), float((off / tol).max()))


@pytest.mark.parametrize("T,keys,H,dk,dv,S", [(200, 2, 4, 64, 64, 1), (300, 2, 4, 40, 72, 3), (130, 1, 1, 64, 16, 1)])
def test_fp32_keeps_its_digits(T, keys, H, dk, dv, S):
    """All outputs of type fp32, each by its error's norm against its own.

    An operand's three terms are 24 bits and an fp32 sum's roundings less than the tensor cores' cuts: of a product's main
    accumulator one for every 16 terms, 2^-24 of what it then holds on average, at most 2 of them in all for 64 terms whose
    partial sums grow to the whole, and the triangles' products the same: 2^-23 a product.  Of the products that follow
    one another, no output has more than 16 in front of it, and their errors are independent: 2^-21.  An operand of 16 bits
    would show: 2^-18 / sqrt(3) and more of what it is multiplied into."""
    cu = [T * s // S for s in range(S + 1)]
    args, dy = inputs(T, keys, H, dk, dv, "f32", 320), make((T, H * dv), "f32", 330)
    s0, ds = make((S, H, dk, dv), "f32", 331, 0.3), make((S, H, dk, dv), "f32", 332, 0.3)
    carry, out, back = eg.delta_carry(T, S, keys, H, dk, dv, DEV), torch.empty_like(s0), ds.clone()
    y = eg.engram_delta(*args, i64(cu), keys, state=s0, state_out=out, carry=carry)
    grads = eg.engram_delta_grad(dy, *args, carry, i64(cu), keys, dstate=back)
    fwd = OB.delta(*d64(*args), cu, keys, dk ** -0.5, state=s0.double())
    want = OB.delta_grad(dy.double(), *d64(*args), cu, keys, dk ** -0.5, state=s0.double(), dstate=ds.double())
    got = dict(y=y, state=out, **dict(zip(("dq", "dk", "dv", "dg", "db"), grads)), dstate=back)
    for name, t in got.items():
        w = fwd[name] if name in ("y", "state") else want[name]
        assert float((t.double() - w).norm() / w.norm()) <= 2.0 ** -21, name
