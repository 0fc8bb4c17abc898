"""Sequences that the forward pass of the gated delta rule took for padding, in its backward pass."""
import pytest
import torch

import hashed_gram_conditional_gb300 as eg
from gpu_util import DEV, i32, i64, require_gpu, status
from test_gpu_delta import inputs, make

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    require_gpu()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("keys,H,dk,dv", [(1, 2, 32, 40), (20, 40, 64, 64)])  # fewer and more heads than the blocks of four quads need
@pytest.mark.parametrize("with_dstate", [False, True])
def test_a_slot_that_the_forward_call_does_not_have(with_dstate, keys, H, dk, dv, kind):
    """Slots 9 and 3 are not among the three of the forward call's states; the carry holds NaN where nothing is left.  The
    gradients are those of a call whose padding is said by negative slots, whether states' gradients are asked for or not."""
    T, cu = 400, i64([0, 90, 90, 220, 300, 400])
    args, dy = inputs(T, keys, H, dk, dv, kind, 500), make((T, H * dv), kind, 510)
    s0, got = make((3, H, dk, dv), "f32", 511, 0.3), {}
    for name, slots in dict(bad=[1, 0, 9, 2, 3], padded=[1, 0, -1, 2, -1]).items():
        carry = eg.delta_carry(T, 5, keys, H, dk, dv, DEV).fill_(float("nan"))
        st = status()
        y = eg.engram_delta(*args, cu, keys, state=s0, slots=i32(slots), state_out=torch.empty_like(s0), carry=carry, status=st)
        assert int(st.item()) == (eg.ST_BAD_SLOT if name == "bad" else 0)
        ds = make((3, H, dk, dv), "f32", 512, 0.3) if with_dstate else None
        st.zero_()
        grads = eg.engram_delta_grad(dy, *args, carry, cu, keys, slots=i32(slots), dstate=ds, status=st)
        assert int(st.item()) == (eg.ST_BAD_SLOT if name == "bad" else 0)
        got[name] = (y, *grads) + (() if ds is None else (ds,))
    for u, w in zip(got["bad"], got["padded"]):
        assert torch.equal(u, w)
    for t in got["bad"][:6]:
        assert (t[90:220] == 0).all() and (t[300:] == 0).all() and torch.isfinite(t).all()
        assert (t[:90] != 0).any() and (t[220:300] != 0).any()


def test_a_carry_that_is_used_again():
    """What was padding in one call is not in the next one on the same carry, and the other way round."""
    T, keys, H, d, cu = 200, 1, 2, 32, i64([0, 100, 200])
    args, dy, s0 = inputs(T, keys, H, d, d, "bf16", 520), make((T, H * d), "bf16", 530), make((2, H, d, d), "f32", 531)
    carry, rows = eg.delta_carry(T, 2, keys, H, d, d, DEV), []
    for slots in ([0, 7], [0, 1], [7, 1], [0, 1]):
        eg.engram_delta(*args, cu, keys, state=s0, slots=i32(slots), state_out=torch.empty_like(s0), carry=carry)
        rows.append(eg.engram_delta_grad(dy, *args, carry, cu, keys, slots=i32(slots)))
    for a, b, c, d_ in zip(*rows):
        assert torch.equal(b, d_)
        assert torch.equal(a[:100], b[:100]) and (a[100:] == 0).all()
        assert torch.equal(c[100:], b[100:]) and (c[:100] == 0).all()


def test_without_a_state_any_slot_will_do():
    """Where no call has states, slots only say what is padding."""
    T, keys, H, d, cu = 150, 1, 2, 32, i64([0, 70, 150])
    args, dy, rows = inputs(T, keys, H, d, d, "bf16", 540), make((T, H * d), "bf16", 550), []
    for slots in ([0, 1], [1000, 5]):
        carry = eg.delta_carry(T, 2, keys, H, d, d, DEV).fill_(float("nan"))
        y = eg.engram_delta(*args, cu, keys, slots=i32(slots), carry=carry)
        rows.append((y, *eg.engram_delta_grad(dy, *args, carry, cu, keys, slots=i32(slots))))
    for u, w in zip(*rows):
        assert torch.equal(u, w)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_the_backward_call_does_not_need_the_values(kind):
    """v may hold anything by then, and the C call takes none at all."""
    T, keys, H, dk, dv, cu = 150, 1, 2, 32, 40, i64([0, 70, 150])
    (q, k, v, g, b), dy = inputs(T, keys, H, dk, dv, kind, 560), make((T, H * dv), kind, 570)
    carry = eg.delta_carry(T, 2, keys, H, dk, dv, DEV)
    eg.engram_delta(q, k, v, g, b, cu, keys, carry=carry)
    want = eg.engram_delta_grad(dy, q, k, v, g, b, carry, cu, keys)
    v.fill_(float("nan"))
    for u, w in zip(eg.engram_delta_grad(dy, q, k, v, g, b, carry, cu, keys), want):
        assert torch.equal(u, w)
    got, ws = [torch.empty_like(t) for t in want], eg.delta_workspace(T, 2, keys, H, dk, dv, DEV, True)
    wk, wv = keys * dk, H * dv
    rc = eg.lib().engram_delta_grad(
        dy.data_ptr(), wv, q.data_ptr(), wk, k.data_ptr(), wk, None, wv, g.data_ptr(), H, b.data_ptr(), H, 0 if kind == "bf16" else 1,
        T, keys, H, dk, dv, dk ** -0.5, cu.data_ptr(), 2, None, None, carry.data_ptr(), None, 0,
        *(x for t in got for x in (t.data_ptr(), t.shape[1])), ws.data_ptr(), ws.numel(), None,
        torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    for u, w in zip(got, want):
        assert torch.equal(u, w)
