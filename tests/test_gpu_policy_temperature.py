"""The policy loss at temperatures far from 1, whose squares no fp32 number holds."""
import pytest
import torch

import hashed_gram_conditional_gb300 as eg
from gpu_util import require_gpu
from oracle import blocks as OB
from test_gpu_policy import check, close, inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    require_gpu()


@pytest.mark.parametrize("tau", [1e-25, 1e-18, 1e-3, 50.0, 1e18, 1e25, 1e30])
@pytest.mark.parametrize("T,V,kind", [(70, 31, "f32"), (70, 31, "bf16"), (400, 20_003, "f32"), (90, 129_280, "bf16"), (3, 600_001, "f32")])
def test_loss_and_gradient(T, V, kind, tau):
    """Short rows, rows that a cluster keeps and rows that are read twice.  A small temperature leaves a row's largest logit
    alone, a large one all of them alike; the gradient is 1 / tau times what lies between.

    The exponential's results below 2^-126 are zero (ex2.approx.ftz), so a probability q < 2^-126 counts as 0, and its
    gradient -L' q / tau, at most 2^-126 |w A| / tau where the ratio is 1 and there is no KL term, is lost: below 1e-38, which
    `close` allows, for tau >= 1, but more for smaller ones.  That is added to the bound."""
    z, ids, adv, old, ref, w = inputs(T, V, kind, 700, tau)
    if tau >= 1.0:
        check(z, ids, adv, tau=tau, weight=w, kind=kind)
        check(z, ids, adv, old, ref, kl=0.1, tau=tau, weight=w, kind=kind)
        return
    dz = torch.empty_like(z)
    loss, logp = eg.engram_policy(z, ids, adv, temperature=tau, weight=w, dlogits=dz)
    want = OB.policy(z.double(), ids, adv.double(), tau=tau, weight=w.double())
    close(loss, want[0], want[1])
    close(logp, want[2], want[3])
    lost = 2.0 ** -126 * (w * adv).double().abs() / tau
    close(dz, want[4], want[5] + lost[:, None], kind)
