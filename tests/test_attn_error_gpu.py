"""The linear attention's errors in the 2-norm, where they average out and a coarser rounding shows (GPU).

Tolerances:
  bf16 results   a stored value is off by at most half a unit of its 8 bits, evenly spread: 2^-7 / sqrt(12) =
                 2.26e-3 of its power of two in the root mean square, and no more of itself.  The
                 operands that the matrix products take rounded (decayed scores; the state in the
                 forward) are terms of sums, each off by as much of itself, independently: as much
                 again.  Together sqrt(2) * 2.26e-3 = 3.2e-3.
  dg             2e-6: its pairs across chunks as in test_attn_linear_gpu.py (1e-6), and as much again
                 for those inside a chunk (fp32 products of the inputs, matrix sums cut off at each of
                 8 steps) and the sums over the tokens.
"""
import pytest
import torch

import depthwise_causal_short_gb300 as cc
from depthwise_causal_short_gb300 import _build
from tests import attn_plain as plain

pytestmark = pytest.mark.gpu
BF16_TOL = 3.2e-3
DG_TOL = 2e-6


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()
    yield
    assert cc.cattn_device_fault() == 0


@pytest.mark.parametrize("lens,Hk,Hv,K,V", [
    ([700, 33, 300], 2, 4, 128, 128), ([1500], 1, 1, 64, 96), ([100, 29, 400], 4, 12, 40, 64),
    ([513, 90], 1, 9, 32, 40), ([128] * 8, 2, 2, 80, 200),
])
@pytest.mark.parametrize("states", [False, True])
def test_errors_in_the_2_norm(lens, Hk, Hv, K, V, states):
    q, k, v, g, do, s0 = plain.linear_inputs(lens, Hk, Hv, K, V, seed=K + V)
    cu = [0] + torch.tensor(lens).cumsum(0).tolist()
    leaves = [t.double().requires_grad_() for t in (q, k, v, g)]
    o, _ = plain.linear(*leaves, cu, K ** -0.5, s0.double() if states else None)
    want = torch.autograd.grad(o, leaves, do.double())
    dcu = torch.tensor(cu, dtype=torch.int32).cuda()
    args, init = [t.cuda() for t in (q, k, v, g)], s0.cuda() if states else None
    got = [cc.cattn_linear_fwd(*args, dcu, initial_state=init)[0],
           *cc.cattn_linear_bwd(*args, do.cuda(), dcu, initial_state=init)[:4]]
    for name, a, b in zip(("o", "dq", "dk", "dv", "dg"), got, (o.detach(), *want)):
        err = float((a.double().cpu() - b).norm() / b.norm())
        assert err <= (DG_TOL if name == "dg" else BF16_TOL), (name, err)
