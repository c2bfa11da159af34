"""The delta rule's results beside the 64-bit results rounded to bf16 once (GPU).

Two results that are rounded alike differ where a step of bf16 lies between them.  With values off by d before the
store (root mean square, of the result's norm) and steps of at most 2^-7 of a value, that happens to a share of at
most d / 2^-7 of them, and leaves a distance of at most sqrt(d 2^-7) of the norm.

  o, dv    d = 1e-6 (products that keep 24 bits of every factor, sums in fp32 of up to 64 + 128 values:
           2^-24 sqrt(192) = 8e-7): 9e-5, so 1e-4
  dq, dk   d = 2^-15: factors of two bf16 terms (2^-18 of each at most, 2^-17 for a product of two), as parts of
           a sum that may cancel to a quarter: 4.9e-4, so 5e-4.  With any factor in one term (2^-9 of it at most,
           2^-9 / sqrt(3) = 1.1e-3 in the root mean square) it is 2e-3 and more.
"""
import pytest
import torch

import depthwise_causal_short_gb300 as cc
from depthwise_causal_short_gb300 import _build
from tests import delta_plain as plain

pytestmark = pytest.mark.gpu

SHAPES = [
    ([700, 33, 300], 2, 4, 128, 128), ([900], 1, 2, 64, 96), ([100, 29, 400], 4, 12, 40, 64),
    ([513, 90], 1, 9, 32, 40), ([64] * 8, 2, 2, 80, 200), ([1, 40, 0, 640], 2, 2, 104, 256),
]


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()
    yield
    assert cc.cattn_device_fault() == 0


def _cu(lens):
    return torch.tensor([0] + list(lens), dtype=torch.int32).cumsum(0).to(torch.int32).cuda()


def _distance(got, want):
    rounded = want.detach().bfloat16().double()
    return float((got.double().cpu() - rounded).norm() / rounded.norm())


@pytest.mark.parametrize("lens,Hk,Hv,K,V", SHAPES)
@pytest.mark.parametrize("states", [False, True])
def test_outputs(lens, Hk, Hv, K, V, states):
    q, k, v, g, beta, do, s0 = plain.delta_inputs(lens, Hk, Hv, K, V, seed=K + V + 1)
    cu = [0] + torch.tensor(lens).cumsum(0).tolist()
    want = plain.delta(*[t.double() for t in (q, k, v, g, beta)], cu, K ** -0.5, s0.double() if states else None)[0]
    args, init = [t.cuda() for t in (q, k, v, g, beta)], s0.cuda() if states else None
    alone = cc.cattn_delta_fwd(*args, _cu(lens), initial_state=init)[0]
    assert _distance(alone, want) <= 1e-4
    # whether a final state is asked for changes nothing in o
    assert torch.equal(alone, cc.cattn_delta_fwd(*args, _cu(lens), initial_state=init, final_state=True)[0])


@pytest.mark.parametrize("lens,Hk,Hv,K,V", SHAPES)
@pytest.mark.parametrize("states", [False, True])
def test_gradients(lens, Hk, Hv, K, V, states):
    q, k, v, g, beta, do, s0 = plain.delta_inputs(lens, Hk, Hv, K, V, seed=K + V + 2)
    cu = [0] + torch.tensor(lens).cumsum(0).tolist()
    leaves = [t.double().requires_grad_() for t in (q, k, v)]
    o = plain.delta(*leaves, g.double(), beta.double(), cu, K ** -0.5, s0.double() if states else None)[0]
    want = torch.autograd.grad(o, leaves, do.double())
    got = cc.cattn_delta_bwd(*[t.cuda() for t in (q, k, v, g, beta, do)], _cu(lens), initial_state=s0.cuda() if states else None)
    for name, tol, a, b in zip(("dq", "dk", "dv"), (5e-4, 5e-4, 1e-4), got, want):
        assert _distance(a, b) <= tol, (name, _distance(a, b))
