"""The delta rule's gradient and its single tokens on inputs that are parts of wider arrays (GPU)."""
import pytest
import torch

import depthwise_causal_short_gb300 as cc
from depthwise_causal_short_gb300 import _build
from tests import delta_plain as plain

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()
    yield
    assert cc.cattn_device_fault() == 0


def _cu(lens):
    return torch.tensor([0] + list(lens), dtype=torch.int32).cumsum(0).to(torch.int32).cuda()


def _inside(t, at, pitch, heads_apart=None):
    """t [rows, H, C] as a part of rows of `pitch` values, or of heads that each hold all rows."""
    rows, H, C = t.shape
    if heads_apart:
        wide = torch.full((H, rows, C + heads_apart), float("nan"), dtype=t.dtype, device=t.device)
        part = wide[:, :, at:at + C].transpose(0, 1)
    else:
        wide = torch.full((rows, pitch), float("nan"), dtype=t.dtype, device=t.device)
        part = wide[:, at:at + H * C].view(rows, H, C)
    part.copy_(t)
    return part


@pytest.mark.parametrize("heads_apart", [None, 24])
@pytest.mark.parametrize("lens,Hk,Hv,K,V", [([70, 31], 2, 4, 64, 40), ([130, 0, 65], 1, 3, 128, 136), ([3], 3, 3, 24, 8)])
def test_gradient(lens, Hk, Hv, K, V, heads_apart):
    q, k, v, g, beta, do, s0 = (t.cuda() for t in plain.delta_inputs(lens, Hk, Hv, K, V, seed=3))
    total = sum(lens)
    gs = torch.rand(Hv).neg().cuda().expand(total, Hv)          # one decay a head
    bs = torch.rand(Hv, total).cuda().t()                       # heads apart
    want = cc.cattn_delta_bwd(q, k, v, gs.contiguous(), bs.contiguous(), do, _cu(lens), initial_state=s0)
    got = cc.cattn_delta_bwd(_inside(q, 8, 1024, heads_apart), _inside(k, 16, 800, heads_apart), _inside(v, 0, 1032, heads_apart),
                             gs, bs, _inside(do, 24, 2000, heads_apart and 40), _cu(lens), initial_state=s0)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("heads_apart", [None, 24])
@pytest.mark.parametrize("N,Hk,Hv,K,V", [(3, 2, 4, 64, 40), (50, 1, 2, 128, 128), (1, 1, 1, 8, 24)])
def test_single_tokens(N, Hk, Hv, K, V, heads_apart):
    q, k, v, g, beta, do, _ = (t.cuda() for t in plain.delta_inputs([N], Hk, Hv, K, V, seed=4))
    gs = torch.rand(Hv).neg().cuda().expand(N, Hv)
    bs = torch.rand(1, 1).cuda().expand(N, Hv)                  # one step size for all
    pool = torch.randn(N + 2, Hv, K, V).cuda()
    idx = torch.randperm(N + 2)[:N].int().cuda()
    a, b = pool.clone(), pool.clone()
    want, _ = cc.cattn_delta_update(q, k, v, gs.contiguous(), bs.contiguous(), a, idx)
    got, status = cc.cattn_delta_update(_inside(q, 8, 1024, heads_apart), _inside(k, 16, 800, heads_apart),
                                        _inside(v, 0, 1032, heads_apart), gs, bs, b, idx)
    assert status.tolist() == [0, 0] and torch.equal(got, want) and torch.equal(a, b)
