"""cattn_qknorm_fwd / _bwd against the definition in 64 bits (GPU).

Tolerances, as max |error| / max |reference|: outputs in bf16 carry one rounding of at most
2^-8 of themselves (8 significand bits) on top of fp32 arithmetic (a few 2^-22): 2^-8 * 1.05; the weights' sums
are fp32 sums of N fp32 products in a fixed order, whose error grows like sqrt(N) 2^-24 against
a sum that grows like sqrt(N) at least, with a safety of 20: 2e-6 (2^-8 * 1.05 in bf16).
"""
import pytest
import torch

import depthwise_causal_short_gb300 as cc
from depthwise_causal_short_gb300 import _build
from tests import attn_plain as plain
from tests.helpers import rel_err

pytestmark = pytest.mark.gpu
BF16_TOL = 1.05 * 2.0 ** -8
F32_TOL = 2e-6


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()
    yield
    assert cc.cattn_device_fault() == 0


def _case(rows, hq, hk, dim, rot, wt, seed=0, tab=50):
    gen = torch.Generator().manual_seed(seed)
    q = torch.randn(rows, hq, dim, generator=gen).bfloat16()
    k = torch.randn(rows, hk, dim, generator=gen).bfloat16()
    dyq = torch.randn(rows, hq, dim, generator=gen).bfloat16()
    dyk = torch.randn(rows, hk, dim, generator=gen).bfloat16()
    wq = wk = None
    if wt is not None:
        wq, wk = ((1 + 0.3 * torch.randn(dim, generator=gen)).to(wt) for _ in range(2))
    cos = sin = pos = None
    if rot:
        ang = torch.rand(tab, rot // 2, generator=gen) * 6.28
        cos, sin = ang.cos(), ang.sin()
        pos = torch.randint(0, tab, (rows,), generator=gen).to(torch.int32)
    return q, k, dyq, dyk, wq, wk, cos, sin, pos


def _d(t):
    return None if t is None else t.double()


def _c(t):
    return None if t is None else t.cuda()


def _reference(case, mode, eps, inter):
    q, k, dyq, dyk, wq, wk, cos, sin, pos = case
    out = []
    grads = []
    for x, dy, w in ((q, dyq, wq), (k, dyk, wk)):
        xd = x.double().requires_grad_()
        wd = None if w is None else w.double().requires_grad_()
        y = plain.norm_rope(xd, wd, _d(cos), _d(sin), pos, mode, eps, inter)
        g = torch.autograd.grad(y, [xd] + ([] if wd is None else [wd]), dy.double())
        out.append(y.detach())
        grads.append((g[0], g[1] if w is not None else None))
    return out, grads


CASES = [
    # rows, hq, hk, dim, rot, weights, mode, interleaved
    (1, 1, 1, 8, 0, None, "rms", False), (1, 8, 8, 128, 128, torch.float32, "rms", False),
    (3, 5, 3, 96, 32, None, "l2", True), (17, 2, 1, 64, 64, torch.bfloat16, "l2", False),
    (33, 3, 4, 80, 48, torch.float32, "rms", True), (130, 1, 2, 256, 256, torch.float32, "rms", False),
    (257, 12, 1, 128, 16, torch.bfloat16, "rms", True), (64, 4, 4, 32, 32, torch.float32, "l2", False),
    (777, 8, 2, 24, 16, torch.float32, "rms", False), (2000, 16, 16, 128, 128, torch.float32, "rms", False),
    (5000, 3, 3, 64, 0, torch.float32, "l2", False),
]


@pytest.mark.parametrize("rows,hq,hk,dim,rot,wt,mode,inter", CASES)
def test_parity(rows, hq, hk, dim, rot, wt, mode, inter):
    case = _case(rows, hq, hk, dim, rot, wt, seed=rows + dim)
    out, grads = _reference(case, mode, 1e-6, inter)
    q, k, dyq, dyk, wq, wk, cos, sin, pos = (_c(t) for t in case)
    kw = dict(wq=wq, wk=wk, cos=cos, sin=sin, positions=pos, mode=mode, interleaved=inter)
    yq, yk = cc.cattn_qknorm_fwd(q, k, **kw)
    dq, dk, dwq, dwk = cc.cattn_qknorm_bwd(q, k, dyq, dyk, **kw)
    again = cc.cattn_qknorm_bwd(q, k, dyq, dyk, **kw)
    assert rel_err(yq.double().cpu(), out[0]) <= BF16_TOL
    assert rel_err(yk.double().cpu(), out[1]) <= BF16_TOL
    assert rel_err(dq.double().cpu(), grads[0][0]) <= BF16_TOL
    assert rel_err(dk.double().cpu(), grads[1][0]) <= BF16_TOL
    if wt is None:
        assert dwq is None and dwk is None
    else:
        tol = F32_TOL if wt == torch.float32 else BF16_TOL
        assert rel_err(dwq.double().cpu(), grads[0][1]) <= tol
        assert rel_err(dwk.double().cpu(), grads[1][1]) <= tol
        assert torch.equal(dwq, again[2]) and torch.equal(dwk, again[3])  # a fixed order


def test_strided_views_without_positions():
    # q and k as views of one [total, D] convolution output, rows of the tables in order
    total, hq, hk, dim = 45, 4, 2, 64
    gen = torch.Generator().manual_seed(1)
    x = torch.randn(total, (hq + hk + 3) * dim, generator=gen).bfloat16().cuda()
    q = x[:, :hq * dim].view(total, hq, dim)
    k = x[:, (hq + 1) * dim:(hq + 1 + hk) * dim].view(total, hk, dim)
    ang = torch.rand(total, dim // 2, generator=gen)
    yq, yk = cc.cattn_qknorm_fwd(q, k, cos=ang.cos().cuda(), sin=ang.sin().cuda())
    for x, y in ((q, yq), (k, yk)):
        ref = plain.norm_rope(x.double().cpu(), None, ang.cos().double(), ang.sin().double(), None,
                              "rms", 1e-6, False)
        assert rel_err(y.double().cpu(), ref) <= BF16_TOL


def test_zero_rows_and_zero_values():
    q, k = torch.zeros(0, 2, 64).bfloat16().cuda(), torch.zeros(0, 1, 64).bfloat16().cuda()
    w = torch.ones(64).cuda()
    yq, yk = cc.cattn_qknorm_fwd(q, k)
    assert yq.shape == (0, 2, 64) and yk.shape == (0, 1, 64)
    _, _, dwq, dwk = cc.cattn_qknorm_bwd(q, k, q, k, wq=w, wk=w)
    assert not dwq.any() and not dwk.any()
    # a head of zeros is left at zero (eps > 0), and its neighbours are untouched by it
    q = torch.zeros(3, 2, 64).bfloat16().cuda()
    q[1, 1] = 2.0
    yq, _ = cc.cattn_qknorm_fwd(q, q[:, :1])
    assert not yq[0].any() and torch.allclose(yq[1, 1].float(), torch.ones(64).cuda())


def test_weight_sums_see_no_dead_heads():
    # eps = 0 makes 1/sqrt(0) of heads that do not exist: they must not reach the sums
    gen = torch.Generator().manual_seed(2)
    q = torch.randn(5, 3, 64, generator=gen).bfloat16()
    w = torch.rand(64, generator=gen)
    dy = torch.randn(5, 3, 64, generator=gen).bfloat16()
    _, _, dwq, dwk = cc.cattn_qknorm_bwd(q.cuda(), q.cuda(), dy.cuda(), dy.cuda(), wq=w.cuda(),
                                         wk=w.cuda(), eps=0.0)
    x, wd = q.double(), w.double().requires_grad_()
    ref = torch.autograd.grad(plain.norm_rope(x, wd, None, None, None, "rms", 0.0, False), wd, dy.double())[0]
    assert rel_err(dwq.double().cpu(), ref) <= F32_TOL and rel_err(dwk.double().cpu(), ref) <= F32_TOL


def test_positions_outside_the_table_are_reported():
    q = torch.randn(4, 1, 32).bfloat16().cuda()
    ang = torch.rand(6, 16)
    cos, sin = ang.cos().cuda(), ang.sin().cuda()
    pos = torch.tensor([0, -3, 9, 5], dtype=torch.int32).cuda()
    yq, _ = cc.cattn_qknorm_fwd(q, q, cos=cos, sin=sin, positions=pos)
    near, _ = cc.cattn_qknorm_fwd(q, q, cos=cos, sin=sin, positions=pos.clamp(0, 5))
    assert torch.equal(yq, near)
    assert cc.cattn_device_fault() == 8
    assert cc.cattn_device_fault() == 0


def test_autograd_stream_and_graph():
    case = [_c(t) for t in _case(100, 4, 2, 64, 32, torch.float32, seed=9)]
    q, k, dyq, dyk, wq, wk, cos, sin, pos = case
    kw = dict(wq=wq, wk=wk, cos=cos, sin=sin, positions=pos)
    want = cc.cattn_qknorm_bwd(q, k, dyq, dyk, **kw)
    leaves = [t.clone().requires_grad_() for t in (q, k, wq, wk)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        yq, yk = cc.qk_norm_rope(leaves[0], leaves[1], leaves[2], leaves[3], cos, sin, pos)
        got = torch.autograd.grad((yq, yk), leaves, (dyq, dyk))
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    yq, yk = (torch.empty_like(t) for t in (q, k))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cc.cattn_qknorm_fwd(q, k, yq=yq, yk=yk, **kw)
    q.mul_(-1)
    graph.replay()
    assert torch.equal(yq, cc.cattn_qknorm_fwd(q, k, **kw)[0])
