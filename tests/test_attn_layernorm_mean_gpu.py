"""Layer norm of rows that are all one value, or a step or two from it, for row lengths whose reciprocal is no
fp32 number (GPU).

A row of C equal bf16 values x has partial sums k x, k <= C, which fp32 holds exactly (8 + 13 bits); so the
mean, correctly rounded, is x, x - mean is 0 exactly, and so are y without a bias, the weight's gradient and the part
of dx that goes with the normalised row.  A mean that is off by one step of fp32 makes x - mean as large as 4.9e-4
for x = 4992, against sqrt(eps) = 1e-3.
"""
import pytest
import torch

import depthwise_causal_short_gb300 as cc
from depthwise_causal_short_gb300 import _build

pytestmark = pytest.mark.gpu
LENGTHS = [24, 56, 120, 200, 504, 1000, 2040, 7168, 8184]


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()


def _rows(C):
    values = torch.tensor([3.0, 300.0, 1000.0, 4992.0, -0.73, 1e-3, -65280.0]).bfloat16()
    return values[:, None].expand(len(values), C).contiguous()


@pytest.mark.parametrize("C", LENGTHS)
def test_rows_of_one_value_are_their_own_mean(C):
    x = _rows(C).cuda()
    w, b = torch.rand(C).cuda(), torch.rand(C).cuda()
    assert not cc.cattn_layernorm_fwd(x).any()
    many = x.repeat(1000, 1)  # enough rows for every kernel that this length can get
    assert not cc.cattn_layernorm_fwd(many).any()
    want = b.bfloat16().expand_as(x)
    assert torch.equal(cc.cattn_layernorm_fwd(x, w, b), want)  # 0 w + b


@pytest.mark.parametrize("C", LENGTHS)
@pytest.mark.parametrize("gated", [False, True])
def test_their_gradient(C, gated):
    x = _rows(C)
    gen = torch.Generator().manual_seed(C)
    dy, z = (torch.randn(x.shape, generator=gen).bfloat16() for _ in range(2))
    w = 1 + torch.rand(C, generator=gen)
    gate = z.cuda() if gated else None
    dx, dw, _, dz = cc.cattn_layernorm_bwd(x.cuda(), dy.cuda(), w.cuda(), gate=gate)
    assert not dw.any()  # the normalised rows are 0
    assert dz is None or not dz.any()
    # dx = r (dn - mean(dn)), r = 1e3: the store's rounding (half of 2^-7 at most), and the mean's in fp32 (a sum
    # of C terms in a tree of at most 32 + 13 steps, 2^-24 of the row's largest sum each)
    dn = dy.double() * w.double()
    if gated:
        dn = dn * z.double() * torch.sigmoid(z.double())
    want = 1e3 * (dn - dn.mean(-1, keepdim=True))
    slack = 1e3 * (45 * 2.0 ** -24 * dn.abs().mean(-1, keepdim=True) + 2.0 ** -20 * dn.abs())
    assert ((dx.double().cpu() - want).abs() <= 2.0 ** -8 * want.abs() + slack).all()


@pytest.mark.parametrize("C", LENGTHS)
def test_rows_a_step_from_one_value(C):
    # one element of each row is one step of bf16 away: with the mean right to 2^-24 of it, x - mean is right to
    # 2^-24 |x| beside values of at least 2^-8 |x| / C and 2^-8 |x|
    x = torch.full((5, C), 128.0)
    x[:, 3] += 1.0
    x[2:] *= -9.0
    x = x.bfloat16()
    X = x.double()
    d = X - X.mean(-1, keepdim=True)
    sd = torch.sqrt(d.square().mean(-1, keepdim=True) + 1e-6)
    want = d / sd
    got = cc.cattn_layernorm_fwd(x.cuda()).double().cpu()
    off = 2.0 ** -24 * X.abs().amax(-1, keepdim=True)  # of the mean: half a step, and of the sum
    slack = 2 * off / sd + want.abs() * (2.0 ** -20 + 2 * off * d.abs().mean(-1, keepdim=True) / sd.square())
    assert ((got - want).abs() <= 2.0 ** -8 * want.abs() + slack).all()
