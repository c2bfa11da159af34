"""Layer norm's forward on both sides of each number of rows where another kernel is taken (GPU)."""
import pytest
import torch

import depthwise_causal_short_gb300 as cc
from depthwise_causal_short_gb300 import _build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()


@pytest.mark.parametrize("C,ctas,rows_of_a_cta", [(136, 8, 32), (256, 8, 32), (264, 1, 16), (512, 1, 16), (520, 1, 8), (1024, 1, 8)])
@pytest.mark.parametrize("mode", ["layer", "rms"])
def test_either_side(C, ctas, rows_of_a_cta, mode):
    least = torch.cuda.get_device_properties(0).multi_processor_count * ctas * rows_of_a_cta
    gen = torch.Generator().manual_seed(C)
    x = (torch.randn(least, C, generator=gen) + 0.5).bfloat16().cuda()
    w, b = torch.randn(C, generator=gen).cuda(), torch.randn(C, generator=gen).cuda()

    def name(rows):
        return cc.attn_describe(lambda: cc.cattn_layernorm_fwd(x[:rows], w, b, mode=mode))[0]["name"]

    assert name(least) != name(least - 1)
    X = x.double()
    m = X.mean(-1, keepdim=True) if mode == "layer" else 0.0
    n = (X - m) / torch.sqrt((X - m).square().mean(-1, keepdim=True) + 1e-6)
    want = n * w.double() + b.double()
    # the store's rounding, half of 2^-7 at most; and 2^-17 of the row's largest value (sums in fp32 of C values)
    slack = 2.0 ** -17 * ((n * w.double()).abs() + b.double().abs()).amax(-1, keepdim=True)
    for rows in (least, least - 1):
        y = cc.cattn_layernorm_fwd(x[:rows], w, b, mode=mode).double()
        assert ((y - want[:rows]).abs() <= 2.0 ** -8 * want[:rows].abs() + slack[:rows]).all()
