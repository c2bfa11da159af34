"""examples/decay_mixer.py: convolution, norm with rotation and linear attention together (GPU)."""
import importlib.util
import os

import pytest
import torch

from depthwise_causal_short_gb300 import _build
from tests import attn_plain as plain

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "decay_mixer.py")
    spec = importlib.util.spec_from_file_location("decay_mixer", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_prompts_and_tokens_agree_and_train(example):
    # both ways round q, k, v and o to bf16; what differs is the rounding inside the attention
    worst, size, grads = example.main()
    assert worst <= 8e-3 * size
    assert all(torch.isfinite(g).all() and g.any() for g in grads)


def test_the_whole_path_against_64_bits(example):
    m = example.DecayMixer(Hk=1, Hv=2, K=32, V=32)
    lens = [70, 9]
    gen = torch.Generator().manual_seed(3)
    x = torch.randn(sum(lens), m.D, generator=gen).bfloat16()
    g = -torch.rand(sum(lens), m.Hv, generator=gen) * 0.2
    pos = example.positions_of(lens)
    o, _ = m.prompt(x.cuda(), g.cuda(), example.offsets(lens).cuda(), pos.cuda(), m.pools(2),
                    torch.tensor([1, 0], dtype=torch.int32).cuda())
    w = m.conv.double().cpu()
    rows = []
    for part in x.double().split(lens):
        padded = torch.cat((torch.zeros(m.W - 1, m.D, dtype=torch.float64), part))
        z = sum(padded[j:j + part.shape[0]] * w[:, j] for j in range(m.W))
        rows.append(z * torch.sigmoid(z))
    q, k, v = m.split(torch.cat(rows))
    q, k = (plain.norm_rope(t, s.double().cpu(), m.cos.double().cpu(), m.sin.double().cpu(), pos, "rms",
                            1e-6, False) for t, s in ((q, m.wq), (k, m.wk)))
    want, _ = plain.linear(q, k, v, g.double(), [0, 70, 79], m.K ** -0.5)
    # four roundings to bf16 of up to 2^-8 on the way (y, q and k, P or S, o), as independent errors
    assert (o.double().cpu() - want).abs().max() <= 2e-2 * want.abs().max()
