"""examples/delta_mixer.py: layer norm, convolution, the delta rule and the gated norm together (GPU)."""
import importlib.util
import os

import pytest
import torch

from depthwise_causal_short_gb300 import _build
from tests import delta_plain as plain

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "delta_mixer.py")
    spec = importlib.util.spec_from_file_location("delta_mixer", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_prompts_and_tokens_agree_and_train(example):
    # both ways round at the same places; what differs is the rounding of products over other numbers of
    # rows, 2^-8 of parts that are as large as the output, in up to four places
    worst, size, grads = example.main()
    assert worst <= 4 * 2.0 ** -8 * size
    assert all(torch.isfinite(g).all() and g.any() for g in grads.values())


def test_the_whole_path_and_its_gradients_against_64_bits(example):
    m = example.DeltaMixer(width=128, Hk=1, Hv=2, K=32, V=32)
    lens = [70, 9]
    gen = torch.Generator().manual_seed(3)
    x = torch.randn(sum(lens), 128, generator=gen).bfloat16()
    cu = example.offsets(lens)

    def norm(t, w, b=None, mean=True):
        c = t - t.mean(-1, keepdim=True) if mean else t
        u = c / torch.sqrt(c.square().mean(-1, keepdim=True) + 1e-6) * w
        return u if b is None else u + b

    def reference(x, w):
        a = norm(x, w["ln_w"], w["ln_b"])
        z = (a @ w["gate"]).view(-1, 2, 32)
        g = -0.1 * torch.nn.functional.softplus(a @ w["decay"])
        beta = torch.sigmoid(a @ w["beta"])
        rows = []
        for part in (a @ w["qkv"]).split(lens):
            padded = torch.cat((torch.zeros(m.W - 1, m.D, dtype=torch.float64), part))
            s = sum(padded[j:j + part.shape[0]] * w["conv"][:, j] for j in range(m.W))
            rows.append(s * torch.sigmoid(s))
        q, k, v = m.split(torch.cat(rows))
        q, k = (t / torch.sqrt(t.square().sum(-1, keepdim=True) + 1e-6) for t in (q, k))
        o, _ = plain.delta(q, k, v, g, beta, cu.tolist(), m.K ** -0.5)
        y = norm(o, w["norm_w"], mean=False) * z * torch.sigmoid(z)
        return x + y.flatten(1) @ w["out"]

    x64 = x.double().requires_grad_()
    w64 = {n: t.double().cpu().requires_grad_() for n, t in m.weights.items()}
    want = reference(x64, w64)
    xg = x.cuda().requires_grad_()
    wg = {n: t.clone().requires_grad_() for n, t in m.weights.items()}
    got = m.train(xg, cu.cuda(), wg)
    prompt, _ = m.prompt(x.cuda(), cu.cuda(), m.pools(2), torch.tensor([1, 0], dtype=torch.int32).cuda())

    def off(a, b):
        return float((a.detach().double().cpu() - b.detach()).norm() / b.detach().norm())

    # a value is rounded to bf16 in eight places on its way (a, the projections, y, q and k, o, the
    # norm, the sum), 2^-8 / sqrt(3) each in the root mean square, and a norm's inputs can be half its size
    assert off(got, want) <= 1e-2 and off(prompt, want) <= 1e-2
    dy = torch.randn(want.shape, generator=gen).bfloat16()
    names = list(wg)
    ours = torch.autograd.grad(got, [xg, *(wg[n] for n in names)], dy.cuda())
    theirs = torch.autograd.grad(want, [x64, *(w64[n] for n in names)], dy.double())
    # and as often again on its way back, through normalised rows whose gradients are differences
    for n, a, b in zip(["x", *names], ours, theirs):
        assert off(a, b) <= 5e-2, (n, off(a, b))
