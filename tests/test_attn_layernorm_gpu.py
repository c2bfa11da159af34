"""cattn_layernorm_fwd / _bwd against the definition in 64 bits (GPU).

Tolerances:
  bf16 results   of an element: 2^-8 of itself (the store's rounding) and, for sums in fp32 of up to C
                 values and exponentials good to 2^-22, 2^-17 of the row's largest value; dx is r
                 times a difference of three terms, so there the row's largest term counts
  dw, db fp32    2e-6 of the largest sum of absolute values over the rows: rows that are summed in
                 order by 13 threads' worth at most between tree steps (40 additions of 2^-24 each
                 along any path), and 2^-20 for the factors
"""
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


def norm(x, w, b, z, mode, eps):
    m = x.mean(-1, keepdim=True) if mode == "layer" else torch.zeros_like(x[..., :1])
    y = (x - m) / torch.sqrt((x - m).square().mean(-1, keepdim=True) + eps)
    y = y if w is None else y * w
    y = y if b is None else y + b
    return y if z is None else y * z * torch.sigmoid(z)


def inputs(shape, wt, bias, gate, seed=0, offset=0.5):
    gen = torch.Generator().manual_seed(seed)

    def randn(*s):
        return torch.randn(*s, generator=gen)

    C = shape[-1]
    x = (randn(*shape) * torch.exp(0.5 * randn(C)) + offset).bfloat16()
    dy = randn(*shape).bfloat16()
    z = randn(*shape).bfloat16() if gate else None
    w = None if wt is None else (1 + 0.2 * randn(C)).to(wt)
    b = (0.2 * randn(C)).to(wt) if bias else None
    return x, dy, w, b, z


def cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


def near(got, want, what, terms=None):
    got, want = got.double().cpu(), want.detach()
    row = (want if terms is None else terms).abs().amax(-1, keepdim=True)
    worst = ((got - want).abs() - 2.0 ** -8 * want.abs() - 2.0 ** -17 * row).max().item() if want.numel() else 0.0
    assert worst <= 0, f"{what}: off by {worst:.3g} more than allowed"


F32, BF16 = torch.float32, torch.bfloat16
CASES = [
    # shape, weight type, bias, gate
    ((1, 8), F32, True, True), ((3, 1, 8), None, False, False), ((5, 3, 24), BF16, True, True),
    ((7, 2, 32), F32, False, True), ((9, 5, 40), F32, True, False), ((33, 64), BF16, False, True),
    ((4, 16, 128), F32, False, True), ((300, 3, 120), F32, True, True), ((100, 136), F32, True, True),
    ((50, 2, 256), BF16, True, False), ((41, 264), F32, True, True), ((17, 2, 512), None, False, True),
    ((13, 520), F32, True, True), ((6, 1024), BF16, True, True), ((11, 1032), F32, True, True),
    ((5, 2048), F32, True, False), ((9, 2056), BF16, True, True), ((700, 4096), F32, True, True),
    ((3, 4104), F32, True, True), ((2, 2, 8192), BF16, True, True), ((2000, 16, 128), F32, True, True),
    ((20000, 8), F32, True, True), ((6000, 200), F32, True, False), ((5000, 256), None, False, False),
    ((2600, 504), BF16, True, False), ((1300, 1000), F32, True, False), ((1250, 1024), F32, True, False),
    ((90, 1000), F32, False, False),
]


@pytest.mark.parametrize("shape,wt,bias,gate", CASES)
@pytest.mark.parametrize("mode", ["layer", "rms"])
def test_parity(shape, wt, bias, gate, mode):
    x, dy, w, b, z = inputs(shape, wt, bias, gate, seed=sum(shape))
    leaves = [None if t is None else t.double().requires_grad_() for t in (x, w, b, z)]
    y = norm(*leaves, mode, 1e-6)
    gx, gdy, gw, gb, gz = cuda(x, dy, w, b, z)
    got = cc.cattn_layernorm_fwd(gx, gw, gb, gate=gz, mode=mode)
    assert got.shape == x.shape and got.dtype == BF16
    near(got, y, "y")
    given = [t for t in leaves if t is not None]
    grads = iter(torch.autograd.grad(y, given, dy.double()))
    dx, dw, db, dz = (None if t is None else next(grads) for t in leaves)
    out = cc.cattn_layernorm_bwd(gx, gdy, gw, gb, gate=gz, mode=mode)
    again = cc.cattn_layernorm_bwd(gx, gdy, gw, gb, gate=gz, mode=mode)
    for a, c in zip(out, again):
        assert (a is None and c is None) or torch.equal(a, c)  # a fixed order
    for a, c in zip(out, (dx, dw, db, dz)):
        assert (a is None) == (c is None)
    # the terms of dx: r dn, and n times a mean of products
    X = leaves[0].detach()
    m = X.mean(-1, keepdim=True) if mode == "layer" else 0.0
    r = 1 / torch.sqrt((X - m).square().mean(-1, keepdim=True) + 1e-6)
    sz = 1.0 if z is None else (z.double() * torch.sigmoid(z.double())).abs()
    du = dy.double().abs() * sz
    dn = du if w is None else du * w.double().abs()
    n = ((X - m) * r).abs()
    near(out[0], dx, "dx", r * (dn + dn.mean(-1, keepdim=True) + n * (dn * n).mean(-1, keepdim=True)))
    if z is not None:
        u = n if w is None else n * w.double().abs()
        u = u if b is None else u + b.double().abs()
        near(out[3], dz, "dz", u * dy.double().abs())
    dims = tuple(range(x.dim() - 1))
    for a, c, sizes, name in ((out[1], dw, du * n, "dw"), (out[2], db, du, "db")):
        if a is None:
            continue
        step = 0.0 if a.dtype == F32 else 2.0 ** -8
        worst = ((a.double().cpu() - c).abs() - step * c.abs()).max().item()
        assert worst <= 2e-6 * sizes.expand(x.shape).sum(dims).max().item(), (name, worst)


def test_strides_and_outputs_in_place_of_new_ones():
    # rows inside wider ones, heads apart, as a projection's output has them
    wide = torch.randn(37, 6, 200).bfloat16().cuda()
    x, z, dy = wide[:, :3, 8:136], wide[:, 3:, 72:200], wide[:, 1:4, :128]
    w = torch.randn(128).cuda()
    want = cc.cattn_layernorm_fwd(x.contiguous(), w, gate=z.contiguous(), mode="rms")
    y = torch.empty_like(want)
    assert cc.cattn_layernorm_fwd(x, w, gate=z, mode="rms", y=y) is not None and torch.equal(y, want)
    a = cc.cattn_layernorm_bwd(x.contiguous(), dy.contiguous(), w, gate=z.contiguous())
    outs = [torch.empty_like(t) for t in (a[0], a[1], a[3])]
    ws = torch.empty(cc.cattn_layernorm_bwd_workspace_bytes(37, 3, 128), dtype=torch.uint8, device="cuda")
    cc.cattn_layernorm_bwd(x, dy, w, gate=z, dx=outs[0], dw=outs[1], dgate=outs[2], workspace=ws)
    assert all(torch.equal(p, q) for p, q in zip(outs, (a[0], a[1], a[3])))


def test_no_rows():
    x = torch.empty(0, 3, 64, dtype=BF16, device="cuda")
    w, b = torch.ones(64, device="cuda"), torch.ones(64, device="cuda")
    assert cc.cattn_layernorm_fwd(x, w, b).shape == x.shape
    dx, dw, db, dz = cc.cattn_layernorm_bwd(x, x, w, b, gate=x)
    assert dx.shape == dz.shape == x.shape and not dw.any() and not db.any()


def test_constant_rows_far_from_zero():
    # the variance of rows that differ from their mean by one step of bf16: summed around the mean
    x = torch.full((5, 256), 128.0)
    x[:, ::2] += 1.0
    x = x.bfloat16()
    y = cc.cattn_layernorm_fwd(x.cuda()).cpu()
    near(y, norm(x.double(), None, None, None, "layer", 1e-6), "y")
    same = torch.full((4, 2, 96), 3.0, dtype=BF16, device="cuda")
    assert not cc.cattn_layernorm_fwd(same).any()  # (x - mean) = 0 exactly


def test_eps_zero_and_idle_rows():
    # 3 rows in a CTA that has room for more: what is not there must not reach the sums
    x, dy, w, b, z = inputs((3, 40), F32, True, True, seed=4)
    gx, gdy, gw, gb, gz = cuda(x, dy, w, b, z)
    for mode in ("layer", "rms"):
        out = cc.cattn_layernorm_bwd(gx, gdy, gw, gb, gate=gz, mode=mode, eps=0.0)
        assert all(torch.isfinite(t).all() for t in out)


def test_a_row_of_nan_stays_in_its_row():
    x, dy, w, b, z = cuda(*inputs((6, 3, 120), F32, True, True, seed=8))
    clean = cc.cattn_layernorm_fwd(x, w, b, gate=z)
    x[2, 1, 7] = float("nan")
    x[4, 0, 3] = float("inf")
    y = cc.cattn_layernorm_fwd(x, w, b, gate=z)
    bad = torch.zeros(6, 3, dtype=torch.bool, device="cuda")
    bad[2, 1] = bad[4, 0] = True
    assert torch.equal(y[~bad], clean[~bad]) and y[2, 1].isnan().all()


def test_gate_far_out():
    # silu and its derivative at the ends: 0 and z, no NaN from exp of large values
    z = torch.tensor([-3e4, -200.0, -90.0, 0.0, 90.0, 200.0, 3e4, 1.0]).bfloat16().expand(2, 8).contiguous()
    x = torch.randn(2, 8).bfloat16()
    dy = torch.randn(2, 8).bfloat16()
    near(cc.cattn_layernorm_fwd(x.cuda(), gate=z.cuda()), norm(x.double(), None, None, z.double(), "layer", 1e-6), "y")
    out = cc.cattn_layernorm_bwd(x.cuda(), dy.cuda(), gate=z.cuda())
    assert all(torch.isfinite(out[i]).all() for i in (0, 3))


def test_on_another_stream_and_in_a_graph():
    x, dy, w, b, z = cuda(*inputs((50, 4, 128), F32, True, True, seed=2))
    want = [cc.cattn_layernorm_fwd(x, w, b, gate=z), *cc.cattn_layernorm_bwd(x, dy, w, b, gate=z)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [cc.cattn_layernorm_fwd(x, w, b, gate=z, stream=side),
           *cc.cattn_layernorm_bwd(x, dy, w, b, gate=z, stream=side)]
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, c) for a, c in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = [cc.cattn_layernorm_fwd(x, w, b, gate=z), *cc.cattn_layernorm_bwd(x, dy, w, b, gate=z)]
    for t in held:
        t.zero_()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(held, want))
