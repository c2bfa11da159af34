"""cattn_linear_fwd / _bwd / _update against the definition in 64 bits (GPU).

Tolerances, as max |error| / max |reference|:
  bf16 results   8e-3: the store rounds by up to 2^-8 (3.9e-3); the matrix operands that are not
                 inputs (decayed scores, the state) are rounded too, and their errors are
                 independent: 1.7e-3 of the result's norm, of which an element sees less than
                 4.5 sigma, against a largest element of at least 3 sigma (2.6e-3), and as much
                 again where terms cancel
  fp32 states    5e-6: products split so that 2^-24 of each is kept, fp32 sums
  dg             2e-5: fp32 sums of pairs whose state factor is kept to 2^-17 (7.6e-6), summed
                 over the tokens after it
"""
import pytest
import torch

import depthwise_causal_short_gb300 as cc
from depthwise_causal_short_gb300 import _build
from tests import attn_plain as plain
from tests.helpers import rel_err

pytestmark = pytest.mark.gpu
BF16_TOL = 8e-3
STATE_TOL = 5e-6
DG_TOL = 2e-5


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()
    yield
    assert cc.cattn_device_fault() == 0


def cu_of(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def _cu(lens):
    return torch.tensor(cu_of(lens), dtype=torch.int32).cuda()


CASES = [
    # lengths, Hk, Hv, K, V
    ([1], 1, 1, 8, 8), ([0], 2, 2, 16, 24), ([0, 1, 0], 1, 2, 64, 64), ([127], 1, 1, 128, 128),
    ([128], 2, 2, 128, 128), ([129], 1, 2, 128, 64), ([63, 64, 65, 0, 1, 200, 31], 2, 4, 128, 128),
    ([257, 300], 1, 3, 96, 40), ([5, 500], 1, 1, 40, 136), ([384], 1, 8, 32, 128),
    ([130, 2, 126], 3, 3, 72, 256), ([700], 1, 1, 64, 96), ([1] * 40, 2, 2, 64, 32),
    ([1000], 1, 1, 128, 128), ([1, 255, 256, 1], 1, 2, 120, 200),
    # more chunks than SMs: ranges of several chunks, heads and sequences
    ([1] * 200, 1, 4, 32, 32), ([128] * 20 + [5] * 20, 2, 8, 32, 32), ([700, 0, 1300], 2, 16, 32, 40),
    ([2500], 8, 8, 16, 16), ([90, 2, 300] * 5, 4, 16, 24, 136),
]


def _check(a, b, tol, what):
    e = rel_err(a.detach().double().cpu(), b)
    assert e <= tol, f"{what}: {e:.3g} > {tol:.3g}"


@pytest.mark.parametrize("lens,Hk,Hv,K,V", CASES)
@pytest.mark.parametrize("states", [False, True])
def test_parity(lens, Hk, Hv, K, V, states):
    q, k, v, g, do, s0 = plain.linear_inputs(lens, Hk, Hv, K, V, seed=sum(lens) + K)
    scale = K ** -0.5
    leaves = [t.double().requires_grad_() for t in (q, k, v, g, s0)]
    o, fin = plain.linear(*leaves[:4], cu_of(lens), scale, leaves[4] if states else None)
    args = [t.cuda() for t in (q, k, v, g)]
    cu = _cu(lens)
    init = s0.cuda() if states else None
    go, gfin, status = cc.cattn_linear_fwd(*args, cu, initial_state=init, final_state=True)
    assert status is None
    _check(gfin, fin.detach(), STATE_TOL, "final state")
    if sum(lens):
        _check(go, o.detach(), BF16_TOL, "o")
    alone, none, _ = cc.cattn_linear_fwd(*args, cu, initial_state=init)
    assert none is None and torch.equal(alone, go)

    grads = cc.cattn_linear_bwd(*args, do.cuda(), cu, initial_state=init)
    again = cc.cattn_linear_bwd(*args, do.cuda(), cu, initial_state=init)
    for a, b in zip(grads, again):
        assert (a is None and b is None) or torch.equal(a, b)  # a fixed order
    if not sum(lens):
        assert not states or not grads[4].any()
        return
    want = torch.autograd.grad(o, leaves if states else leaves[:4], do.double(), allow_unused=True)
    for name, a, b in zip(("dq", "dk", "dv"), grads, want):
        _check(a, b, BF16_TOL, name)
    _check(grads[3], want[3], DG_TOL, "dg")
    if states:
        _check(grads[4], want[4], STATE_TOL, "d_initial_state")


@pytest.mark.parametrize("lens,Hk,Hv,K,V,states", [
    ([90, 2, 300] * 5, 4, 16, 24, 136, False), ([1] * 300, 2, 4, 32, 32, False),
    ([128, 5, 0, 129] * 12, 4, 8, 64, 64, True), ([1500, 33, 800], 8, 16, 128, 128, False),
    ([64, 400, 1, 128, 0, 0] * 8, 1, 8, 72, 256, False),
])
def test_repeats_are_bit_identical(lens, Hk, Hv, K, V, states):
    # many chunks that need no state, short ranges, several tiles of V: the roles of a CTA drift
    # apart as far as they can here, and every run must still meet at the same places
    q, k, v, g, do, s0 = (t.cuda() for t in plain.linear_inputs(lens, Hk, Hv, K, V, seed=K))
    cu, init = _cu(lens), s0 if states else None
    first = None
    for _ in range(25):
        got = [t for t in (*cc.cattn_linear_bwd(q, k, v, g, do, cu, initial_state=init),
                           *cc.cattn_linear_fwd(q, k, v, g, cu, initial_state=init, final_state=True)[:2])
               if t is not None]
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(got, first))
    assert cc.cattn_device_fault() == 0


def test_gradients_against_differences():
    # the loss's change along random directions, from the 64-bit forward, against the kernel's
    # gradients: they carry the bf16 tolerance, of the sum of their parts' sizes
    lens, Hk, Hv, K, V = [90, 170], 1, 2, 64, 64
    q, k, v, g, do, s0 = plain.linear_inputs(lens, Hk, Hv, K, V, seed=5)
    cu = cu_of(lens)
    grads = cc.cattn_linear_bwd(q.cuda(), k.cuda(), v.cuda(), g.cuda(), do.cuda(), _cu(lens),
                                initial_state=s0.cuda())
    base = [t.double() for t in (q, k, v, g, s0)]
    gen = torch.Generator().manual_seed(7)
    for i in range(5):
        d = torch.randn(base[i].shape, generator=gen, dtype=torch.float64)
        loss = []
        for sign in (1, -1):
            args = list(base)
            args[i] = base[i] + sign * 1e-4 * d
            loss.append((plain.linear(*args[:4], cu, K ** -0.5, args[4])[0] * do.double()).sum())
        slope = (loss[0] - loss[1]).item() / 2e-4
        got = (grads[i].double().cpu() * d).sum().item()
        size = (grads[i].double().cpu() * d).norm().item()
        assert abs(slope - got) <= 1e-2 * size + 1e-4 * abs(slope), (i, slope, got, size)


def _views(lens, Hk, Hv, K, V, seed):
    """q, k, v as views into one [total, D] buffer, g as a transposed view."""
    q, k, v, g, do, s0 = plain.linear_inputs(lens, Hk, Hv, K, V, seed)
    total = sum(lens)
    buf = torch.zeros(total, 2 * Hk * K + Hv * V + 16).bfloat16()
    at = 8
    out = []
    for t, n in ((q, Hk * K), (k, Hk * K), (v, Hv * V)):
        buf[:, at:at + n] = t.reshape(total, n)
        out.append((at, n, t.shape))
        at += n
    gb = buf.cuda()
    views = [gb[:, a:a + n].view(shape) for a, n, shape in out]
    gt = g.t().contiguous().cuda().t()
    return (q, k, v, g, do, s0), views, gt


def test_strided_inputs_and_shared_gate():
    lens, Hk, Hv, K, V = [70, 190], 2, 4, 64, 80
    (q, k, v, g, do, s0), views, gt = _views(lens, Hk, Hv, K, V, 11)
    cu = _cu(lens)
    want = cc.cattn_linear_fwd(q.cuda(), k.cuda(), v.cuda(), g.cuda(), cu)[0]
    assert torch.equal(cc.cattn_linear_fwd(*views, gt, cu)[0], want)
    a = cc.cattn_linear_bwd(q.cuda(), k.cuda(), v.cuda(), g.cuda(), do.cuda(), cu)
    b = cc.cattn_linear_bwd(*views, gt, do.transpose(0, 1).contiguous().cuda().transpose(0, 1), cu)
    for x, y in zip(a[:4], b[:4]):
        assert torch.equal(x, y)
    # one decay per head, expanded over the tokens; its gradient is the sum over them
    lam = -torch.rand(Hv).cuda() * 0.1
    lam.requires_grad_()
    o, _ = cc.decay_attention(q.cuda(), k.cuda(), v.cuda(), lam.expand(sum(lens), Hv), cu)
    dlam = torch.autograd.grad(o, lam, do.cuda())[0]
    lam64 = lam.detach().double().cpu().requires_grad_()
    ref, _ = plain.linear(q.double(), k.double(), v.double(), lam64.expand(sum(lens), Hv), cu_of(lens),
                          K ** -0.5)
    want = torch.autograd.grad(ref, lam64, do.double())[0]
    _check(o, ref.detach(), BF16_TOL, "o")
    _check(dlam, want, DG_TOL, "dlam")


@pytest.mark.parametrize("kind", ["reset", "zero", "steep", "mixed"])
def test_extreme_decays(kind):
    lens, Hk, Hv, K, V = [300, 40], 1, 2, 64, 64
    q, k, v, g, do, s0 = plain.linear_inputs(lens, Hk, Hv, K, V, seed=13)
    if kind == "reset":
        g[[5, 100, 127, 128, 129, 310]] = float("-inf")
    elif kind == "zero":
        g.zero_()
    elif kind == "steep":
        g.fill_(-60.0)
    else:
        g[::3] = -40.0
        g[1::50] = -1e30
    leaves = [t.double().requires_grad_() for t in (q, k, v, g.clamp(min=-1e4), s0)]
    o, fin = plain.linear(*leaves[:4], cu_of(lens), K ** -0.5, leaves[4])
    want = torch.autograd.grad(o, leaves, do.double())
    args = [t.cuda() for t in (q, k, v, g)]
    go, gfin, _ = cc.cattn_linear_fwd(*args, _cu(lens), initial_state=s0.cuda(), final_state=True)
    grads = cc.cattn_linear_bwd(*args, do.cuda(), _cu(lens), initial_state=s0.cuda())
    _check(go, o.detach(), BF16_TOL, "o")
    _check(gfin, fin.detach(), STATE_TOL, "final state")
    for name, a, b in zip(("dq", "dk", "dv"), grads, want):
        _check(a, b, BF16_TOL, name)
    _check(grads[3], want[3], DG_TOL, "dg")
    _check(grads[4], want[4], STATE_TOL, "d_initial_state")


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_other_sequences_never_see_non_finite_values(bad):
    lens, Hk, Hv, K, V = [70, 33, 200, 0, 9], 1, 2, 64, 64
    q, k, v, g, do, s0 = plain.linear_inputs(lens, Hk, Hv, K, V, seed=17)
    cu = cu_of(lens)
    clean = [t.cuda() for t in (q, k, v, g)]
    want = cc.cattn_linear_fwd(*clean, _cu(lens), initial_state=s0.cuda(), final_state=True)
    gwant = cc.cattn_linear_bwd(*clean, do.cuda(), _cu(lens), initial_state=s0.cuda())
    for which in range(6):
        t = [x.clone() for x in (q, k, v, g, do, s0)]
        t[which][1 if which == 5 else slice(cu[1], cu[2])] = bad
        c = [x.cuda() for x in t]
        o, fin, _ = cc.cattn_linear_fwd(*c[:4], _cu(lens), initial_state=c[5], final_state=True)
        grads = cc.cattn_linear_bwd(*c[:5], _cu(lens), initial_state=c[5])
        rows = [i for i in range(sum(lens)) if not cu[1] <= i < cu[2]]
        seqs = [0, 2, 3, 4]
        assert torch.equal(o[rows], want[0][rows]) and torch.equal(fin[seqs], want[1][seqs])
        for a, b in zip(grads[:4], gwant[:4]):
            assert torch.equal(a[rows], b[rows])
        assert torch.equal(grads[4][seqs], gwant[4][seqs])


def test_pool_slots_in_place_and_bad_indices():
    lens, Hk, Hv, K, V = [150, 0, 40, 290], 1, 2, 64, 32
    q, k, v, g, do, _ = plain.linear_inputs(lens, Hk, Hv, K, V, seed=19)
    args = [t.cuda() for t in (q, k, v, g)]
    pool0 = torch.randn(9, Hv, K, V).cuda()
    idx = torch.tensor([7, 0, 3, 5], dtype=torch.int32).cuda()
    want, fin, _ = cc.cattn_linear_fwd(*args, _cu(lens), initial_state=pool0[idx.long()].contiguous(),
                                       final_state=True)
    pool = pool0.clone()
    o, out, status = cc.cattn_linear_fwd(*args, _cu(lens), initial_state=pool, final_state=pool,
                                         state_indices=idx)
    assert out is pool and status.tolist() == [0, 0]
    assert torch.equal(o, want) and torch.equal(pool[idx.long()], fin)
    rest = [s for s in range(9) if s not in idx.tolist()]
    assert torch.equal(pool[rest], pool0[rest])
    ref = cc.cattn_linear_bwd(*args, do.cuda(), _cu(lens), initial_state=pool0[idx.long()].contiguous())
    st = torch.zeros(2, dtype=torch.int32).cuda()
    got = cc.cattn_linear_bwd(*args, do.cuda(), _cu(lens), initial_state=pool0, state_indices=idx,
                              status=st)
    for a, b in zip(got, ref):
        assert torch.equal(a, b)
    for vec, bits in (([7, -1, 3, 5], 1), ([7, 9, 3, 5], 2), ([7, 3, 3, 5], 4), ([-2, 11, 5, 5], 7)):
        pool = pool0.clone()
        bad = torch.tensor(vec, dtype=torch.int32).cuda()
        o, _, status = cc.cattn_linear_fwd(*args, _cu(lens), initial_state=pool, final_state=pool,
                                           state_indices=bad)
        assert status.tolist() == [-8, bits] and torch.equal(pool, pool0)
        zero = torch.cat([pool0, torch.zeros_like(pool0[:1])])
        use = torch.tensor([s if 0 <= s < 9 else 9 for s in vec]).cuda()
        want = cc.cattn_linear_fwd(*args, _cu(lens), initial_state=zero[use].contiguous())[0]
        assert torch.equal(o, want)


def test_ill_formed_offsets_are_reported_and_stay_inside():
    lens, Hk, Hv, K, V = [50, 60], 1, 1, 64, 64
    q, k, v, g, do, _ = (t.cuda() for t in plain.linear_inputs(lens, Hk, Hv, K, V, seed=23))
    for vec in ([0, 90, 70], [0, 50, 5000], [-7, 50, 110], [3, 50, 110]):
        cu = torch.tensor(vec, dtype=torch.int32).cuda()
        cc.cattn_linear_fwd(q, k, v, g, cu, final_state=True)
        assert cc.cattn_device_fault() == 4
        cc.cattn_linear_bwd(q, k, v, g, do, cu)
        assert cc.cattn_device_fault() == 4
    assert cc.cattn_device_fault() == 0


def test_streams_graph_and_workspace():
    lens, Hk, Hv, K, V = [400, 120], 2, 4, 128, 128
    q, k, v, g, do, s0 = (t.cuda() for t in plain.linear_inputs(lens, Hk, Hv, K, V, seed=29))
    cu = _cu(lens)
    want = cc.cattn_linear_fwd(q, k, v, g, cu, initial_state=s0, final_state=True)
    gwant = cc.cattn_linear_bwd(q, k, v, g, do, cu, initial_state=s0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ws = torch.full((cc.cattn_linear_bwd_workspace_bytes(520, 2, Hk, Hv, K, V),), 255,
                    dtype=torch.uint8, device="cuda")
    got = cc.cattn_linear_bwd(q, k, v, g, do, cu, initial_state=s0, workspace=ws, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(got, gwant):
        assert torch.equal(a, b)
    o = torch.empty_like(want[0])
    ws = torch.full((max(16, cc.cattn_linear_fwd_workspace_bytes(520, 2, Hk, Hv, K, V)),), 255,
                    dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cc.cattn_linear_fwd(q, k, v, g, cu, initial_state=s0, o=o, workspace=ws)
    o.zero_()
    graph.replay()
    assert torch.equal(o, want[0])
    v.neg_()
    s0.neg_()
    graph.replay()
    assert torch.equal(o, -want[0])
    with pytest.raises(cc.CConvError, match="WORKSPACE"):
        cc.cattn_linear_bwd(q, k, v, g, do, cu, workspace=ws[:16])


def test_autograd():
    lens, Hk, Hv, K, V = [64, 100], 1, 2, 64, 64
    q, k, v, g, do, s0 = (t.cuda() for t in plain.linear_inputs(lens, Hk, Hv, K, V, seed=31))
    cu = _cu(lens)
    leaves = [t.clone().requires_grad_() for t in (q, k, v, g, s0)]
    o, fin = cc.decay_attention(*leaves[:4], cu, leaves[4], scale=0.5, output_final_state=True)
    assert not fin.requires_grad
    got = torch.autograd.grad(o, leaves, do)
    want = cc.cattn_linear_bwd(q, k, v, g, do, cu, scale=0.5, initial_state=s0)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


# ---------------------------------------------------------------------------------------
# single tokens
# ---------------------------------------------------------------------------------------

@pytest.mark.parametrize("N,S,Hk,Hv,K,V", [
    (1, 1, 1, 1, 8, 8), (1, 4, 8, 16, 128, 128), (3, 7, 1, 2, 64, 96), (5, 5, 2, 2, 40, 24),
    (17, 40, 1, 3, 72, 256), (70, 90, 2, 4, 128, 64), (2, 3, 1, 1, 128, 136),
])
def test_update(N, S, Hk, Hv, K, V):
    q, k, v, g, _, _ = plain.linear_inputs([1] * N, Hk, Hv, K, V, seed=N + V)
    pool = torch.randn(S, Hv, K, V)
    idx = torch.randperm(S)[:N].to(torch.int32)
    s0 = pool[idx.long()].double()
    o, fin = plain.linear(q.double(), k.double(), v.double(), g.double(), list(range(N + 1)),
                          K ** -0.5, s0)
    gp = pool.cuda()
    args = [t.cuda() for t in (q, k, v, g)]
    go, status = cc.cattn_linear_update(*args, gp, idx.cuda())
    assert status.tolist() == [0, 0]
    _check(go, o, 1.05 * 2 ** -8, "o")
    # one multiply-add a value and expf: a few 2^-23
    _check(gp[idx.long().cuda()], fin, 1e-6, "state")
    rest = [s for s in range(S) if s not in idx.tolist()]
    assert torch.equal(gp.cpu()[rest], pool[rest])
    # without indices row i is slot i
    gp2 = pool[idx.long()].contiguous().cuda()
    go2, status = cc.cattn_linear_update(*args, gp2, status=torch.full((2,), 9, dtype=torch.int32).cuda())
    assert status.tolist() == [0, 0]
    assert torch.equal(go2, go) and torch.equal(gp2, gp[idx.long().cuda()])


def test_update_padding_and_bad_indices():
    N, S, Hk, Hv, K, V = 6, 9, 1, 2, 64, 64
    q, k, v, g, _, _ = (t.cuda() for t in plain.linear_inputs([1] * N, Hk, Hv, K, V, seed=3))
    pool0 = torch.randn(S, Hv, K, V).cuda()
    idx = torch.tensor([4, -1, 2, 8, -1, 0], dtype=torch.int32).cuda()
    pool, o = pool0.clone(), torch.full((N, Hv, V), 7.0).bfloat16().cuda()
    cc.cattn_linear_update(q, k, v, g, pool, idx, pad_rows=True, o=o)
    live = [0, 2, 3, 5]
    want, _ = cc.cattn_linear_update(q[live], k[live], v[live], g[live].contiguous(), p2 := pool0.clone(),
                                     idx[live])
    assert torch.equal(o[live], want) and torch.equal(pool, p2)
    assert (o[[1, 4]] == 7).all()
    for vec, pad, bits in (([4, -1, 2, 8, 1, 0], False, 1), ([4, -2, 2, 8, 1, 0], True, 1),
                           ([4, 9, 2, 8, 1, 0], True, 2), ([4, 3, 3, 8, 1, 0], True, 4)):
        pool, o = pool0.clone(), torch.full((N, Hv, V), 7.0).bfloat16().cuda()
        _, status = cc.cattn_linear_update(q, k, v, g, pool, torch.tensor(vec, dtype=torch.int32).cuda(),
                                           pad_rows=pad, o=o)
        assert status.tolist() == [-8, bits]
        assert torch.equal(pool, pool0) and (o == 7).all()


@pytest.mark.parametrize("nseq", [31, 32, 33, 70])
def test_state_indices_of_few_and_many_sequences(nseq):
    # up to 32 sequences (rows) the kernels check indices and offsets themselves
    lens = [(7 * i) % 5 for i in range(nseq)]
    Hk, Hv, K, V = 1, 2, 16, 16
    q, k, v, g, do, _ = (t.cuda() for t in plain.linear_inputs(lens, Hk, Hv, K, V, seed=nseq))
    pool0 = torch.randn(nseq + 3, Hv, K, V).cuda()
    idx = torch.randperm(nseq + 3)[:nseq].to(torch.int32).cuda()
    ref, fin, _ = cc.cattn_linear_fwd(q, k, v, g, _cu(lens), final_state=True,
                                      initial_state=pool0[idx.long()].contiguous())
    rq, rk, rv, rg, _, _ = (t.cuda() for t in plain.linear_inputs([1] * nseq, Hk, Hv, K, V, seed=1))
    for at, bad, bits in ((0, None, 0), (nseq - 1, -1, 1), (nseq - 2, nseq + 3, 2), (nseq - 1, int(idx[0]), 4)):
        use = idx.clone()
        if bad is not None:
            use[at] = bad
        pool = pool0.clone()
        o, _, status = cc.cattn_linear_fwd(q, k, v, g, _cu(lens), initial_state=pool, final_state=pool,
                                           state_indices=use)
        st = torch.full((2,), 9, dtype=torch.int32).cuda()
        cc.cattn_linear_bwd(q, k, v, g, do, _cu(lens), initial_state=pool0, state_indices=use, status=st)
        assert status.tolist() == st.tolist() == [-8 if bits else 0, bits]
        _, up = cc.cattn_linear_update(rq, rk, rv, rg, p2 := pool0.clone(), use)
        assert up.tolist() == status.tolist()
        if bits:
            assert torch.equal(pool, pool0) and torch.equal(p2, pool0)
        else:
            assert torch.equal(o, ref) and torch.equal(pool[idx.long()], fin)
    cu = _cu(lens)
    cu[nseq // 2] = 1 << 20
    cc.cattn_linear_fwd(q, k, v, g, cu)
    assert cc.cattn_device_fault() == 4
    cc.cattn_linear_bwd(q, k, v, g, do, cu)
    assert cc.cattn_device_fault() == 4


def test_prompt_then_tokens_equal_the_whole_sequence():
    lens, Hk, Hv, K, V = [140], 1, 2, 64, 64
    q, k, v, g, _, _ = plain.linear_inputs(lens, Hk, Hv, K, V, seed=41)
    o, fin = plain.linear(q.double(), k.double(), v.double(), g.double(), [0, 140], K ** -0.5)
    args = [t.cuda() for t in (q, k, v, g)]
    pool = torch.zeros(3, Hv, K, V).cuda()
    idx = torch.tensor([2], dtype=torch.int32).cuda()
    cc.cattn_linear_fwd(*[t[:130] for t in args], _cu([130]), final_state=pool, state_indices=idx)
    for t in range(130, 140):
        y, _ = cc.cattn_linear_update(*[x[t:t + 1] for x in args], pool, idx)
        _check(y, o[t:t + 1], BF16_TOL, f"token {t}")
    _check(pool[2:], fin, STATE_TOL, "state")


def test_one_head_over_many_ranges_equals_pieces():
    # one head, so that its chain of ranges is as long as the machine is wide: whole against
    # halves that hand their state on through memory
    Hk, Hv, K, V, n = 1, 1, 64, 64, 9000
    q, k, v, g, do, _ = (t.cuda() for t in plain.linear_inputs([n], Hk, Hv, K, V, seed=43, reach=4.0))
    g = g * 0.02
    o, fin, _ = cc.cattn_linear_fwd(q, k, v, g, _cu([n]), final_state=True)
    a = 4500
    first = [t[:a] for t in (q, k, v)] + [g[:a].contiguous()]
    rest = [t[a:] for t in (q, k, v)] + [g[a:].contiguous()]
    o1, mid, _ = cc.cattn_linear_fwd(*first, _cu([a]), final_state=True)
    o2, end, _ = cc.cattn_linear_fwd(*rest, _cu([n - a]), initial_state=mid, final_state=True)
    _check(torch.cat((o1, o2)), o.double().cpu(), 2 * BF16_TOL, "o")
    _check(end, fin.double().cpu(), 2 * STATE_TOL, "state")
    whole = cc.cattn_linear_bwd(q, k, v, g, do, _cu([n]))
    part = cc.cattn_linear_bwd(*rest, do[a:], _cu([n - a]), initial_state=mid)
    for name, x, y, tol in zip(("dq", "dk", "dv", "dg"), whole, part, (BF16_TOL,) * 3 + (DG_TOL,)):
        _check(x[a:], y.double().cpu(), 2 * tol, name)


@pytest.mark.parametrize("K", [8, 24, 40, 128])
@pytest.mark.parametrize("Hk,Hv,V", [(3, 6, 64), (2, 8, 40), (2, 2, 200), (1, 2, 136), (1, 3, 64), (1, 6, 8),
                                     (2, 10, 136)])
def test_sums_over_a_key_heads_members(Hk, Hv, V, K):
    # 2 and 4 members (value heads and their column tiles) are added up by a cluster, a share of the
    # columns each (at K = 8 one member has them all), other numbers through memory
    lens = [128, 0, 300, 1, 640, 77]
    q, k, v, g, do, s0 = plain.linear_inputs(lens, Hk, Hv, K, V, seed=K + Hv)
    leaves = [t.double().requires_grad_() for t in (q, k, v, g, s0)]
    o, _ = plain.linear(*leaves[:4], cu_of(lens), K ** -0.5, leaves[4])
    want = torch.autograd.grad(o, leaves, do.double())
    args = [t.cuda() for t in (q, k, v, g, do)]
    grads = cc.cattn_linear_bwd(*args, _cu(lens), initial_state=s0.cuda())
    for name, a, b, tol in zip(("dq", "dk", "dv", "dg", "d_initial_state"), grads, want,
                               (BF16_TOL, BF16_TOL, BF16_TOL, DG_TOL, STATE_TOL)):
        _check(a, b, tol, name)


def test_backwards_side_by_side():
    # the CTAs of a cluster wait for one another: they must be there whatever else runs
    cases = []
    for seed, (Hk, Hv, V) in enumerate([(4, 8, 128), (2, 8, 128), (4, 4, 256), (1, 1, 64)]):
        lens = [700 + 100 * seed, 33, 1200]
        cases.append((_cu(lens), [t.cuda() for t in plain.linear_inputs(lens, Hk, Hv, 64, V, seed=seed)[:5]]))
    want = [cc.cattn_linear_bwd(*args, cu) for cu, args in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [[] for _ in cases]
    for _ in range(20):
        for i, (cu, args) in enumerate(cases):
            with torch.cuda.stream(streams[i]):
                got[i].append(cc.cattn_linear_bwd(*args, cu))
    torch.cuda.synchronize()
    for runs, ref in zip(got, want):
        for grads in runs:
            assert all(torch.equal(a, b) for a, b in zip(grads[:4], ref[:4]))


@pytest.mark.parametrize("lens,Hk,Hv,K,V", [
    ([6, 1, 2], 3, 3, 32, 64), ([40] * 5, 2, 2, 128, 256), ([200, 130], 2, 8, 128, 128), ([1] * 9, 1, 2, 64, 40),
])
def test_dg_where_initial_states_outweigh_the_tokens(lens, Hk, Hv, K, V):
    # with states of size 8 nearly all of dg is q (S do): S must be read with all its 24 bits.  In the 2-norm,
    # where 16 bits would show as 2^-17 / 3 (2.5e-6) of each pair: 1e-6, the products' 2^-24 (6e-8), the matrix
    # sums cut off at each of up to 24 steps of 16 terms (24 * 2^-24 / 2 = 7e-7) and the fp32 sums over K and
    # the tokens, rounded and so of the order of 2^-24 times the root of their number (1e-7)
    q, k, v, g, do, s0 = plain.linear_inputs(lens, Hk, Hv, K, V, seed=K + V)
    s0 = 8 * s0
    leaves = [t.double().requires_grad_() for t in (q, k, v, g, s0)]
    o, _ = plain.linear(*leaves[:4], cu_of(lens), K ** -0.5, leaves[4])
    want = torch.autograd.grad(o, leaves[3], do.double())[0]
    dg = cc.cattn_linear_bwd(*(t.cuda() for t in (q, k, v, g, do)), _cu(lens), initial_state=s0.cuda())[3]
    err = float((dg.double().cpu() - want).norm() / want.norm())
    assert err <= 1e-6, err


@pytest.mark.parametrize("lens,Hk,Hv,K,V", [([1], 1, 2, 128, 256), ([3, 0, 2], 2, 4, 32, 96), ([40], 1, 3, 64, 64),
                                           ([63, 1], 2, 2, 96, 128)])
def test_few_tokens_are_rounded_at_the_store_only(lens, Hk, Hv, K, V):
    # up to 64 rows keep their scores in two bf16 terms (2^-17): what is left is the store, which rounds by
    # up to 2^-8 of a value
    q, k, v, g, do, _ = plain.linear_inputs(lens, Hk, Hv, K, V, seed=V)
    leaves = [t.double().requires_grad_() for t in (q, k, v, g)]
    o, _ = plain.linear(*leaves, cu_of(lens), K ** -0.5, None)
    want = torch.autograd.grad(o, leaves[:3], do.double(), allow_unused=True)
    args = [t.cuda() for t in (q, k, v, g)]
    got = [cc.cattn_linear_fwd(*args, _cu(lens))[0], *cc.cattn_linear_bwd(*args, do.cuda(), _cu(lens))[:3]]
    for name, a, b in zip(("o", "dq", "dk", "dv"), got, (o.detach(), *want)):
        _check(a, b, 1.05 * 2.0 ** -8, name)
