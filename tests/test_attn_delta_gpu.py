"""cattn_delta_fwd / _bwd / _update against the definition in 64 bits (GPU).

Tolerances, as max |error| / max |reference|:
  o              4e-3: the store's rounding (2^-8 of an element); the products keep 24 bits of every
                 factor, and of P~ and the state too
  fp32 states    5e-6: products split so that 2^-24 of each is kept, fp32 sums of up to 64 + 128
                 values; errors of earlier chunks decay with the state
  dv             4e-3: the store's rounding of a sum that keeps 24 bits
  dq, dk         8e-3: the store rounds by up to 2^-8 (3.9e-3); the matrix operands that are not
                 inputs (decayed pairs, the states) are rounded too, with independent errors: as for
                 the linear attention's gradients
  dg, dbeta      2e-5: fp32 sums of products that keep 24 bits, over up to 128 + 256 channels and
                 64 tokens; dg is summed up over the tokens behind it, where parts of both signs
                 cancel down to a tenth
"""
import pytest
import torch

import depthwise_causal_short_gb300 as cc
from depthwise_causal_short_gb300 import _build
from tests import delta_plain as plain
from tests.helpers import rel_err

pytestmark = pytest.mark.gpu
O_TOL = 4e-3
STATE_TOL = 5e-6
GRAD_TOL = 8e-3
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
    ([1], 1, 1, 8, 8), ([0], 2, 2, 16, 24), ([0, 1, 0], 1, 2, 64, 64), ([63], 1, 1, 128, 128),
    ([64], 2, 2, 128, 128), ([65], 1, 2, 128, 64), ([127, 128, 129], 1, 1, 72, 40),
    ([63, 64, 65, 0, 1, 200, 31], 2, 4, 128, 128), ([257, 300], 1, 3, 96, 40), ([5, 500], 1, 1, 40, 136),
    ([384], 1, 8, 32, 128), ([130, 2, 126], 3, 3, 72, 256), ([700], 1, 1, 64, 96), ([1] * 40, 2, 2, 64, 32),
    ([1, 255, 256, 1], 1, 2, 120, 200), ([1] * 200, 1, 4, 32, 32), ([90, 2, 300] * 5, 4, 16, 24, 136),
    ([2200], 1, 2, 64, 64), ([1100, 3], 8, 16, 32, 200),
]


def _check(a, b, tol, what):
    e = rel_err(a.detach().double().cpu(), b)
    assert e <= tol, f"{what}: {e:.3g} > {tol:.3g}"


@pytest.mark.parametrize("lens,Hk,Hv,K,V", CASES)
@pytest.mark.parametrize("states", [False, True])
def test_parity(lens, Hk, Hv, K, V, states):
    q, k, v, g, beta, do, s0 = plain.delta_inputs(lens, Hk, Hv, K, V, seed=sum(lens) + K)
    leaves = [t.double().requires_grad_() for t in (q, k, v, g, beta, s0)]
    o, fin = plain.delta(*leaves[:5], cu_of(lens), K ** -0.5, leaves[5] if states else None)
    args = [t.cuda() for t in (q, k, v, g, beta)]
    cu = _cu(lens)
    init = s0.cuda() if states else None
    go, gfin, status = cc.cattn_delta_fwd(*args, cu, initial_state=init, final_state=True)
    assert status is None
    _check(gfin, fin.detach(), STATE_TOL, "final state")
    if sum(lens):
        _check(go, o.detach(), O_TOL, "o")
    # without a final state the factors have 16 bits each, not 24: a result that is stored with 9 bits (half a
    # step: 2^-9 of a value at least, 2^-8 at most) moves by no more than 2^-17 a factor, so O_TOL holds for it too
    alone, none, _ = cc.cattn_delta_fwd(*args, cu, initial_state=init)
    assert none is None and torch.equal(alone, cc.cattn_delta_fwd(*args, cu, initial_state=init)[0])
    if sum(lens):
        _check(alone, o.detach(), O_TOL, "o alone")

    grads = cc.cattn_delta_bwd(*args, do.cuda(), cu, initial_state=init)
    again = cc.cattn_delta_bwd(*args, do.cuda(), cu, initial_state=init)
    for a, b in zip(grads, again):
        assert (a is None and b is None) or torch.equal(a, b)  # a fixed order
    if not sum(lens):
        assert not states or not grads[5].any()
        return
    want = torch.autograd.grad(o, leaves if states else leaves[:5], do.double(), allow_unused=True)
    for name, tol, a, b in zip(("dq", "dk", "dv", "dg", "dbeta"), (GRAD_TOL, GRAD_TOL, O_TOL, DG_TOL, DG_TOL), grads, want):
        _check(a, b, tol, name)
    if states:
        _check(grads[5], want[5], STATE_TOL, "d_initial_state")


@pytest.mark.parametrize("kind", ["beta_zero", "beta_two", "forget", "keep", "same_keys", "no_decay"])
def test_ends_of_the_ranges(kind):
    # step sizes of 0 (nothing is learnt) and near 2 (the reflection), decays of 0 and 1, keys that are
    # all the same (the triangular system at its worst)
    lens, Hk, Hv, K, V = [150, 64, 3], 2, 4, 64, 64
    q, k, v, g, beta, do, s0 = plain.delta_inputs(lens, Hk, Hv, K, V, seed=11)
    if kind == "beta_zero":
        beta[:, ::2] = 0.0
        beta[::3] = 0.0
    elif kind == "beta_two":
        beta = 1.9 + 0.08 * torch.rand(beta.shape)
    elif kind == "forget":
        g[::5] = float("-inf")
        g[1::7] = -300.0
    elif kind == "keep":
        g = g * 1e-4
    elif kind == "no_decay":
        g = torch.zeros_like(g)
    else:
        k = k[:1].expand_as(k).contiguous()
    ref_g = g.clamp(min=-128.0).double()
    o, fin = plain.delta(q.double(), k.double(), v.double(), ref_g, beta.double(), cu_of(lens), K ** -0.5, s0.double())
    args = [t.cuda() for t in (q, k, v, g, beta)]
    go, gfin, _ = cc.cattn_delta_fwd(*args, _cu(lens), initial_state=s0.cuda(), final_state=True)
    _check(go, o, O_TOL, "o")
    alone = cc.cattn_delta_fwd(*args, _cu(lens), initial_state=s0.cuda())[0]
    _check(alone, o, O_TOL, "o alone")
    _check(gfin, fin, STATE_TOL, "final state")


def test_linear_attention_is_what_is_left_without_the_old_value():
    # one token after another with beta = 1 and orthogonal keys: nothing is there to be replaced
    K = V = 64
    k = torch.eye(K).bfloat16()[:, None, :].contiguous()
    q, v = torch.randn(K, 1, K).bfloat16(), torch.randn(K, 1, V).bfloat16()
    g, beta = torch.zeros(K, 1), torch.ones(K, 1)
    args = [t.cuda() for t in (q, k, v, g)]
    cu = _cu([K])
    a = cc.cattn_delta_fwd(*args, beta.cuda(), cu, final_state=True)
    b = cc.cattn_linear_fwd(*args, cu, final_state=True)
    assert torch.equal(a[1], b[1])
    _check(a[0], b[0].double().cpu(), 2 * O_TOL, "o")


def test_strided_inputs_and_expanded_gates():
    lens, Hk, Hv, K, V = [70, 31], 2, 4, 64, 40
    total = sum(lens)
    q, k, v, g, beta, do, s0 = plain.delta_inputs(lens, Hk, Hv, K, V, seed=3)
    wide = torch.randn(total, 1024).bfloat16().cuda()
    qs, ks, vs = wide[:, :Hk * K].view(total, Hk, K), wide[:, 256:256 + Hk * K].view(total, Hk, K), \
        wide[:, 512:512 + Hv * V].view(total, Hv, V)
    for dst, src in ((qs, q), (ks, k), (vs, v)):
        dst.copy_(src)
    gs = torch.randn(Hv).neg().abs().neg().cuda().expand(total, Hv)          # one decay a head
    bs = torch.rand(Hv, total).cuda().t()                                     # heads apart
    want = cc.cattn_delta_fwd(q.cuda(), k.cuda(), v.cuda(), gs.contiguous(), bs.contiguous(), _cu(lens), final_state=True)
    got = cc.cattn_delta_fwd(qs, ks, vs, gs, bs, _cu(lens), final_state=True)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_state_slots_in_place_and_bad_ones():
    lens, Hk, Hv, K, V = [40, 100, 7], 1, 2, 32, 64
    q, k, v, g, beta, do, _ = plain.delta_inputs(lens, Hk, Hv, K, V, seed=9)
    pool = torch.randn(6, Hv, K, V)
    idx = [4, 0, 5]
    o, fin = plain.delta(*[t.double() for t in (q, k, v, g, beta)], cu_of(lens), K ** -0.5, pool[idx].double())
    args = [t.cuda() for t in (q, k, v, g, beta)]
    p = pool.cuda()
    go, gp, status = cc.cattn_delta_fwd(*args, _cu(lens), initial_state=p, final_state=p,
                                        state_indices=torch.tensor(idx, dtype=torch.int32).cuda())
    assert status.tolist() == [0, 0] and gp.data_ptr() == p.data_ptr()
    _check(go, o, O_TOL, "o")
    _check(p[idx], fin, STATE_TOL, "states")
    others = [i for i in range(6) if i not in idx]
    assert torch.equal(p[others].cpu(), pool[others])
    for bad, bits in (([4, 4, 1], cc.IDX_DUPLICATE), ([4, -1, 1], cc.IDX_NEGATIVE), ([4, 6, 1], cc.IDX_OUT_OF_RANGE)):
        p = pool.cuda()
        slots = torch.tensor(bad, dtype=torch.int32)
        go, _, status = cc.cattn_delta_fwd(*args, _cu(lens), initial_state=p, final_state=p, state_indices=slots.cuda())
        assert status.tolist() == [-8, bits] or (status[0].item() < 0 and status[1].item() == bits)
        assert torch.equal(p.cpu(), pool)
        first = torch.stack([pool[s] if 0 <= s < 6 else torch.zeros(Hv, K, V) for s in bad])
        o, _ = plain.delta(*[t.double() for t in (q, k, v, g, beta)], cu_of(lens), K ** -0.5, first.double())
        _check(go, o, O_TOL, "o")


def test_many_sequences_with_slots():
    lens = [3, 0, 65, 1] * 12  # more sequences than a kernel checks by itself
    Hk, Hv, K, V = 1, 2, 32, 40
    q, k, v, g, beta, do, _ = plain.delta_inputs(lens, Hk, Hv, K, V, seed=10)
    pool = torch.randn(60, Hv, K, V)
    idx = torch.randperm(60)[:len(lens)]
    o, fin = plain.delta(*[t.double() for t in (q, k, v, g, beta)], cu_of(lens), K ** -0.5, pool[idx].double())
    args = [t.cuda() for t in (q, k, v, g, beta)]
    p = pool.cuda()
    go, _, status = cc.cattn_delta_fwd(*args, _cu(lens), initial_state=p, final_state=p, state_indices=idx.int().cuda())
    assert status.tolist() == [0, 0]
    _check(go, o, O_TOL, "o")
    _check(p[idx.cuda()], fin, STATE_TOL, "states")
    idx[5] = idx[17]
    p = pool.cuda()
    _, _, status = cc.cattn_delta_fwd(*args, _cu(lens), initial_state=p, final_state=p, state_indices=idx.int().cuda())
    assert status[1].item() == cc.IDX_DUPLICATE and torch.equal(p.cpu(), pool)


def test_sequences_do_not_meet():
    # NaN and infinity in one sequence leave the others' results as they were
    lens, Hk, Hv, K, V = [70, 50, 130], 1, 2, 64, 64
    args = [t.cuda() for t in plain.delta_inputs(lens, Hk, Hv, K, V, seed=6)[:5]]
    cu = _cu(lens)
    clean = cc.cattn_delta_fwd(*args, cu, final_state=True)
    for i, bad in ((0, float("nan")), (1, float("inf")), (2, float("nan")), (3, float("nan")), (4, float("inf"))):
        other = [t.clone() for t in args]
        other[i][70:120] = bad
        got = cc.cattn_delta_fwd(*other, cu, final_state=True)
        assert torch.equal(got[0][:70], clean[0][:70]) and torch.equal(got[0][120:], clean[0][120:])
        assert torch.equal(got[1][[0, 2]], clean[1][[0, 2]])
        assert not torch.isfinite(got[0][120 - 1]).all()


def test_ill_formed_offsets_are_reported():
    lens, Hk, Hv, K, V = [40, 40], 1, 1, 32, 32
    args = [t.cuda() for t in plain.delta_inputs(lens, Hk, Hv, K, V)[:5]]
    for cu in ([0, 90, 80], [0, -5, 80], [3, 40, 80], [0, 40, 79], [0, 40, 400]):
        cc.cattn_delta_fwd(*args, torch.tensor(cu, dtype=torch.int32).cuda(), final_state=True)
        assert cc.cattn_device_fault() == 4, cu


def test_graph_replays():
    lens, Hk, Hv, K, V = [100, 28], 2, 4, 64, 96
    args = [t.cuda() for t in plain.delta_inputs(lens, Hk, Hv, K, V, seed=2)[:5]]
    cu = _cu(lens)
    want = cc.cattn_delta_fwd(*args, cu, final_state=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = cc.cattn_delta_fwd(*args, cu, final_state=True, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = cc.cattn_delta_fwd(*args, cu, final_state=True)
    held[0].zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(held[0], want[0]) and torch.equal(held[1], want[1])


@pytest.mark.parametrize("N,Hk,Hv,K,V", [(1, 1, 1, 8, 8), (3, 2, 4, 40, 56), (33, 1, 3, 128, 128), (5, 2, 2, 96, 256),
                                         (70, 1, 2, 64, 32), (2, 4, 4, 128, 24)])
def test_update(N, Hk, Hv, K, V):
    q, k, v, g, beta, do, _ = plain.delta_inputs([1] * N, Hk, Hv, K, V, seed=N)
    pool = torch.randn(N + 5, Hv, K, V)
    idx = torch.randperm(N + 5)[:N]
    o, fin = plain.delta(*[t.double() for t in (q, k, v, g, beta)], list(range(N + 1)), K ** -0.5, pool[idx].double())
    args = [t.cuda() for t in (q, k, v, g, beta)]
    p = pool.cuda()
    go, status = cc.cattn_delta_update(*args, p, idx.int().cuda())
    assert status.tolist() == [0, 0]
    _check(go, o, O_TOL, "o")
    _check(p[idx.cuda()], fin, STATE_TOL, "state")
    rest = torch.ones(N + 5, dtype=torch.bool)
    rest[idx] = False
    assert torch.equal(p.cpu()[rest], pool[rest])
    # row i uses slot i
    p = pool.cuda()
    go, _ = cc.cattn_delta_update(*args, p)
    o, fin = plain.delta(*[t.double() for t in (q, k, v, g, beta)], list(range(N + 1)), K ** -0.5, pool[:N].double())
    _check(go, o, O_TOL, "o")
    _check(p[:N], fin, STATE_TOL, "state")


@pytest.mark.parametrize("N", [5, 40])
def test_update_padding_and_bad_indices(N):
    Hk, Hv, K, V = 1, 2, 32, 64
    q, k, v, g, beta, do, _ = plain.delta_inputs([1] * N, Hk, Hv, K, V, seed=N)
    pool = torch.randn(N + 3, Hv, K, V)
    args = [t.cuda() for t in (q, k, v, g, beta)]
    idx = torch.randperm(N + 3)[:N].int()
    idx[N - 2:] = -1
    o0 = torch.full((N, Hv, V), 7.0).bfloat16().cuda()
    p = pool.cuda()
    go, status = cc.cattn_delta_update(*args, p, idx.cuda(), pad_rows=True, o=o0)
    assert status.tolist() == [0, 0] and (go[N - 2:] == 7.0).all()
    n = N - 2
    o, fin = plain.delta(*[t[:n].double() for t in (q, k, v, g, beta)], list(range(n + 1)), K ** -0.5,
                         pool[idx[:n].long()].double())
    _check(go[:n], o, O_TOL, "o")
    _check(p[idx[:n].long().cuda()], fin, STATE_TOL, "state")
    for where, value, bits in ((1, int(idx[0]), cc.IDX_DUPLICATE), (2, N + 3, cc.IDX_OUT_OF_RANGE)):
        bad = idx.clone()
        bad[where] = value
        p = pool.cuda()
        go, status = cc.cattn_delta_update(*args, p, bad.cuda(), pad_rows=True, o=o0.fill_(7.0))
        assert status[0].item() < 0 and status[1].item() == bits
        assert torch.equal(p.cpu(), pool) and (go == 7.0).all()


def test_a_prompt_in_parts_and_tokens():
    # a prompt whole; in two parts through a pool; and its last tokens one by one
    n, Hk, Hv, K, V = 150, 2, 4, 64, 64
    args = [t.cuda() for t in plain.delta_inputs([n], Hk, Hv, K, V, seed=12)[:5]]
    whole, fin, _ = cc.cattn_delta_fwd(*args, _cu([n]), final_state=True)
    pool = torch.zeros(3, Hv, K, V).cuda()
    slot = torch.tensor([1], dtype=torch.int32).cuda()
    outs = []
    for a, b in ((0, 97), (97, 140)):
        part = [t[a:b] for t in args]
        outs.append(cc.cattn_delta_fwd(*part, _cu([b - a]), initial_state=pool, final_state=pool, state_indices=slot)[0])
    for t in range(140, n):
        outs.append(cc.cattn_delta_update(*[x[t:t + 1] for x in args], pool, slot)[0])
    got = torch.cat(outs)
    _check(got, whole.double().cpu(), 2 * O_TOL, "o")
    _check(pool[1], fin[0].double().cpu(), 2 * STATE_TOL, "state")
