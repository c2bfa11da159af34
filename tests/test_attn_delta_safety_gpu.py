"""The delta rule's and layer norm's kernels where their parts meet each other, earlier kernels, other streams
and graphs, and their errors in the 2-norm (GPU).

Tolerances in the 2-norm:
  bf16 results   a stored value is off by at most half a unit of its 8 bits, evenly spread: 2^-7 / sqrt(12) =
                 2.26e-3 of its power of two in the root mean square, and no more of itself.  dq and dk are
                 sums of terms with operands rounded like that (the states, dv), each independently: as
                 much again, sqrt(2) * 2.26e-3 = 3.2e-3.  o and dv have no such operands: 2.4e-3
  states         1e-6: products of 24 bits, sums in fp32 of 64 + 128 values (2^-24 sqrt(192) = 8e-7)
  dbeta          2e-6: a product of two such vectors over V channels
  dg             4e-6: sums over the tokens behind, of terms of both signs with errors like dbeta's
"""
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


def _inputs(lens, Hk, Hv, K, V, seed=0):
    return plain.delta_inputs(lens, Hk, Hv, K, V, seed=seed)


@pytest.mark.parametrize("lens,Hk,Hv,K,V", [
    ([700, 33, 300], 2, 4, 128, 128), ([900], 1, 2, 64, 96), ([100, 29, 400], 4, 12, 40, 64),
    ([513, 90], 1, 9, 32, 40), ([64] * 8, 2, 2, 80, 200),
])
@pytest.mark.parametrize("states", [False, True])
def test_errors_in_the_2_norm(lens, Hk, Hv, K, V, states):
    q, k, v, g, beta, do, s0 = _inputs(lens, Hk, Hv, K, V, seed=K + V)
    cu = [0] + torch.tensor(lens).cumsum(0).tolist()
    leaves = [t.double().requires_grad_() for t in (q, k, v, g, beta, s0)]
    o, fin = plain.delta(*leaves[:5], cu, K ** -0.5, leaves[5] if states else None)
    want = torch.autograd.grad(o, leaves if states else leaves[:5], do.double())
    args, init = [t.cuda() for t in (q, k, v, g, beta)], s0.cuda() if states else None
    got = [*cc.cattn_delta_fwd(*args, _cu(lens), initial_state=init, final_state=True)[:2],
           *cc.cattn_delta_bwd(*args, do.cuda(), _cu(lens), initial_state=init)]
    names = ("o", "final", "dq", "dk", "dv", "dg", "dbeta", "ds")
    tols = (2.4e-3, 1e-6, 3.2e-3, 3.2e-3, 2.4e-3, 4e-6, 2e-6, 1e-6)
    for name, tol, a, b in zip(names, tols, got, (o.detach(), fin.detach(), *want)):
        err = float((a.double().cpu() - b).norm() / b.norm())
        assert err <= tol, (name, err)


def test_gradients_against_differences():
    # the loss's change along random directions, from the 64-bit forward, against the kernel's gradients:
    # they carry the bf16 tolerance, of the sum of their parts' sizes
    lens, Hk, Hv, K, V = [70, 90], 1, 2, 64, 64
    inputs = _inputs(lens, Hk, Hv, K, V, seed=5)
    q, k, v, g, beta, do, s0 = inputs
    cu = [0, 70, 160]
    grads = cc.cattn_delta_bwd(*[t.cuda() for t in (q, k, v, g, beta, do)], _cu(lens), initial_state=s0.cuda())
    base = [t.double() for t in (q, k, v, g, beta, s0)]
    gen = torch.Generator().manual_seed(7)
    for i in range(6):
        d = torch.randn(base[i].shape, generator=gen, dtype=torch.float64)
        loss = []
        for sign in (1, -1):
            args = list(base)
            args[i] = base[i] + sign * 1e-4 * d
            loss.append((plain.delta(*args[:5], cu, K ** -0.5, args[5])[0] * do.double()).sum())
        slope = (loss[0] - loss[1]).item() / 2e-4
        got = (grads[i].double().cpu() * d).sum().item()
        size = (grads[i].double().cpu() * d).norm().item()
        assert abs(slope - got) <= 1e-2 * size + 1e-4 * abs(slope), (i, slope, got, size)


@pytest.mark.parametrize("lens,Hk,Hv,K,V,states", [
    ([90, 2, 300] * 5, 4, 16, 24, 136, False), ([1] * 300, 2, 4, 32, 32, False),
    ([128, 5, 0, 129] * 12, 4, 8, 64, 64, True), ([1500, 33, 800], 8, 16, 128, 128, False),
    ([64, 400, 1, 128, 0, 0] * 8, 1, 8, 72, 256, False),
])
def test_repeats_are_bit_identical(lens, Hk, Hv, K, V, states):
    q, k, v, g, beta, do, s0 = (t.cuda() for t in _inputs(lens, Hk, Hv, K, V, seed=K))
    cu, init = _cu(lens), s0 if states else None
    first = None
    for _ in range(20):
        got = [t for t in (*cc.cattn_delta_bwd(q, k, v, g, beta, do, cu, initial_state=init),
                           *cc.cattn_delta_fwd(q, k, v, g, beta, cu, initial_state=init, final_state=True)[:2])
               if t is not None]
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(got, first))
    assert all(torch.isfinite(t).all() for t in first)


@pytest.mark.parametrize("Hk,Hv", [(1, 1), (1, 3)])
@pytest.mark.parametrize("K,V", [(8, 8), (40, 40), (72, 136), (104, 200), (64, 24), (24, 256)])
def test_results_do_not_depend_on_what_ran_before(K, V, Hk, Hv):
    # calls on NaN leave NaN in shared and tensor memory of every SM, and in the memory that workspaces get
    n = 64 * 600
    g, beta = torch.zeros(n, 1).cuda(), torch.ones(n, 1).cuda()
    lens = [100, 0, 65, 1, 128]
    q, k, v, gates, betas, do, s0 = (t.cuda() for t in _inputs(lens, Hk, Hv, K, V, seed=K))

    def after(value):
        x = torch.full((n, 1, 128), value, dtype=torch.bfloat16).cuda()
        out = []
        for states in (None, s0):
            cc.cattn_delta_fwd(x, x, x, g, beta, _cu([64] * 600))
            out += cc.cattn_delta_fwd(q, k, v, gates, betas, _cu(lens), initial_state=states, final_state=True)[:2]
            cc.cattn_delta_bwd(x, x, x, g, beta, x, _cu([64] * 600))
            out += [t for t in cc.cattn_delta_bwd(q, k, v, gates, betas, do, _cu(lens), initial_state=states)
                    if t is not None]
        return out

    for a, b in zip(after(float("nan")), after(0.0)):
        assert torch.isfinite(a).all() and torch.equal(a, b)


def test_sequences_do_not_meet_in_the_gradient():
    lens, Hk, Hv, K, V = [70, 50, 130], 1, 2, 64, 64
    args = [t.cuda() for t in _inputs(lens, Hk, Hv, K, V, seed=6)]
    cu = _cu(lens)
    clean = cc.cattn_delta_bwd(*args[:6], cu, initial_state=args[6])
    for i in range(6):
        other = [t.clone() for t in args]
        other[i][70:120] = float("nan")
        got = cc.cattn_delta_bwd(*other[:6], cu, initial_state=args[6])
        for a, b in zip(got[:5], clean[:5]):
            assert torch.equal(a[:70], b[:70]) and torch.equal(a[120:], b[120:])
        assert torch.equal(got[5][[0, 2]], clean[5][[0, 2]])
        # (v has no part in the gradient of the states, which is linear in do)
        assert not torch.isfinite(got[0][70:120] if i == 2 else got[5][1]).all()


def test_the_gradient_reads_states_through_their_slots():
    lens, Hk, Hv, K, V = [40, 0, 100, 7], 1, 2, 32, 64
    q, k, v, g, beta, do, _ = (t.cuda() for t in _inputs(lens, Hk, Hv, K, V, seed=9))
    pool = torch.randn(6, Hv, K, V).cuda()
    status = torch.empty(2, dtype=torch.int32, device="cuda")
    for idx, bits in (([4, 1, 0, 5], 0), ([4, 4, 0, 5], cc.IDX_DUPLICATE), ([4, -1, 0, 7], cc.IDX_NEGATIVE | cc.IDX_OUT_OF_RANGE)):
        slots = torch.tensor(idx, dtype=torch.int32).cuda()
        got = cc.cattn_delta_bwd(q, k, v, g, beta, do, _cu(lens), initial_state=pool, state_indices=slots, status=status)
        dense = torch.stack([pool[i] if 0 <= i < 6 else torch.zeros_like(pool[0]) for i in idx])
        want = cc.cattn_delta_bwd(q, k, v, g, beta, do, _cu(lens), initial_state=dense)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert status[1].item() == bits and not got[5][1].any()


@pytest.mark.parametrize("raw", [False, True])
def test_a_given_streams_calls_keep_their_memory_until_it_has_used_it(raw):
    # the calls wait on a busy stream while the current one takes and fills all the memory it is given
    lens, Hk, Hv, K, V = [700, 300], 2, 4, 64, 64
    q, k, v, g, beta, do, s0 = (t.cuda() for t in _inputs(lens, Hk, Hv, K, V, seed=3))
    cu, w = _cu(lens), torch.rand(V).cuda()
    pool = torch.randn(2, Hv, K, V).cuda()

    def calls(**kw):
        state = pool.clone()
        torch.cuda.synchronize()
        if kw:
            with torch.cuda.stream(side):
                torch.cuda._sleep(200_000_000)  # some 0.1 s
        return (*cc.cattn_delta_fwd(q, k, v, g, beta, cu, initial_state=s0, final_state=True, **kw)[:2],
                *cc.cattn_delta_bwd(q, k, v, g, beta, do, cu, initial_state=s0, **kw),
                *cc.cattn_delta_update(q[:2], k[:2], v[:2], g[:2], beta[:2], state, **kw), state,
                cc.cattn_layernorm_fwd(v, w, w, gate=do, **kw),
                *cc.cattn_layernorm_bwd(v, do, w, w, gate=do, **kw))

    sizes = [16, 512, 2048, 1 << 20, 2 << 20, 8 << 20, 20 << 20, 64 << 20] * 6
    sizes += [cc.cattn_delta_fwd_workspace_bytes(1000, 2, Hk, Hv, K, V),
              cc.cattn_delta_bwd_workspace_bytes(1000, 2, Hk, Hv, K, V),
              cc.cattn_layernorm_bwd_workspace_bytes(1000, Hv, V)] * 4
    want = calls()
    side = torch.cuda.Stream()
    stream = side.cuda_stream if raw else side
    for first in (True, False):  # the first time, memory comes from the device, which waits for the streams
        got = calls(stream=stream)
        fill = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in sizes]
        if first:
            torch.cuda.synchronize()
            del got, fill
    torch.cuda.current_stream().synchronize()
    assert not side.query()  # the calls are still to run
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(bool((t == 255).all()) for t in fill)


def test_two_calls_at_once():
    # on two streams, with workspaces of their own
    lens, Hk, Hv, K, V = [300, 200], 2, 4, 64, 64
    one = [t.cuda() for t in _inputs(lens, Hk, Hv, K, V, seed=1)]
    two = [t.cuda() for t in _inputs(lens, Hk, Hv, K, V, seed=2)]
    cu = _cu(lens)
    want = [cc.cattn_delta_bwd(*x[:6], cu, initial_state=x[6]) for x in (one, two)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [cc.cattn_delta_bwd(*x[:6], cu, initial_state=x[6], stream=s) for x, s in zip((one, two), streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_a_training_step_in_a_graph():
    lens, Hk, Hv, K, V = [100, 28], 2, 4, 64, 96
    base = [t.cuda() for t in _inputs(lens, Hk, Hv, K, V, seed=2)]
    cu, w = _cu(lens), torch.rand(V).cuda()

    def step(q, k, v, g, beta, s0, w):
        o, _ = cc.delta_attention(q, k, v, g, beta, cu, s0)
        return cc.layer_norm(o, w, gate=v, mode="rms")

    def run():
        leaves = [t.detach().clone().requires_grad_() for t in (*base[:5], base[6], w)]
        y = step(*leaves)
        return [y, *torch.autograd.grad(y, leaves, base[5])]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = run()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(held, want))


def test_autograd_asks_for_what_is_needed_and_refuses_second_derivatives():
    lens = [20, 7]
    q, k, v, g, beta, do, s0 = (t.cuda() for t in _inputs(lens, 1, 2, 32, 32))
    w = torch.ones(32).cuda()
    v.requires_grad_()
    beta.requires_grad_()
    o, fin = cc.delta_attention(q, k, v, g, beta, _cu(lens), s0, output_final_state=True)
    assert not fin.requires_grad and o.requires_grad
    dv, dbeta = torch.autograd.grad(o, (v, beta), do, retain_graph=True)
    want = cc.cattn_delta_bwd(q, k, v.detach(), g, beta.detach(), do, _cu(lens), initial_state=s0)
    assert torch.equal(dv, want[2]) and torch.equal(dbeta, want[4])
    w.requires_grad_()
    y = cc.layer_norm(v, w, gate=o.detach())
    dw, dx = torch.autograd.grad(y, (w, v), do, retain_graph=True)
    full = cc.cattn_layernorm_bwd(v.detach(), do, w.detach(), gate=o.detach())
    assert torch.equal(dw, full[1]) and torch.equal(dx, full[0])
    for out, leaf in ((o, v), (y, w)):
        grad, = torch.autograd.grad(out.float().sum(), leaf, create_graph=True)
        with pytest.raises(RuntimeError, match="no gradients of their own"):
            grad.float().square().sum().backward()


def test_rows_behind_the_last_sequence_of_a_pool_stay():
    # a state array of more slots than sequences: the others are left as they were
    lens, Hk, Hv, K, V = [5, 70], 1, 1, 16, 24
    args = [t.cuda() for t in _inputs(lens, Hk, Hv, K, V, seed=4)[:5]]
    fin = torch.full((4, Hv, K, V), 7.0).cuda()
    cc.cattn_delta_fwd(*args, _cu(lens), final_state=fin)
    assert (fin[2:] == 7.0).all() and torch.isfinite(fin).all() and not (fin[:2] == 7.0).any()


def test_a_nan_gate_or_step_reaches_what_comes_after_it():
    n, at = 300, 130
    q, k, v, g, beta, do, s0 = (t.cuda() for t in _inputs([n], 1, 2, 64, 64, seed=n))
    clean = cc.cattn_delta_fwd(q, k, v, g, beta, _cu([n]), initial_state=s0, final_state=True)[0]
    for i in (3, 4):
        args = [t.clone() for t in (q, k, v, g, beta)]
        args[i][at, 1] = float("nan")
        o, fin, _ = cc.cattn_delta_fwd(*args, _cu([n]), initial_state=s0, final_state=True)
        assert o[at:, 1].isnan().all() and fin[0, 1].isnan().all()
        # (tokens of the same chunk before it may see it too)
        assert torch.equal(o[:at - 63], clean[:at - 63]) and torch.equal(o[:, 0], clean[:, 0])


def test_a_cache_behind_2_to_the_31_elements():
    # offsets into the inputs and the pool that 32 bits do not hold
    free, _ = torch.cuda.mem_get_info()
    if free < 40 << 30:
        pytest.skip("not enough memory")
    Hv, K, V = 16, 128, 128
    slots = (1 << 31) // (Hv * K * V) + 8
    pool = torch.zeros(slots, Hv, K, V, device="cuda")
    q, k, v, g, beta, do, s0 = (t.cuda() for t in _inputs([70, 3], 8, Hv, K, V, seed=8))
    idx = torch.tensor([slots - 1, slots - 5], dtype=torch.int32).cuda()
    pool[idx.long()] = s0
    want = cc.cattn_delta_fwd(q, k, v, g, beta, _cu([70, 3]), initial_state=s0, final_state=True)
    o, _, status = cc.cattn_delta_fwd(q, k, v, g, beta, _cu([70, 3]), initial_state=pool, final_state=pool, state_indices=idx)
    assert status.tolist() == [0, 0] and torch.equal(o, want[0]) and torch.equal(pool[idx.long()], want[1])
    one = [t[:2].contiguous() for t in (q, k, v, g, beta)]
    a, b = want[1].clone(), pool
    want_o, _ = cc.cattn_delta_update(*one, a)
    got_o, _ = cc.cattn_delta_update(*one, b, idx)
    assert torch.equal(got_o, want_o) and torch.equal(b[idx.long()], a)
    # rows far apart
    wide = torch.empty(73, 1 << 25, dtype=torch.bfloat16, device="cuda")[:, -Hv * V:].view(73, Hv, V)
    wide.copy_(v)
    assert wide.stride(0) * 72 > 1 << 31
    o, _, _ = cc.cattn_delta_fwd(q, k, wide, g, beta, _cu([70, 3]), initial_state=s0, final_state=True)
    assert torch.equal(o, want[0])
    assert torch.equal(cc.cattn_layernorm_fwd(wide), cc.cattn_layernorm_fwd(v))
