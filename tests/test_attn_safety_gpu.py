"""The mixer's kernels where their parts meet each other, earlier kernels and other streams (GPU).

Tolerances are those of test_attn_linear_gpu.py, where they are derived.
"""
import pytest
import torch

import depthwise_causal_short_gb300 as cc
from depthwise_causal_short_gb300 import _build
from tests import attn_plain as plain
from tests.helpers import rel_err

pytestmark = pytest.mark.gpu
BF16_TOL = 8e-3
DG_TOL = 2e-5


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
    return plain.linear_inputs(lens, Hk, Hv, K, V, seed=seed)


@pytest.mark.parametrize("lens,Hk,Hv,K,V", [
    ([128] * 40, 16, 16, 64, 64), ([128] * 24, 4, 12, 128, 128), ([256, 128] * 10, 1, 9, 32, 128),
])
def test_whole_chunks_without_a_state_share_the_staging_buffer(lens, Hk, Hv, K, V):
    # Members of a key head that are no cluster (1, 3 and 9 of them) finish their chunks in the staging
    # buffer; whole chunks that need no state follow one another there with nothing else to wait for.
    q, k, v, g, do, _ = _inputs(lens, Hk, Hv, K, V, seed=V)
    leaves = [t.double().requires_grad_() for t in (q, k, v, g)]
    cu = [0] + torch.tensor(lens).cumsum(0).tolist()
    want = torch.autograd.grad(plain.linear(*leaves, cu, K ** -0.5)[0], leaves, do.double())
    args = [t.cuda() for t in (q, k, v, g, do)]
    first = cc.cattn_linear_bwd(*args, _cu(lens))[:4]
    for name, a, b, tol in zip(("dq", "dk", "dv", "dg"), first, want, (BF16_TOL,) * 3 + (DG_TOL,)):
        assert rel_err(a.double().cpu(), b) <= tol, name
    for _ in range(20):
        assert all(torch.equal(a, b) for a, b in zip(cc.cattn_linear_bwd(*args, _cu(lens))[:4], first))


@pytest.mark.parametrize("Hk,Hv", [(2, 2), (1, 2)])
@pytest.mark.parametrize("K", [8, 16, 40, 48, 72, 80, 104, 112])
def test_dg_does_not_see_what_tensor_memory_held(K, Hk, Hv):
    # Products over K channels write a multiple of 16 columns; the rows' dots must not read on to the next
    # multiple of 32.  A forward on NaN leaves NaN there.
    n = 128 * 300
    bad = torch.full((n, 1, 128), float("nan"), dtype=torch.bfloat16).cuda()
    bad_g = torch.zeros(n, 1).cuda()
    lens = [300, 129, 1]
    q, k, v, g, do, s0 = (t.cuda() for t in _inputs(lens, Hk, Hv, K, 64, seed=K))
    cc.cattn_linear_fwd(*(torch.zeros_like(bad),) * 3, bad_g, _cu([n]))
    want = cc.cattn_linear_bwd(q, k, v, g, do, _cu(lens), initial_state=s0)
    cc.cattn_linear_fwd(bad, bad, bad, bad_g, _cu([n]))
    got = cc.cattn_linear_bwd(q, k, v, g, do, _cu(lens), initial_state=s0)
    for a, b in zip(got, want):
        assert torch.isfinite(a).all() and torch.equal(a, b)


@pytest.mark.parametrize("Hv,n", [(1, 5000), (2, 4000), (8, 3000)])
def test_a_nan_gate_reaches_all_that_comes_after_it(Hv, n):
    # few heads and long sequences: the states that ranges hand on are joined by a kernel of their own
    Hk, K, V, at = 1, 64, 64, n // 2 - 77
    q, k, v, g, do, s0 = (t.cuda() for t in _inputs([n], Hk, Hv, K, V, seed=n))
    g = g * 1e-3  # nothing is forgotten
    clean = cc.cattn_linear_fwd(q, k, v, g, _cu([n]), initial_state=s0)[0]
    g[at, Hv - 1] = float("nan")
    o, fin, _ = cc.cattn_linear_fwd(q, k, v, g, _cu([n]), initial_state=s0, final_state=True)
    assert o[at:, Hv - 1].isnan().all() and fin[0, Hv - 1].isnan().all()
    # (tokens of the same chunk before it may see it too)
    assert torch.equal(o[:at - 127], clean[:at - 127]) and torch.equal(o[:, :Hv - 1], clean[:, :Hv - 1])
    dq, dk, dv, dg, ds = cc.cattn_linear_bwd(q, k, v, g, do, _cu([n]), initial_state=s0)
    assert dq[at:].isnan().all() and dk[:at].isnan().all() and dv[:at, Hv - 1].isnan().all()
    assert dg[:, Hv - 1].isnan().all() and ds[0, Hv - 1].isnan().all()
    for t in (dv[:, :Hv - 1], dg[:, :Hv - 1], ds[0, :Hv - 1]):
        assert torch.isfinite(t).all()


@pytest.mark.parametrize("raw", [False, True])
def test_a_given_streams_calls_keep_their_memory_until_it_has_used_it(raw):
    # the calls wait on a busy stream while the current one takes and fills all the memory it is given
    lens, Hk, Hv, K, V = [700, 300], 2, 4, 64, 64
    q, k, v, g, do, s0 = (t.cuda() for t in _inputs(lens, Hk, Hv, K, V, seed=3))
    cu, w = _cu(lens), torch.rand(K).cuda()
    pool = torch.randn(2, Hv, K, V).cuda()

    def calls(**kw):
        state = pool.clone()
        torch.cuda.synchronize()
        if kw:
            with torch.cuda.stream(side):
                torch.cuda._sleep(200_000_000)  # some 0.1 s
        return (*cc.cattn_linear_fwd(q, k, v, g, cu, initial_state=s0, final_state=True, **kw)[:2],
                *cc.cattn_linear_bwd(q, k, v, g, do, cu, initial_state=s0, **kw),
                *cc.cattn_qknorm_fwd(q, k, wq=w, wk=w, **kw),
                *cc.cattn_qknorm_bwd(q, k, k, q, wq=w, wk=w, **kw),
                *cc.cattn_linear_update(q[:2], k[:2], v[:2], g[:2], state, **kw), state)

    sizes = [16, 512, 2048, 1 << 20, 2 << 20, 8 << 20, 20 << 20, 64 << 20] * 6
    sizes += [cc.cattn_linear_fwd_workspace_bytes(1000, 2, Hk, Hv, K, V),
              cc.cattn_linear_bwd_workspace_bytes(1000, 2, Hk, Hv, K, V),
              cc.cattn_qknorm_bwd_workspace_bytes(1000, Hk, Hk, K)] * 4

    def take():  # blocks of every size that a call has just freed, and many more
        return [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in sizes]

    want = calls()
    side = torch.cuda.Stream()
    stream = side.cuda_stream if raw else side
    for first in (True, False):  # the first time, memory comes from the device, which waits for the streams
        got = calls(stream=stream)
        fill = take()
        if first:
            torch.cuda.synchronize()
            del got, fill
    torch.cuda.current_stream().synchronize()
    assert not side.query()  # the calls are still to run
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert all(bool((t == 255).all()) for t in fill)


def test_what_a_given_streams_call_returns_is_free_for_the_caller_to_use():
    # a result that is dropped while the caller's stream still reads it is not given to the next call
    q = torch.randn(4096, 8, 128).bfloat16().cuda()
    side, here = torch.cuda.Stream(), torch.cuda.current_stream()
    first = cc.cattn_qknorm_fwd(q, q)[0]
    torch.cuda.synchronize()
    y, _ = cc.cattn_qknorm_fwd(q, q, stream=side)
    here.wait_stream(side)
    torch.cuda._sleep(200_000_000)
    copy = y.clone()  # after the sleep
    del y, _
    for _ in range(4):
        cc.cattn_qknorm_fwd(-q, -q, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(copy, first)


def test_a_new_final_state_with_slots_of_a_larger_pool_is_refused():
    lens, Hk, Hv, K, V = [5, 3], 1, 1, 16, 16
    q, k, v, g, _, _ = (t.cuda() for t in _inputs(lens, Hk, Hv, K, V))
    pool = torch.randn(9, Hv, K, V).cuda()
    idx = torch.tensor([7, 1], dtype=torch.int32).cuda()
    with pytest.raises(ValueError, match="final_state"):
        cc.cattn_linear_fwd(q, k, v, g, _cu(lens), initial_state=pool, final_state=True, state_indices=idx)
    # as many slots as sequences: any order of them
    pool, idx = pool[:2].contiguous(), torch.tensor([1, 0], dtype=torch.int32).cuda()
    want = cc.cattn_linear_fwd(q, k, v, g, _cu(lens), initial_state=pool[[1, 0]].contiguous(), final_state=True)
    o, fin, status = cc.cattn_linear_fwd(q, k, v, g, _cu(lens), initial_state=pool, final_state=True,
                                         state_indices=idx)
    assert status.tolist() == [0, 0]
    assert torch.equal(o, want[0]) and torch.equal(fin[[1, 0]], want[1])


@pytest.mark.parametrize("constant", [False, True])
def test_second_derivatives_are_refused(constant):
    # the gradients' kernels have no gradient of their own: an error, not a penalty of zero (with a
    # constant gradient of the outputs too: dq still depends on k)
    q, k, v, g, do, s0 = (t.cuda().requires_grad_() for t in _inputs([20, 7], 1, 2, 32, 32))
    w = torch.ones(32).cuda().requires_grad_()
    x, cw = torch.randn(1, 30, 64).bfloat16().cuda().requires_grad_(), torch.rand(64, 4).cuda().requires_grad_()
    for o, leaves in ((cc.decay_attention(q, k, v, g, _cu([20, 7]), s0)[0], (q, k, v, g, s0)),
                      (cc.qk_norm_rope(q, k, w, w)[0], (q, w)),
                      (cc.causal_conv1d(x, cw)[0], (x, cw)),
                      (cc.causal_conv1d(x, cw, cu_seqlens=_cu([12, 18]))[0], (x, cw))):
        loss = o.float().sum() if constant else o.float().square().sum()
        grads = torch.autograd.grad(loss, leaves, create_graph=True)
        plain_grads = torch.autograd.grad(loss, leaves, retain_graph=True)
        for a, b in zip(grads, plain_grads):
            assert torch.equal(a, b) and not b.requires_grad
            with pytest.raises(RuntimeError, match="no gradients of their own"):
                (loss + a.float().square().sum()).backward(retain_graph=True)


@pytest.mark.parametrize("Hk,Hv", [(1, 1), (1, 2), (1, 3)])
@pytest.mark.parametrize("K,V", [(8, 8), (40, 40), (72, 136), (104, 200), (64, 24), (24, 256)])
def test_results_do_not_depend_on_what_ran_before(K, V, Hk, Hv):
    # calls on NaN leave NaN in shared and tensor memory of every SM
    n = 128 * 300
    g = torch.zeros(n, 1).cuda()
    lens = [200, 0, 129, 1, 384]
    q, k, v, gates, do, s0 = (t.cuda() for t in _inputs(lens, Hk, Hv, K, V, seed=K))

    def after(value):
        x = torch.full((n, 1, 128), value, dtype=torch.bfloat16).cuda()
        out = []
        for states in (None, s0):
            cc.cattn_linear_fwd(x, x, x, g, _cu([n]))
            out += cc.cattn_linear_fwd(q, k, v, gates, _cu(lens), initial_state=states, final_state=True)[:2]
            cc.cattn_linear_bwd(x, x, x, g, x, _cu([n]))
            out += [t for t in cc.cattn_linear_bwd(q, k, v, gates, do, _cu(lens), initial_state=states)
                    if t is not None]
        return out

    for a, b in zip(after(float("nan")), after(0.0)):
        assert torch.isfinite(a).all() and torch.equal(a, b)
