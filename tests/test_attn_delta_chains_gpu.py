"""The two ways in which the delta rule's gradient runs its chains: both in one launch where SMs are free, one
behind the other where they are not (GPU)."""
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


def _at_once(call):
    return any("delta_both" in d["name"] for d in cc.attn_describe(call))


@pytest.mark.parametrize("lens,K,V", [([1100, 200, 0, 90, 1], 64, 64), ([700], 128, 128), ([63, 640], 40, 200)])
def test_a_heads_gradient_is_the_same_either_way(lens, K, V):
    heads, few = 160, 2
    q, k, v, g, beta, do, s0 = (t.cuda() for t in plain.delta_inputs(lens, heads, heads, K, V, seed=K))
    cu = _cu(lens)

    def some(n):
        a = [t[:, :n].contiguous() for t in (q, k, v, g, beta, do)]
        return lambda: cc.cattn_delta_bwd(*a, cu, initial_state=s0[:, :n].contiguous())

    assert not _at_once(some(heads)) and _at_once(some(few))
    whole, part = some(heads)(), some(few)()
    for name, a, b in zip(("dq", "dk", "dv", "dg", "dbeta", "ds"), whole, part):
        a = a[:, :few]
        if name in ("dg", "dbeta"):
            # the same terms, summed in another order: 2^-24 a step of sums of V products, and for dg of the tokens'
            worst = ((a - b).abs().amax(0) / b.abs().amax(0)).max().item()
            assert worst <= 2e-5, (name, worst)
        else:
            assert torch.equal(a, b), name


@pytest.mark.parametrize("lens,Hv", [([400, 300, 64], 2), ([900], 16), ([300, 200], 40)])
def test_inputs_written_by_the_kernel_before(lens, Hv):
    # nothing is read before the kernels that write it have ended
    Hk, K, V = Hv, 64, 96
    sets = [[t.cuda() for t in plain.delta_inputs(lens, Hk, Hv, K, V, seed=s)] for s in (1, 2)]
    cu = _cu(lens)
    want = []
    for s in sets:
        want.append(cc.cattn_delta_bwd(*s[:6], cu, initial_state=s[6]))
        torch.cuda.synchronize()
    held = [t.clone() for t in sets[0]]
    ws = torch.empty(cc.cattn_delta_bwd_workspace_bytes(sum(lens), len(lens), Hk, Hv, K, V), dtype=torch.uint8, device="cuda")
    out = [torch.empty_like(t) for t in want[0]]
    names = ("dq", "dk", "dv", "dg", "dbeta", "d_initial_state")
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for i in range(60):
        ws.fill_(255)
        for t in out:
            t.zero_()
        torch._foreach_copy_(held, sets[i % 2])
        cc.cattn_delta_bwd(*held[:6], cu, initial_state=held[6], workspace=ws, **dict(zip(names, out)))
        for a, b in zip(out, want[i % 2]):
            wrong += (a != b).sum()
    assert wrong.item() == 0


@pytest.mark.parametrize("nseq", [1, 2])
def test_where_the_chains_run_at_once(nseq):
    # half of the SMs for the chain of one sequence, 5/8 with several; a CTA a head here
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    most = (sms // 2 if nseq == 1 else 5 * sms // 8) // nseq
    lens = [70] * nseq

    def call(heads):
        a = [t.cuda() for t in plain.delta_inputs(lens, heads, heads, 32, 32, seed=heads)[:6]]
        return lambda: cc.cattn_delta_bwd(*a, _cu(lens))

    assert _at_once(call(most)) and not _at_once(call(most + 1))
    for heads in (most, most + 1):
        assert all(bool(torch.isfinite(t).all()) for t in call(heads)() if t is not None)
