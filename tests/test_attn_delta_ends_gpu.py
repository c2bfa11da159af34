"""The delta rule's gradient at the ends of the ranges of its inputs (GPU).

Tolerances, as max |error| / max |reference| but for dg:
  dv, dq, dk   4.2e-3: the store's rounding, 2^-8 = 3.9e-3, and what the factors of 16 bits leave, 2^-15 of sums that
               may be a few times the result
  dbeta        2e-5, d_initial_state 5e-6: products that keep 24 bits, sums in fp32
  dg           of each head for itself.  dg_t is the sum of o_i.do_i - v_i.dv_i over up to 512 tokens, where o_i and
               dv_i are right to 1e-6 of their norm (products of 24 bits, sums of 64 + 128 values) and the
               dot products add 2^-24 sqrt(V) of the norms: 1.5e-6 |o_i| |do_i| a token, independent of
               one another, and as much for dv.  So 4 standard deviations are 4 sqrt(2 512) 1.5e-6 = 2e-4 of the
               head's largest |o_i| |do_i| + |v_i| |dv_i|; a token's part itself is of that size.
               Where exp(g) is 0, dg is 0.
"""
import pytest
import torch

import depthwise_causal_short_gb300 as cc
from depthwise_causal_short_gb300 import _build
from tests import delta_plain as plain

pytestmark = pytest.mark.gpu
NAMES = ("dq", "dk", "dv", "dg", "dbeta", "d_initial_state")
TOLS = (4.2e-3, 4.2e-3, 4.2e-3, None, 2e-5, 5e-6)


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()
    yield
    assert cc.cattn_device_fault() == 0


def _cu(lens):
    return torch.tensor([0] + list(lens), dtype=torch.int32).cumsum(0).to(torch.int32).cuda()


def _check(lens, q, k, v, g, beta, do, s0):
    scale = q.shape[2] ** -0.5
    leaves = [t.double().requires_grad_() for t in (q, k, v, g.clamp(min=-128.0), beta, s0)]
    cu = [0] + torch.tensor(lens).cumsum(0).tolist()
    o, _ = plain.delta(*leaves[:5], cu, scale, leaves[5])
    want = torch.autograd.grad(o, leaves, do.double())
    got = cc.cattn_delta_bwd(*[t.cuda() for t in (q, k, v, g, beta, do)], _cu(lens), initial_state=s0.cuda())
    sizes = o.detach().norm(dim=-1) * do.double().norm(dim=-1) + v.double().norm(dim=-1) * want[2].norm(dim=-1)
    for name, tol, a, b in zip(NAMES, TOLS, got, want):
        a = a.double().cpu()
        if name == "dg":
            off = (a - b).abs().amax(0) / sizes.amax(0)
            assert (off <= 2e-4).all(), off
            assert not a[torch.exp(g) == 0].any()
        else:
            # (a reference below fp32's smallest number: e^-128 = 2.6e-56 of a state behind a shut gate, which is 0 here)
            off, most = (a - b).abs().max().item(), b.abs().max().item()
            assert off <= tol * most + 2.0 ** -126, (name, off, most)


def _inputs(lens, seed=11, Hk=2, Hv=4, K=64, V=64):
    return plain.delta_inputs(lens, Hk, Hv, K, V, seed=seed)


@pytest.mark.parametrize("kind", ["beta_zero", "beta_two", "forget", "keep", "same_keys", "no_decay", "fast"])
@pytest.mark.parametrize("lens", [[150, 64, 3], [700]])
def test_ends_of_the_ranges(kind, lens):
    q, k, v, g, beta, do, s0 = _inputs(lens)
    if kind == "beta_zero":
        beta[:, ::2] = 0.0
        beta[::3] = 0.0
    elif kind == "beta_two":
        beta = 1.9 + 0.08 * torch.rand(beta.shape, generator=torch.Generator().manual_seed(1))
    elif kind == "forget":
        g[::5] = float("-inf")
        g[1::7] = -300.0
    elif kind == "keep":
        g = g * 1e-4
    elif kind == "no_decay":
        g = torch.zeros_like(g)
    elif kind == "fast":  # heads that keep next to nothing of a token: e^-20 and less
        g[:, ::2] = -20.0 + g[:, ::2]
    else:
        k = k[:1].expand_as(k).contiguous()
    _check(lens, q, k, v, g, beta, do, s0)


def test_shut_gates_at_the_borders():
    # gates shut at the ends of chunks, at the start of every eighth chunk, in whole chunks, in one head only
    lens = [1300, 65, 1]
    q, k, v, g, beta, do, s0 = _inputs(lens, seed=5, Hk=1, Hv=3, K=32, V=40)
    shut = float("-inf")
    g[[0, 63, 64, 127, 511, 512, 513, 640, 1299], 0] = shut
    g[[511, 1024], 1] = shut
    g[576:640, 1] = shut
    g[1300:1365, 2] = shut
    g[1365, 0] = shut
    _check(lens, q, k, v, g, beta, do, s0)


def test_what_is_before_a_shut_gate_does_not_count_on_what_is_behind():
    # dg before the gate is bit for bit that of a sequence which ends there
    lens = [640, 260]
    q, k, v, g, beta, do, s0 = (t.cuda() for t in _inputs(lens, seed=3))
    g[640] = float("-inf")
    whole = cc.cattn_delta_bwd(q, k, v, g, beta, do, _cu([900]), initial_state=s0[:1])
    alone = cc.cattn_delta_bwd(*[t[:640] for t in (q, k, v, g, beta, do)], _cu([640]), initial_state=s0[:1])
    assert torch.equal(whole[3][:640], alone[3]) and not whole[3][640].any()


@pytest.mark.parametrize("lens", [[1], [1, 0, 1, 130, 64, 1, 700]])
def test_the_first_gate_on_no_state(lens):
    # it acts on nothing: dg is 0, and the gates behind it are as right as ever
    q, k, v, g, beta, do, s0 = _inputs(lens, seed=8)
    leaf = g.double().requires_grad_()
    cu = [0] + torch.tensor(lens).cumsum(0).tolist()
    o, _ = plain.delta(q.double(), k.double(), v.double(), leaf, beta.double(), cu, 0.125)
    want, = torch.autograd.grad(o, leaf, do.double())
    args = [t.cuda() for t in (q, k, v, g, beta, do)]
    dg = cc.cattn_delta_bwd(*args, _cu(lens))[3].double().cpu()
    first = [a for a, b in zip(cu, cu[1:]) if b > a]
    assert not want[first].any() and not dg[first].any()
    off = (dg - want).abs().amax(0) / (o.detach().norm(dim=-1) * do.double().norm(dim=-1)).amax(0)
    assert (off <= 2e-4).all(), off
    # on a state it has one
    assert cc.cattn_delta_bwd(*args, _cu(lens), initial_state=s0.cuda())[3][first].any()
