"""The delta rule and layer norm without a GPU: host checks of the C ABI and of the binding, and the 64-bit
plain form against differences."""
import ctypes

import pytest
import torch

import depthwise_causal_short_gb300 as cc
from depthwise_causal_short_gb300 import _build, attn

P = 0x100000  # a fake, 16-byte aligned device address; never dereferenced by these tests
OK, ENULL, ESHAPE, EALIGN, ESTRIDE, EDTYPE, EWORK = 0, -1, -2, -4, -5, -6, -7


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return attn.load()


def _fwd(lib, q=P, sqt=128, sqh=64, k=P, v=P, svt=256, svh=64, g=P, sgt=4, sgh=1, beta=P, sbt=4, sbh=1, total=8,
         Hk=2, Hv=4, K=64, V=64, cu=P, nseq=2, init=None, fin=None, idx=None, S=2, status=None, o=P, ws=P,
         wsb=1 << 40):
    return lib.cattn_delta_fwd(q, sqt, sqh, k, 128, 64, v, svt, svh, g, sgt, sgh, beta, sbt, sbh, total, Hk, Hv,
                               K, V, cu, nseq, 1.0, init, fin, idx, S, status, o, ws, wsb, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(q=None), ENULL), (dict(k=None), ENULL), (dict(v=None), ENULL), (dict(g=None), ENULL),
    (dict(beta=None), ENULL), (dict(o=None), ENULL), (dict(cu=None), ENULL), (dict(idx=P), ENULL),
    (dict(total=-1), ESHAPE), (dict(total=1 << 31), ESHAPE), (dict(Hk=0), ESHAPE), (dict(Hv=3), ESHAPE),
    (dict(K=136), ESHAPE), (dict(V=264), ESHAPE), (dict(nseq=0), ESHAPE), (dict(fin=P, S=1), ESHAPE),
    (dict(idx=P, status=P, S=0), ESHAPE), (dict(nseq=1 << 29, S=1 << 29), ESHAPE), (dict(K=60), EALIGN),
    (dict(V=12), EALIGN), (dict(q=P + 2), EALIGN), (dict(beta=P + 2), EALIGN), (dict(o=P + 8), EALIGN),
    (dict(cu=P + 2), EALIGN), (dict(init=P + 4), EALIGN), (dict(sqt=132), EALIGN), (dict(svt=0), ESTRIDE),
    (dict(sbt=-1), ESTRIDE), (dict(sbh=-1), ESTRIDE), (dict(ws=None), EWORK), (dict(wsb=1000), EWORK),
    (dict(ws=P + 8), EALIGN),
])
def test_fwd_rejects(lib, kw, expect):
    assert _fwd(lib, **kw) == expect


def _bwd(lib, do=P, sot=256, dq=P, dk=P, dv=P, dg=P, dbeta=P, dinit=None, ws=P, wsb=1 << 40, beta=P, sbt=4, init=None,
         idx=None, S=2, status=None):
    return lib.cattn_delta_bwd(P, 128, 64, P, 128, 64, P, 256, 64, P, 4, 1, beta, sbt, 1, do, sot, 64, 8, 2, 4, 64,
                               64, P, 2, 1.0, init, idx, S, status, dq, dk, dv, dg, dbeta, dinit, ws, wsb, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(do=None), ENULL), (dict(dq=None), ENULL), (dict(dk=None), ENULL), (dict(dv=None), ENULL),
    (dict(dg=None), ENULL), (dict(dbeta=None), ENULL), (dict(beta=None), ENULL), (dict(idx=P), ENULL),
    (dict(init=P, S=1), ESHAPE), (dict(do=P + 2), EALIGN), (dict(dq=P + 8), EALIGN), (dict(dbeta=P + 4), EALIGN),
    (dict(dinit=P + 4), EALIGN), (dict(sot=20), EALIGN), (dict(sot=-8), ESTRIDE), (dict(sbt=-4), ESTRIDE),
    (dict(ws=None), EWORK), (dict(wsb=5000), EWORK), (dict(ws=P + 8), EALIGN),
])
def test_bwd_rejects(lib, kw, expect):
    assert _bwd(lib, **kw) == expect


def _upd(lib, q=P, g=P, beta=P, N=4, Hk=2, Hv=4, K=64, V=64, state=P, S=8, idx=P, o=P, status=P, sqt=128, sbt=4):
    return lib.cattn_delta_update(q, sqt, 64, P, 128, 64, P, 256, 64, g, 4, 1, beta, sbt, 1, N, Hk, Hv, K, V, 1.0,
                                  state, S, idx, 0, o, status, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(q=None), ENULL), (dict(g=None), ENULL), (dict(beta=None), ENULL), (dict(state=None), ENULL),
    (dict(o=None), ENULL), (dict(status=None), ENULL), (dict(N=0), ESHAPE), (dict(S=0), ESHAPE),
    (dict(idx=None, S=3), ESHAPE), (dict(Hv=5), ESHAPE), (dict(K=144), ESHAPE), (dict(K=68), EALIGN),
    (dict(state=P + 8), EALIGN), (dict(status=P + 2), EALIGN), (dict(beta=P + 1), EALIGN), (dict(sqt=0), ESTRIDE),
    (dict(sbt=-1), ESTRIDE),
])
def test_update_rejects(lib, kw, expect):
    assert _upd(lib, **kw) == expect


def _ln(lib, x=P, sxt=128, sxh=64, gate=P, szt=128, szh=64, total=4, H=2, C=64, w=P, b=P, wdt=1, mode=2, eps=1e-6, y=P):
    return lib.cattn_layernorm_fwd(x, sxt, sxh, gate, szt, szh, total, H, C, w, b, wdt, mode, eps, y, None)


LN_BAD = [
    (dict(x=None), ENULL), (dict(total=-1), ESHAPE), (dict(total=1 << 31), ESHAPE), (dict(H=0), ESHAPE),
    (dict(H=65536), ESHAPE), (dict(C=0), ESHAPE), (dict(C=8200), ESHAPE), (dict(mode=1), ESHAPE), (dict(mode=3), ESHAPE),
    (dict(eps=-1.0), ESHAPE), (dict(eps=float("nan")), ESHAPE), (dict(wdt=3), EDTYPE), (dict(C=60), EALIGN),
    (dict(x=P + 2), EALIGN), (dict(gate=P + 8), EALIGN), (dict(w=P + 2), EALIGN), (dict(b=P + 1, wdt=0), EALIGN),
    (dict(sxt=132), EALIGN), (dict(szh=4), EALIGN), (dict(sxt=0), ESTRIDE), (dict(szt=-8), ESTRIDE),
]


@pytest.mark.parametrize("kw,expect", LN_BAD + [(dict(y=None), ENULL), (dict(y=P + 8), EALIGN)])
def test_layernorm_fwd_rejects(lib, kw, expect):
    assert _ln(lib, **kw) == expect


def test_layernorm_fwd_nothing_to_do(lib):
    assert _ln(lib, total=0, x=None, gate=None, y=None) == OK


def _lnb(lib, x=P, sxt=128, sxh=64, dy=P, syt=128, gate=P, szt=128, szh=64, total=4, H=2, C=64, w=P, b=P, wdt=1, mode=2,
         eps=1e-6, dx=P, dgate=P, dw=P, db=P, ws=P, wsb=1 << 30):
    return lib.cattn_layernorm_bwd(x, sxt, sxh, dy, syt, 64, gate, szt, szh, total, H, C, w, b, wdt, mode, eps, dx, dgate,
                                   dw, db, ws, wsb, None)


@pytest.mark.parametrize("kw,expect", LN_BAD + [
    (dict(dy=None), ENULL), (dict(dx=None), ENULL), (dict(dgate=None), ENULL), (dict(dy=P + 4), EALIGN),
    (dict(syt=12), EALIGN), (dict(syt=-8), ESTRIDE), (dict(dx=P + 8), EALIGN), (dict(dgate=P + 2), EALIGN),
    (dict(dw=P + 2), EALIGN), (dict(db=P + 1, wdt=0), EALIGN),
])
def test_layernorm_bwd_rejects(lib, kw, expect):
    assert _lnb(lib, **kw) == expect


def test_workspace_queries(lib):
    n = ctypes.c_size_t(0)
    for fn in (lib.cattn_delta_fwd_workspace_bytes, lib.cattn_delta_bwd_workspace_bytes):
        assert fn(1, 1, 1, 1, 8, 8, None) == ENULL
        assert fn(-1, 1, 1, 1, 8, 8, ctypes.byref(n)) == ESHAPE
        assert fn(1, 0, 1, 1, 8, 8, ctypes.byref(n)) == ESHAPE
        assert fn(1, 1, 2, 3, 8, 8, ctypes.byref(n)) == ESHAPE
        assert fn(1, 1 << 29, 1, 8, 8, 64, ctypes.byref(n)) == ESHAPE  # more CTAs than a grid has
        sizes = []
        for total in (0, 1, 64, 65, 1000):
            assert fn(total, 3, 2, 4, 64, 64, ctypes.byref(n)) == OK
            sizes.append(n.value)
        assert sizes == sorted(sizes) and sizes[0] < 4096
    assert lib.cattn_layernorm_bwd_workspace_bytes(1, 1, 8, None) == ENULL
    assert lib.cattn_layernorm_bwd_workspace_bytes(1, 1, 8200, ctypes.byref(n)) == ESHAPE


# ---------------------------------------------------------------------------------------
# the binding: shapes, types, layouts and overlaps first, then the device
# ---------------------------------------------------------------------------------------

def _bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def _args(**kw):
    a = dict(q=_bf(6, 2, 64), k=_bf(6, 2, 64), v=_bf(6, 4, 32), g=torch.zeros(6, 4), beta=torch.zeros(6, 4),
             cu_seqlens=torch.tensor([0, 2, 6], dtype=torch.int32))
    a.update(kw)
    return a


@pytest.mark.parametrize("kw,err", [
    (dict(q=torch.zeros(6, 2, 64)), TypeError), (dict(k=_bf(6, 1, 64)), ValueError), (dict(v=_bf(6, 3, 32)), ValueError),
    (dict(beta=torch.zeros(6, 2)), ValueError), (dict(beta=torch.zeros(6)), ValueError), (dict(beta=None), TypeError),
    (dict(beta=_bf(6, 4)), TypeError), (dict(g=torch.zeros(6, 2)), ValueError),
    (dict(cu_seqlens=torch.tensor([0, 6])), TypeError), (dict(initial_state=torch.zeros(1, 4, 64, 32)), ValueError),
    (dict(initial_state=_bf(2, 4, 64, 32)), TypeError), (dict(o=_bf(6, 4, 64)), ValueError), (dict(), ValueError),
])
def test_fwd_binding_checks(kw, err):
    _build.build()
    with pytest.raises(err):
        cc.cattn_delta_fwd(**_args(**kw))


def test_bwd_and_update_binding_checks():
    _build.build()
    a = _args()
    with pytest.raises(ValueError):
        cc.cattn_delta_bwd(do=_bf(6, 4, 64), **a)
    with pytest.raises(ValueError, match="status"):
        cc.cattn_delta_bwd(do=_bf(6, 4, 32), state_indices=torch.zeros(2, dtype=torch.int32), **a)
    with pytest.raises(ValueError, match="dbeta"):
        cc.cattn_delta_bwd(do=_bf(6, 4, 32), dbeta=torch.zeros(6, 2), **a)
    with pytest.raises(ValueError, match="CUDA"):
        cc.cattn_delta_bwd(do=_bf(6, 4, 32), **a)
    a.pop("cu_seqlens")
    with pytest.raises(ValueError, match="slot"):
        cc.cattn_delta_update(**a, state=torch.zeros(2, 4, 64, 32))
    with pytest.raises(ValueError, match="beta"):
        cc.cattn_delta_update(**dict(a, beta=torch.zeros(5, 4)), state=torch.zeros(8, 4, 64, 32))


def _overlaps(fn, *args, **kw):
    with pytest.raises(ValueError, match="overlaps"):
        fn(*args, **kw)


def _passes(fn, *args, **kw):  # as far as the device check
    with pytest.raises(ValueError, match="CUDA"):
        fn(*args, **kw)


def test_what_is_written_overlaps_nothing():
    _build.build()
    a = _args()
    both = torch.zeros(12, 4)
    _passes(cc.cattn_delta_fwd, **a)
    _overlaps(cc.cattn_delta_fwd, **a, workspace=a["beta"])
    pool = torch.zeros(6, 4, 64, 32)
    _passes(cc.cattn_delta_fwd, **a, initial_state=pool, final_state=pool)
    _overlaps(cc.cattn_delta_fwd, **a, initial_state=pool[:4], final_state=pool[1:5])
    _overlaps(cc.cattn_delta_fwd, **dict(a, beta=pool.flatten()[:24].view(6, 4)), final_state=pool)
    b = dict(a, do=_bf(6, 4, 32))
    _passes(cc.cattn_delta_bwd, **b, dg=both[:6], dbeta=both[6:])
    _overlaps(cc.cattn_delta_bwd, **b, dg=both[:6], dbeta=both[5:11])
    _overlaps(cc.cattn_delta_bwd, **b, dbeta=a["beta"])
    _overlaps(cc.cattn_delta_bwd, **b, dbeta=a["g"])
    a.pop("cu_seqlens")
    _passes(cc.cattn_delta_update, **a, state=pool)
    _overlaps(cc.cattn_delta_update, **dict(a, beta=pool.flatten()[:24].view(6, 4)), state=pool)


@pytest.mark.parametrize("kw,err", [
    (dict(x=torch.zeros(6, 64)), TypeError), (dict(x=_bf(6, 2, 3, 64)), ValueError), (dict(x=_bf(64)), ValueError),
    (dict(x=_bf(6, 128)[:, ::2]), ValueError), (dict(w=torch.ones(32)), ValueError), (dict(w=torch.ones(64).half()), TypeError),
    (dict(w=torch.ones(64), b=_bf(64)), TypeError), (dict(b=torch.ones(64, 1)), ValueError), (dict(gate=_bf(6, 32)), ValueError),
    (dict(gate=torch.zeros(6, 64)), TypeError), (dict(mode="l2"), ValueError), (dict(mode=2), ValueError),
    (dict(eps="x"), TypeError), (dict(y=_bf(5, 64)), ValueError), (dict(), ValueError),
])
def test_layernorm_binding_checks(kw, err):
    _build.build()
    a = dict(x=_bf(6, 64))
    a.update(kw)
    with pytest.raises(err):
        cc.cattn_layernorm_fwd(**a)


def test_layernorm_gradient_binding_checks():
    _build.build()
    x, dy, w = _bf(6, 2, 64), _bf(6, 2, 64), torch.ones(64)
    bwd = cc.cattn_layernorm_bwd
    _passes(bwd, x, dy, w, gate=x)
    with pytest.raises(ValueError, match="dw without w"):
        bwd(x, dy, dw=torch.ones(64))
    with pytest.raises(ValueError, match="dgate without gate"):
        bwd(x, dy, w, dgate=_bf(6, 2, 64))
    with pytest.raises(ValueError):
        bwd(x, _bf(6, 2, 32), w)
    _overlaps(bwd, x, dy, w, dx=x)
    _overlaps(bwd, x, dy, w, dw=w)
    _overlaps(bwd, x, dy, w, dx=dy)
    _overlaps(bwd, x, dy, w, gate=_bf(6, 2, 64), dx=(y := _bf(6, 2, 64)), dgate=y)
    _overlaps(cc.cattn_layernorm_fwd, x, w, y=x)


def test_autograd_refuses_missing_states():
    with pytest.raises(ValueError):
        cc.delta_attention(**_args(), initial_state=torch.zeros(1, 4, 64, 32))


def test_plain_gradients_against_differences():
    from tests import delta_plain as plain
    q, k, v, g, beta, do, s0 = (t.double() for t in plain.delta_inputs([3, 0, 5], 1, 2, 8, 8, seed=3))
    leaves = [t.clone().requires_grad_() for t in (q, k, v, g, beta, s0)]
    assert torch.autograd.gradcheck(lambda *a: plain.delta(*a[:5], [0, 3, 3, 8], 0.3, a[5])[0], leaves)


def test_the_chunked_form_is_the_recurrence():
    """The identities that the kernels compute by, in 64 bits: J, P~, and the gradient with J's transpose."""
    n, K, V = 9, 5, 4
    gen = torch.Generator().manual_seed(0)

    def randn(*s):
        return torch.randn(*s, generator=gen, dtype=torch.float64)

    q, k, v, s0, do = randn(n, K), randn(n, K) / 3, randn(n, V), randn(K, V), randn(n, V)
    g, beta = -torch.rand(n, generator=gen, dtype=torch.float64), torch.rand(n, generator=gen, dtype=torch.float64)
    beta[3] = 0.0
    leaves = [t.clone().requires_grad_() for t in (q, k, v, g, beta, s0)]
    from tests import delta_plain as plain
    o, fin = plain.delta(leaves[0][:, None], leaves[1][:, None], leaves[2][:, None], leaves[3][:, None],
                         leaves[4][:, None], [0, n], 0.7, leaves[5][None, None])
    want = torch.autograd.grad(o[:, 0], leaves, do)
    G = g.cumsum(0)
    L = torch.exp(G[:, None] - G[None, :]).tril()
    ef, eb, total = torch.exp(G)[:, None], torch.exp(G[-1] - G)[:, None], torch.exp(G[-1])
    M, P, B = (k @ k.T * L).tril(-1), q @ k.T * L, torch.diag(beta)
    one = torch.eye(n, dtype=torch.float64)
    inv = torch.linalg.inv(one + B @ M)
    J, Pt = -M @ inv, P @ inv
    r = v - ef * (k @ s0)
    z = r + J @ (B @ r)
    u = B @ z
    assert torch.allclose(0.7 * (ef * (q @ s0) + Pt @ (B @ r)), o[:, 0])
    assert torch.allclose(total * s0 + k.T @ (eb * u), fin[0, 0])
    D = torch.zeros(K, V, dtype=torch.float64)
    rp = eb * (k @ D)
    du = rp + J.T @ (B @ rp) + 0.7 * Pt.T @ do
    dv = B @ du
    X, Y = (do @ u.T) * L, ((dv @ u.T) * L).tril(-1)
    assert torch.allclose(dv, want[2])
    assert torch.allclose((du * z).sum(1), want[4])
    assert torch.allclose(0.7 * (X @ k + ef * (do @ s0.T)), want[0])
    assert torch.allclose(0.7 * X.T @ q - (Y + Y.T) @ k + eb * (u @ D.T) - ef * (dv @ s0.T), want[1])
    dG = (o[:, 0].detach() * do).sum(1) - (v * dv).sum(1)
    assert torch.allclose(dG.flip(0).cumsum(0).flip(0), want[3])
    assert torch.allclose(total * D + 0.7 * q.T @ (ef * do) - k.T @ (ef * dv), want[5])
