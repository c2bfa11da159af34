"""libcattn.so without a GPU: exports, host checks of the C ABI and of the binding."""
import ctypes
import subprocess

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


def test_exports_match_header(lib):
    out = subprocess.run(["nm", "-D", "--defined-only", str(attn.lib_path())],
                         capture_output=True, text=True, check=True).stdout
    names = {ln.split()[-1] for ln in out.splitlines() if " T " in ln}
    assert names == set(attn.header_functions()) == set(attn._SIGNATURES)


def _norm(lib, q=P, sqt=128, sqh=64, k=P, skt=64, skh=64, total=4, Hq=2, Hk=1, K=64, wq=None,
          wk=None, wdt=1, mode=0, eps=1e-6, cos=P, sin=P, tab=16, R=32, pos=P, yq=P, yk=P):
    return lib.cattn_qknorm_fwd(q, sqt, sqh, k, skt, skh, total, Hq, Hk, K, wq, wk, wdt, mode, eps,
                                cos, sin, tab, R, 0, pos, yq, yk, None)


NORM_BAD = [
    (dict(q=None), ENULL), (dict(k=None), ENULL), (dict(cos=None), ENULL), (dict(sin=None), ENULL),
    (dict(total=-1), ESHAPE), (dict(Hq=0), ESHAPE), (dict(Hk=0), ESHAPE), (dict(K=0), ESHAPE),
    (dict(K=264), ESHAPE), (dict(mode=2), ESHAPE), (dict(eps=-1.0), ESHAPE),
    (dict(eps=float("nan")), ESHAPE), (dict(R=80), ESHAPE), (dict(R=-16), ESHAPE),
    (dict(tab=0), ESHAPE), (dict(pos=None, tab=3), ESHAPE), (dict(total=1 << 31), ESHAPE),
    (dict(K=60), EALIGN), (dict(R=24), EALIGN), (dict(q=P + 2), EALIGN), (dict(cos=P + 4), EALIGN),
    (dict(pos=P + 2), EALIGN), (dict(sqt=132), EALIGN), (dict(sqh=4), EALIGN),
    (dict(sqt=0), ESTRIDE), (dict(sqh=-64), ESTRIDE), (dict(wdt=3), EDTYPE),
    (dict(wq=P + 2), EALIGN), (dict(wk=P + 1, wdt=0), EALIGN),
]


@pytest.mark.parametrize("kw,expect", NORM_BAD)
def test_qknorm_fwd_rejects(lib, kw, expect):
    assert _norm(lib, **kw) == expect


def test_qknorm_fwd_output_rules(lib):
    assert _norm(lib, yq=None) == ENULL
    assert _norm(lib, yk=P + 8) == EALIGN
    assert _norm(lib, total=0, q=None, k=None, yq=None, yk=None) == OK  # nothing to do


def _normb(lib, dyq=P, dyk=P, total=4, dq=P, dk=P, dwq=None, dwk=None, ws=P, wsb=1 << 30, eps=0.0,
           syqt=128):
    return lib.cattn_qknorm_bwd(P, 128, 64, P, 64, 64, dyq, syqt, 64, dyk, 64, 64, total, 2, 1, 64,
                                None, None, 1, 0, eps, None, None, 0, 0, 0, None, dq, dk, dwq, dwk,
                                ws, wsb, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(dyq=None), ENULL), (dict(dyk=None), ENULL), (dict(dq=None), ENULL), (dict(dk=None), ENULL),
    (dict(dyq=P + 4), EALIGN), (dict(syqt=12), EALIGN), (dict(syqt=-8), ESTRIDE),
    (dict(dwq=P + 2), EALIGN), (dict(eps=-1.0), ESHAPE),
])
def test_qknorm_bwd_rejects(lib, kw, expect):
    assert _normb(lib, **kw) == expect


def _lin(lib, q=P, sqt=128, sqh=64, k=P, v=P, svt=256, svh=64, g=P, sgt=4, sgh=1, total=8, Hk=2,
         Hv=4, K=64, V=64, cu=P, nseq=2, init=None, fin=None, idx=None, S=2, status=None, o=P, ws=P,
         wsb=1 << 40):
    return lib.cattn_linear_fwd(q, sqt, sqh, k, 128, 64, v, svt, svh, g, sgt, sgh, total, Hk, Hv, K,
                                V, cu, nseq, 1.0, init, fin, idx, S, status, o, ws, wsb, None)


LIN_BAD = [
    (dict(q=None), ENULL), (dict(k=None), ENULL), (dict(v=None), ENULL), (dict(g=None), ENULL),
    (dict(o=None), ENULL), (dict(cu=None), ENULL), (dict(idx=P), ENULL), (dict(total=-1), ESHAPE),
    (dict(total=1 << 31), ESHAPE), (dict(Hk=0), ESHAPE), (dict(Hv=3), ESHAPE), (dict(Hv=0), ESHAPE),
    (dict(K=136), ESHAPE), (dict(K=0), ESHAPE), (dict(V=264), ESHAPE), (dict(nseq=0), ESHAPE),
    (dict(fin=P, S=1), ESHAPE), (dict(idx=P, status=P, S=0), ESHAPE),
    (dict(idx=P, status=P, S=393217), ESHAPE), (dict(K=60), EALIGN), (dict(V=12), EALIGN),
    (dict(q=P + 2), EALIGN), (dict(v=P + 8), EALIGN), (dict(g=P + 2), EALIGN),
    (dict(o=P + 8), EALIGN), (dict(cu=P + 2), EALIGN), (dict(init=P + 4), EALIGN),
    (dict(fin=P + 8), EALIGN), (dict(idx=P + 2, status=P), EALIGN), (dict(sqt=132), EALIGN),
    (dict(svh=68), EALIGN), (dict(svt=0), ESTRIDE), (dict(sqh=-8), ESTRIDE), (dict(sgt=-1), ESTRIDE),
]


@pytest.mark.parametrize("kw,expect", LIN_BAD)
def test_linear_fwd_rejects(lib, kw, expect):
    assert _lin(lib, **kw) == expect


def _linb(lib, do=P, sot=256, dq=P, dk=P, dv=P, dg=P, dinit=None, ws=P, wsb=1 << 40, init=None,
          idx=None, S=2, status=None):
    return lib.cattn_linear_bwd(P, 128, 64, P, 128, 64, P, 256, 64, P, 4, 1, do, sot, 64, 8, 2, 4, 64,
                                64, P, 2, 1.0, init, idx, S, status, dq, dk, dv, dg, dinit, ws, wsb,
                                None)


@pytest.mark.parametrize("kw,expect", [
    (dict(do=None), ENULL), (dict(dq=None), ENULL), (dict(dk=None), ENULL), (dict(dv=None), ENULL),
    (dict(dg=None), ENULL), (dict(idx=P), ENULL), (dict(init=P, S=1), ESHAPE),
    (dict(do=P + 2), EALIGN), (dict(dq=P + 8), EALIGN), (dict(dg=P + 4), EALIGN),
    (dict(dinit=P + 4), EALIGN), (dict(sot=20), EALIGN), (dict(sot=-8), ESTRIDE),
])
def test_linear_bwd_rejects(lib, kw, expect):
    assert _linb(lib, **kw) == expect


def _upd(lib, q=P, g=P, N=4, Hk=2, Hv=4, K=64, V=64, state=P, S=8, idx=P, o=P, status=P, sqt=128):
    return lib.cattn_linear_update(q, sqt, 64, P, 128, 64, P, 256, 64, g, 4, 1, N, Hk, Hv, K, V, 1.0,
                                   state, S, idx, 0, o, status, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(q=None), ENULL), (dict(g=None), ENULL), (dict(state=None), ENULL), (dict(o=None), ENULL),
    (dict(status=None), ENULL), (dict(N=0), ESHAPE), (dict(S=0), ESHAPE), (dict(idx=None, S=3), ESHAPE),
    (dict(S=393217), ESHAPE), (dict(Hv=5), ESHAPE), (dict(K=72 * 2), ESHAPE), (dict(K=68), EALIGN),
    (dict(state=P + 8), EALIGN), (dict(status=P + 2), EALIGN), (dict(idx=P + 1), EALIGN),
    (dict(sqt=130), EALIGN), (dict(sqt=0), ESTRIDE),
])
def test_linear_update_rejects(lib, kw, expect):
    assert _upd(lib, **kw) == expect


def test_workspace_queries_reject(lib):
    n = ctypes.c_size_t(0)
    for fn in (lib.cattn_linear_fwd_workspace_bytes, lib.cattn_linear_bwd_workspace_bytes):
        assert fn(1, 1, 1, 1, 8, 8, None) == ENULL
        assert fn(-1, 1, 1, 1, 8, 8, ctypes.byref(n)) == ESHAPE
        assert fn(1, 0, 1, 1, 8, 8, ctypes.byref(n)) == ESHAPE
        assert fn(1, 1, 2, 3, 8, 8, ctypes.byref(n)) == ESHAPE
    assert lib.cattn_qknorm_bwd_workspace_bytes(1, 1, 1, 8, None) == ENULL
    assert lib.cattn_qknorm_bwd_workspace_bytes(1, 1, 1, 300, ctypes.byref(n)) == ESHAPE
    assert lib.cattn_device_fault(None) == ENULL


# ---------------------------------------------------------------------------------------
# the binding's checks: shapes, types and layouts first, then the device
# ---------------------------------------------------------------------------------------

def _bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def _args(**kw):
    a = dict(q=_bf(6, 2, 64), k=_bf(6, 2, 64), v=_bf(6, 4, 32), g=torch.zeros(6, 4),
             cu_seqlens=torch.tensor([0, 6], dtype=torch.int32))
    a.update(kw)
    return a


@pytest.mark.parametrize("kw,err", [
    (dict(q=torch.zeros(6, 2, 64)), TypeError), (dict(q=_bf(6, 128)), ValueError),
    (dict(k=_bf(6, 1, 64)), ValueError), (dict(k=_bf(6, 2, 128)[..., ::2]), ValueError),
    (dict(v=_bf(5, 4, 32)), ValueError), (dict(v=_bf(6, 3, 32)), ValueError),
    (dict(g=torch.zeros(6, 2)), ValueError), (dict(g=torch.zeros(6, 4).bfloat16()), TypeError),
    (dict(g=None), TypeError), (dict(cu_seqlens=torch.tensor([0, 6])), TypeError),
    (dict(initial_state=torch.zeros(1, 4, 32, 64)), ValueError),
    (dict(initial_state=_bf(1, 4, 64, 32)), TypeError),
    (dict(cu_seqlens=torch.tensor([0, 3, 6], dtype=torch.int32),
          initial_state=torch.zeros(1, 4, 64, 32)), ValueError),
    (dict(state_indices=torch.tensor([0, 1], dtype=torch.int32)), ValueError),
    (dict(o=_bf(6, 4, 64)), ValueError), (dict(), ValueError),  # the last: not CUDA tensors
])
def test_linear_fwd_binding_checks(kw, err):
    with pytest.raises(err):
        cc.cattn_linear_fwd(**_args(**kw))


def test_linear_bwd_binding_checks():
    a = _args()
    with pytest.raises(ValueError):
        cc.cattn_linear_bwd(do=_bf(6, 4, 64), **a)
    with pytest.raises(ValueError, match="status"):
        cc.cattn_linear_bwd(do=_bf(6, 4, 32), state_indices=torch.zeros(1, dtype=torch.int32), **a)
    with pytest.raises(ValueError, match="CUDA"):
        cc.cattn_linear_bwd(do=_bf(6, 4, 32), **a)


def test_linear_update_binding_checks():
    a = _args()
    a.pop("cu_seqlens")
    with pytest.raises(ValueError, match="slot"):
        cc.cattn_linear_update(**a, state=torch.zeros(2, 4, 64, 32))
    with pytest.raises(ValueError):
        cc.cattn_linear_update(**a, state=torch.zeros(8, 4, 32, 32))
    with pytest.raises(ValueError, match="overlaps"):
        v = a["v"]
        cc.cattn_linear_update(**a, state=torch.zeros(8, 4, 64, 32), o=v)


@pytest.mark.parametrize("kw,err", [
    (dict(k=_bf(6, 2, 32)), ValueError), (dict(k=_bf(5, 2, 64)), ValueError),
    (dict(mode="layer"), ValueError), (dict(cos=torch.zeros(8, 16)), ValueError),
    (dict(cos=torch.zeros(5, 16), sin=torch.zeros(5, 16)), ValueError),
    (dict(positions=torch.zeros(6, dtype=torch.int32)), ValueError),
    (dict(cos=torch.zeros(8, 16), sin=torch.zeros(8, 16), positions=torch.zeros(6)), TypeError),
    (dict(wq=torch.ones(32)), ValueError), (dict(wq=torch.ones(64).half()), TypeError),
    (dict(wq=torch.ones(64), wk=torch.ones(64).bfloat16()), TypeError), (dict(), ValueError),
])
def test_qknorm_binding_checks(kw, err):
    a = dict(q=_bf(6, 2, 64), k=_bf(6, 2, 64))
    a.update(kw)
    with pytest.raises(err):
        cc.cattn_qknorm_fwd(**a)


def test_autograd_refuses_missing_states():
    a = _args(cu_seqlens=torch.tensor([0, 3, 6], dtype=torch.int32))
    with pytest.raises(ValueError):
        cc.decay_attention(**a, initial_state=torch.zeros(1, 4, 64, 32))


# ---------------------------------------------------------------------------------------
# the 64-bit plain forms against differences
# ---------------------------------------------------------------------------------------

def test_plain_gradients_against_differences():
    from tests import attn_plain as plain
    q, k, v, g, do, s0 = (t.double() for t in plain.linear_inputs([3, 0, 5], 1, 2, 8, 8, seed=3))
    cu = [0, 3, 3, 8]
    leaves = [t.clone().requires_grad_() for t in (q, k, v, g, s0)]
    assert torch.autograd.gradcheck(
        lambda *a: plain.linear(a[0], a[1], a[2], a[3], cu, 0.3, a[4])[0], leaves)
    x = torch.randn(4, 2, 32, dtype=torch.float64, requires_grad=True)
    w = torch.rand(32, dtype=torch.float64, requires_grad=True)
    ang = torch.rand(9, 8, dtype=torch.float64)
    pos = torch.tensor([8, 0, 3, 3])
    for mode in ("rms", "l2"):
        for inter in (False, True):
            assert torch.autograd.gradcheck(
                lambda a, b: plain.norm_rope(a, b, ang.cos(), ang.sin(), pos, mode, 1e-3, inter),
                (x, w))
