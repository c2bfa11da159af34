"""The mixer's binding refuses what its kernels would answer wrongly (no GPU needed: shapes, layouts
and overlaps are checked before the device)."""
import pytest
import torch

import depthwise_causal_short_gb300 as cc
from depthwise_causal_short_gb300 import _build


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()


def _bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def _linear(**kw):
    a = dict(q=_bf(6, 2, 64), k=_bf(6, 2, 64), v=_bf(6, 4, 32), g=torch.zeros(6, 4),
             cu_seqlens=torch.tensor([0, 2, 6], dtype=torch.int32))
    a.update(kw)
    return a


def test_a_new_final_state_and_slots_of_a_larger_pool():
    idx = torch.tensor([4, 0], dtype=torch.int32)
    with pytest.raises(ValueError, match="final_state=True"):
        cc.cattn_linear_fwd(**_linear(), initial_state=torch.zeros(5, 4, 64, 32), final_state=True,
                            state_indices=idx)
    for n in (1, 2):  # no more slots than sequences: as far as the device check
        with pytest.raises(ValueError, match="CUDA"):
            cc.cattn_linear_fwd(**_linear(), initial_state=torch.zeros(n, 4, 64, 32), final_state=True,
                                state_indices=idx)


def _overlaps(fn, *args, **kw):
    with pytest.raises(ValueError, match="overlaps"):
        fn(*args, **kw)


def _passes(fn, *args, **kw):  # as far as the device check
    with pytest.raises(ValueError, match="CUDA"):
        fn(*args, **kw)


def test_what_a_forward_writes_overlaps_nothing():
    pool = torch.zeros(6, 4, 64, 32)
    a = _linear()
    fwd = cc.cattn_linear_fwd
    _passes(fwd, **a, initial_state=pool, final_state=pool)
    _passes(fwd, **a, initial_state=pool[:4], final_state=pool[:2])  # the same array, fewer slots
    _passes(fwd, **a, initial_state=pool[:3], final_state=pool[3:])
    _overlaps(fwd, **a, initial_state=pool[:4], final_state=pool[1:5])
    _overlaps(fwd, **a, initial_state=pool[1:], final_state=pool[:5])
    flat = pool.view(torch.uint8).flatten()
    _overlaps(fwd, **a, initial_state=pool, workspace=flat[64:128])
    _overlaps(fwd, **a, final_state=pool, workspace=flat[64:128])
    _overlaps(fwd, **a, final_state=pool, o=pool.view(torch.bfloat16).flatten()[:768].view(6, 4, 32))
    idx = torch.zeros(2, dtype=torch.int32)
    _overlaps(fwd, **a, initial_state=pool, state_indices=idx, status=idx)
    _overlaps(fwd, **a, initial_state=pool, state_indices=idx, status=a["cu_seqlens"])
    _passes(fwd, **a, initial_state=pool, state_indices=idx, status=idx.clone())


def test_what_a_gradient_writes_overlaps_nothing():
    a, bwd = dict(_linear(), do=_bf(6, 4, 32)), cc.cattn_linear_bwd
    s0 = torch.zeros(2, 4, 64, 32)
    ds = torch.zeros(2, 4, 64, 32)
    half = ds.view(torch.bfloat16).flatten()
    _passes(bwd, **a, initial_state=s0, d_initial_state=ds)
    _overlaps(bwd, **a, initial_state=s0, d_initial_state=s0)
    for name, n, shape in (("dq", 768, (6, 2, 64)), ("dk", 768, (6, 2, 64)), ("dv", 768, (6, 4, 32))):
        _overlaps(bwd, **a, initial_state=s0, d_initial_state=ds, **{name: half[8:8 + n].view(shape)})
    _overlaps(bwd, **a, initial_state=s0, d_initial_state=ds, dg=ds.flatten()[:24].view(6, 4))
    _overlaps(bwd, **a, initial_state=s0, d_initial_state=ds, workspace=half[:64])
    _overlaps(bwd, **a, dq=a["q"])
    _overlaps(bwd, **a, dq=half[:768].view(6, 2, 64), dv=half[760:1528].view(6, 4, 32))


def test_what_a_token_writes_overlaps_nothing():
    a, up = _linear(), cc.cattn_linear_update
    a.pop("cu_seqlens")
    state = torch.zeros(6, 4, 64, 32)
    half, ints = state.view(torch.bfloat16).flatten(), state.view(torch.int32).flatten()
    _passes(up, **a, state=state)
    _overlaps(up, **a, state=state, o=half[:768].view(6, 4, 32))
    _overlaps(up, **dict(a, v=half[:768].view(6, 4, 32)), state=state)
    _overlaps(up, **dict(a, g=state.flatten()[:24].view(6, 4)), state=state)
    _overlaps(up, **a, state=state, state_indices=ints[:6])
    _overlaps(up, **a, state=state, status=ints[:2])


def test_what_a_norm_writes_overlaps_nothing():
    q, k, w = _bf(6, 2, 64), _bf(6, 2, 64), torch.ones(64)
    tab = torch.zeros(8, 32)
    kw = dict(cos=tab, sin=tab.clone())
    fwd, bwd = cc.cattn_qknorm_fwd, cc.cattn_qknorm_bwd
    _passes(fwd, q, k, wq=w, wk=w, **kw)  # what is only read may be shared
    _overlaps(fwd, q, k, yq=q)
    _overlaps(fwd, q, k, yq=(y := _bf(6, 2, 64)), yk=y)
    wb = _bf(7, 2, 64)
    _overlaps(fwd, q, k, wq=wb.flatten()[:64], yq=wb.flatten()[:768].view(6, 2, 64))
    big = torch.zeros(16, 32)
    _overlaps(fwd, q, k, cos=big[:8], sin=tab, yq=big.view(torch.bfloat16).flatten()[:768].view(6, 2, 64))
    _passes(bwd, q, k, q, k, wq=w, wk=w, dwq=torch.ones(64), dwk=torch.ones(64))
    _overlaps(bwd, q, k, q, k, wq=w, wk=w, dwq=w)
    _overlaps(bwd, q, k, q, k, wq=w, wk=w, dwq=(d := torch.ones(64)), dwk=d)
    _overlaps(bwd, q, k, q, k, wq=w, wk=w, dwq=d, workspace=d)
    _overlaps(bwd, q, k, q, k, dq=(y := _bf(6, 2, 64)), dk=y)
    _overlaps(bwd, q, k, q, k, dq=q)
