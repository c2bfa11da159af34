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
