"""The gated delta rule in 64 bits, from its definition, for the tests (CPU torch)."""
from __future__ import annotations

import torch


def delta(q, k, v, g, beta, cu, scale, s0=None):
    """(o [total, Hv, V], final states [nseq, Hv, K, V]) by the recurrence, token by token;
    differentiable."""
    total, Hv, V = v.shape
    r = Hv // q.shape[1]
    q, k = q.repeat_interleave(r, 1), k.repeat_interleave(r, 1)
    outs, fins = [], []
    for i in range(len(cu) - 1):
        S = torch.zeros(Hv, q.shape[2], V, dtype=v.dtype) if s0 is None else s0[i]
        for t in range(cu[i], cu[i + 1]):
            S = g[t].exp()[:, None, None] * S
            u = beta[t][:, None] * (v[t] - torch.einsum("hk,hkv->hv", k[t], S))
            S = S + k[t][:, :, None] * u[:, None, :]
            outs.append(scale * torch.einsum("hk,hkv->hv", q[t], S))
        fins.append(S)
    o = torch.stack(outs) if outs else torch.zeros(0, Hv, V, dtype=v.dtype)
    return o, torch.stack(fins)


def delta_inputs(lens, Hk, Hv, K, V, seed=0, reach=64.0, most_beta=1.0):
    """(q, k, v, g, beta, do, s0) on the CPU: q, k, v, do bf16, g, beta and s0 fp32.  Keys of norm 1
    that are not orthogonal (normalised SiLU of normal values)."""
    gen = torch.Generator().manual_seed(seed)
    total = sum(lens)
    silu, norm = torch.nn.functional.silu, torch.nn.functional.normalize

    def randn(*s):
        return torch.randn(*s, generator=gen)

    q = (norm(silu(randn(total, Hk, K)), dim=-1) * K ** 0.5).bfloat16()
    k = norm(silu(randn(total, Hk, K)), dim=-1).bfloat16()
    v = silu(randn(total, Hv, V)).bfloat16()
    rate = torch.exp(-torch.linspace(0, 1, Hv) * torch.log(torch.tensor(reach)))
    g = -rate * torch.nn.functional.softplus(randn(total, Hv))
    beta = most_beta * torch.sigmoid(randn(total, Hv))
    do = randn(total, Hv, V).bfloat16()
    s0 = randn(len(lens), Hv, K, V)
    return q, k, v, g, beta, do, s0
