"""The mixer operators in 64 bits, from their definitions, for the tests (CPU torch)."""
from __future__ import annotations

import torch


def norm_rope(x, w, cos, sin, pos, mode, eps, interleaved):
    """x [rows, heads, dim] double -> normed, weighted and rotated; differentiable."""
    m = x.square().mean(-1, keepdim=True) if mode == "rms" else x.square().sum(-1, keepdim=True)
    u = x / torch.sqrt(m + eps)
    if w is not None:
        u = u * w
    if cos is None:
        return u
    r = 2 * cos.shape[1]
    at = torch.arange(x.shape[0]) if pos is None else pos.long()
    c, s = cos[at][:, None, :], sin[at][:, None, :]
    head, rest = u[..., :r], u[..., r:]
    if interleaved:
        a, b = head[..., 0::2], head[..., 1::2]
        return torch.cat((torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2), rest), -1)
    a, b = head[..., :r // 2], head[..., r // 2:]
    return torch.cat((a * c - b * s, b * c + a * s, rest), -1)


def linear(q, k, v, g, cu, scale, s0=None):
    """(o [total, Hv, V], final states [nseq, Hv, K, V]) by the recurrence, token by token;
    differentiable."""
    total, Hv, V = v.shape
    r = Hv // q.shape[1]
    q, k = q.repeat_interleave(r, 1), k.repeat_interleave(r, 1)
    outs, fins = [], []
    for i in range(len(cu) - 1):
        S = torch.zeros(Hv, q.shape[2], V, dtype=v.dtype) if s0 is None else s0[i]
        for t in range(cu[i], cu[i + 1]):
            S = g[t].exp()[:, None, None] * S + k[t][:, :, None] * v[t][:, None, :]
            outs.append(scale * torch.einsum("hk,hkv->hv", q[t], S))
        fins.append(S)
    o = torch.stack(outs) if outs else torch.zeros(0, Hv, V, dtype=v.dtype)
    return o, torch.stack(fins)


def linear_inputs(lens, Hk, Hv, K, V, seed=0, reach=64.0):
    """(q, k, v, g, do, s0) on the CPU: q, k, v, do bf16, g and s0 fp32."""
    gen = torch.Generator().manual_seed(seed)
    total = sum(lens)

    def randn(*s):
        return torch.randn(*s, generator=gen)

    q = (randn(total, Hk, K)).bfloat16()
    k = (randn(total, Hk, K) / K ** 0.5).bfloat16()
    v = torch.nn.functional.silu(randn(total, Hv, V)).bfloat16()
    rate = torch.exp(-torch.linspace(0, 1, Hv) * torch.log(torch.tensor(reach)))
    g = -rate * torch.nn.functional.softplus(randn(total, Hv))
    do = randn(total, Hv, V).bfloat16()
    s0 = randn(len(lens), Hv, K, V)
    return q, k, v, g, do, s0
