"""A token mixer out of the library's operators: short convolution, norm and rotation of queries
and keys, linear attention with a decay for each token and head.

    python examples/decay_mixer.py

One layer's path from its packed projections to the mixer's output, as a model would run it:

  prompt   packed prompts of different lengths; the convolution's and the attention's states
           land in the slots of two pools
  step     one token for each sequence, from and to the same slots
  train    the same path, differentiable, with one backward

main() runs a prompt whole, and in part with the rest token by token, and compares the two; then
one training step.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import depthwise_causal_short_gb300 as cc  # noqa: E402


class DecayMixer:
    """Hk heads of queries and keys and Hv of values, K and V channels each, behind one
    depthwise convolution of width W over the packed [q | k | v] projection."""

    def __init__(self, Hk=8, Hv=16, K=128, V=128, W=4, positions=4096, device="cuda", seed=0):
        g = torch.Generator().manual_seed(seed)
        self.Hk, self.Hv, self.K, self.V, self.W = Hk, Hv, K, V, W
        self.D = 2 * Hk * K + Hv * V
        self.conv = (torch.rand(self.D, W, generator=g) - 0.5).to(device)
        self.wq = (1 + 0.1 * torch.randn(K, generator=g)).to(device)
        self.wk = (1 + 0.1 * torch.randn(K, generator=g)).to(device)
        freq = 10000.0 ** (-torch.arange(0, K, 2, dtype=torch.float64) / K)
        angle = torch.arange(positions, dtype=torch.float64)[:, None] * freq
        self.cos, self.sin = angle.cos().float().to(device), angle.sin().float().to(device)

    def split(self, x: torch.Tensor):
        """Views of the convolution's output [rows, D] as heads; nothing is copied."""
        a, b = self.Hk * self.K, 2 * self.Hk * self.K
        rows = x.shape[0]
        return (x[:, :a].view(rows, self.Hk, self.K), x[:, a:b].view(rows, self.Hk, self.K),
                x[:, b:].view(rows, self.Hv, self.V))

    def pools(self, slots: int):
        """The decode state of `slots` sequences: the convolution's last W - 1 rows (bf16) and the
        attention's states (fp32)."""
        dev = self.conv.device
        return (torch.zeros(slots, self.D, self.W - 1, dtype=torch.bfloat16, device=dev),
                torch.zeros(slots, self.Hv, self.K, self.V, device=dev))

    def prompt(self, x, g, cu, positions, pools, slots):
        """x [total, D] bf16, g [total, Hv] log decays, cu int32 [nseq + 1], positions int32 [total],
        slots int32 [nseq]; continues from the pools' states and leaves the new ones there."""
        y, _, _ = cc.cconv_fwd_varlen(x, cu, self.conv, initial_state=pools[0], final_state=pools[0],
                                      state_indices=slots)
        q, k, v = self.split(y)
        q, k = cc.cattn_qknorm_fwd(q, k, wq=self.wq, wk=self.wk, cos=self.cos, sin=self.sin,
                                   positions=positions)
        o, _, status = cc.cattn_linear_fwd(q, k, v, g, cu, initial_state=pools[1], final_state=pools[1],
                                           state_indices=slots)
        return o, status

    def step(self, x, g, positions, pools, slots):
        """One token for each of N sequences: x [N, D], g [N, Hv], positions and slots int32 [N]."""
        y, _ = cc.cconv_update(x, pools[0], self.conv, None, slots)
        q, k, v = self.split(y)
        q, k = cc.cattn_qknorm_fwd(q, k, wq=self.wq, wk=self.wk, cos=self.cos, sin=self.sin,
                                   positions=positions)
        return cc.cattn_linear_update(q, k, v, g, pools[1], slots)

    def train(self, x, g, cu, positions, weights=None):
        """The differentiable path from zero states; weights: (conv, wq, wk) that ask for gradients."""
        conv, wq, wk = weights or (self.conv, self.wq, self.wk)
        y, _ = cc.causal_conv1d(x[None], conv, cu_seqlens=cu)
        q, k, v = self.split(y[0])
        q, k = cc.qk_norm_rope(q, k, wq, wk, self.cos, self.sin, positions)
        return cc.decay_attention(q, k, v, g, cu)[0]


def positions_of(lens, start=0):
    return torch.cat([torch.arange(start, start + n, dtype=torch.int32) for n in lens])


def offsets(lens):
    return torch.tensor([0] + list(lens), dtype=torch.int32).cumsum(0).to(torch.int32)


def main(lens=(300, 41, 170), tail=5, seed=1):
    """Returns (largest difference between the two ways, largest output, gradients)."""
    m = DecayMixer(Hk=2, Hv=4, K=64, V=64)
    gen = torch.Generator().manual_seed(seed)
    total = sum(lens)
    x = torch.randn(total, m.D, generator=gen).bfloat16().cuda()
    g = (-torch.rand(total, m.Hv, generator=gen) * 0.1).cuda()
    slots = torch.tensor([4, 0, 2], dtype=torch.int32).cuda()
    cu, pos = offsets(lens).cuda(), positions_of(lens).cuda()

    whole, status = m.prompt(x, g, cu, pos, m.pools(6), slots)
    assert status.tolist() == [0, 0]

    # all but the last `tail` tokens as prompts, the rest one by one
    ends = cu[1:].tolist()
    keep = torch.cat([torch.arange(e - n, e - tail) for e, n in zip(ends, lens)]).cuda()
    short = [n - tail for n in lens]
    pools = m.pools(6)
    m.prompt(x[keep], g[keep], offsets(short).cuda(), pos[keep].contiguous(), pools, slots)
    worst = 0.0
    for t in range(tail):
        rows = torch.tensor([e - tail + t for e in ends]).cuda()
        o, status = m.step(x[rows], g[rows], pos[rows].contiguous(), pools, slots)
        assert status.tolist() == [0, 0]
        worst = max(worst, (o.float() - whole[rows].float()).abs().max().item())

    leaves = [t.clone().requires_grad_() for t in (x, g, m.conv, m.wq, m.wk)]
    loss = m.train(leaves[0], leaves[1], cu, pos, leaves[2:]).float().square().mean()
    grads = torch.autograd.grad(loss, leaves)
    assert cc.cconv_device_fault() == 0 and cc.cattn_device_fault() == 0
    return worst, whole.float().abs().max().item(), grads


if __name__ == "__main__":
    worst, size, grads = main()
    print(f"prompt against tokens: largest difference {worst:.3g} of {size:.3g}")
    print("gradient norms:", ", ".join(f"{n} {g.float().norm():.3g}" for n, g in
                                       zip(("x", "g", "conv", "wq", "wk"), grads)))
