"""A gated delta-rule block out of the library's operators: layer norm, short convolution, norm of
queries and keys, the delta rule, and the gated norm of its outputs, between plain projections.

    python examples/delta_mixer.py

    a = layer_norm(x);  [q k v] = silu(conv(a W)),  z = a Wz,  g, beta from a
    y = x + (norm(delta(l2norm(q), l2norm(k), v, g, beta)) * silu(z)) Wo

  prompt   packed prompts of different lengths; the convolution's and the rule's states land in
           the slots of two pools
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


class DeltaMixer:
    """Hk heads of queries and keys and Hv of values, K and V channels each, over rows of `width`
    channels."""

    def __init__(self, width=512, Hk=2, Hv=4, K=64, V=64, W=4, device="cuda", seed=0):
        g = torch.Generator().manual_seed(seed)
        self.Hk, self.Hv, self.K, self.V, self.W = Hk, Hv, K, V, W
        self.D = 2 * Hk * K + Hv * V

        def weight(rows, cols):
            return (torch.randn(rows, cols, generator=g) / rows ** 0.5).bfloat16().to(device)

        self.weights = {
            "ln_w": (1 + 0.1 * torch.randn(width, generator=g)).to(device),
            "ln_b": (0.1 * torch.randn(width, generator=g)).to(device),
            "qkv": weight(width, self.D), "gate": weight(width, Hv * V), "decay": weight(width, Hv),
            "beta": weight(width, Hv), "conv": (torch.rand(self.D, W, generator=g) - 0.5).to(device),
            "norm_w": (1 + 0.1 * torch.randn(V, generator=g)).to(device), "out": weight(Hv * V, width),
        }

    def split(self, y: torch.Tensor):
        """Views of the convolution's output [rows, D] as heads; nothing is copied."""
        a, b, rows = self.Hk * self.K, 2 * self.Hk * self.K, y.shape[0]
        return (y[:, :a].view(rows, self.Hk, self.K), y[:, a:b].view(rows, self.Hk, self.K),
                y[:, b:].view(rows, self.Hv, self.V))

    def pools(self, slots: int):
        """The decode state of `slots` sequences: the convolution's last W - 1 rows (bf16) and the
        rule's states (fp32)."""
        dev = self.weights["qkv"].device
        return (torch.zeros(slots, self.D, self.W - 1, dtype=torch.bfloat16, device=dev),
                torch.zeros(slots, self.Hv, self.K, self.V, device=dev))

    def gates(self, a, w):
        """The gate z of the outputs, log decays and step sizes of rows a."""
        z = (a @ w["gate"]).view(-1, self.Hv, self.V)
        g = -torch.nn.functional.softplus((a @ w["decay"]).float())
        return z, 0.1 * g, torch.sigmoid((a @ w["beta"]).float())

    def prompt(self, x, cu, pools, slots):
        """x [total, width] bf16, cu int32 [nseq + 1], slots int32 [nseq]; continues from the pools'
        states and leaves the new ones there."""
        w = self.weights
        a = cc.cattn_layernorm_fwd(x, w["ln_w"], w["ln_b"])
        z, g, beta = self.gates(a, w)
        y, _, _ = cc.cconv_fwd_varlen(a @ w["qkv"], cu, w["conv"], initial_state=pools[0],
                                      final_state=pools[0], state_indices=slots)
        q, k, v = self.split(y)
        q, k = cc.cattn_qknorm_fwd(q, k, mode="l2")
        o, _, status = cc.cattn_delta_fwd(q, k, v, g, beta, cu, initial_state=pools[1],
                                          final_state=pools[1], state_indices=slots)
        o = cc.cattn_layernorm_fwd(o, w["norm_w"], gate=z, mode="rms")
        return x + o.flatten(1) @ w["out"], status

    def step(self, x, pools, slots):
        """One token for each of N sequences: x [N, width], slots int32 [N]."""
        w = self.weights
        a = cc.cattn_layernorm_fwd(x, w["ln_w"], w["ln_b"])
        z, g, beta = self.gates(a, w)
        y, _ = cc.cconv_update(a @ w["qkv"], pools[0], w["conv"], None, slots)
        q, k, v = self.split(y)
        q, k = cc.cattn_qknorm_fwd(q, k, mode="l2")
        o, status = cc.cattn_delta_update(q, k, v, g, beta, pools[1], slots)
        o = cc.cattn_layernorm_fwd(o, w["norm_w"], gate=z, mode="rms")
        return x + o.flatten(1) @ w["out"], status

    def train(self, x, cu, weights=None):
        """The differentiable path from zero states; weights: those that ask for gradients."""
        w = {**self.weights, **(weights or {})}
        a = cc.layer_norm(x, w["ln_w"], w["ln_b"])
        z, g, beta = self.gates(a, w)
        y, _ = cc.causal_conv1d((a @ w["qkv"])[None], w["conv"], cu_seqlens=cu)
        q, k, v = self.split(y[0])
        q, k = cc.qk_norm_rope(q, k, mode="l2")
        o, _ = cc.delta_attention(q, k, v, g, beta, cu)
        return x + cc.layer_norm(o, w["norm_w"], gate=z, mode="rms").flatten(1) @ w["out"]


def offsets(lens):
    return torch.tensor([0] + list(lens), dtype=torch.int32).cumsum(0).to(torch.int32)


def main(lens=(300, 41, 170), tail=5, seed=1):
    """Returns (largest difference between the two ways, largest output, gradients by name)."""
    m = DeltaMixer()
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(sum(lens), 512, generator=gen).bfloat16().cuda()
    slots = torch.tensor([4, 0, 2], dtype=torch.int32).cuda()
    cu = offsets(lens).cuda()

    whole, status = m.prompt(x, cu, m.pools(6), slots)
    assert status.tolist() == [0, 0]

    # all but the last `tail` tokens as prompts, the rest one by one
    ends = cu[1:].tolist()
    keep = torch.cat([torch.arange(e - n, e - tail) for e, n in zip(ends, lens)]).cuda()
    pools = m.pools(6)
    m.prompt(x[keep], offsets([n - tail for n in lens]).cuda(), pools, slots)
    worst = 0.0
    for t in range(tail):
        rows = torch.tensor([e - tail + t for e in ends]).cuda()
        y, status = m.step(x[rows], pools, slots)
        assert status.tolist() == [0, 0]
        worst = max(worst, (y.float() - whole[rows].float()).abs().max().item())

    leaves = {n: t.clone().requires_grad_() for n, t in m.weights.items()}
    inputs = x.clone().requires_grad_()
    loss = m.train(inputs, cu, leaves).float().square().mean()
    grads = dict(zip(["x", *leaves], torch.autograd.grad(loss, [inputs, *leaves.values()])))
    assert cc.cconv_device_fault() == 0 and cc.cattn_device_fault() == 0
    return worst, whole.float().abs().max().item(), grads


if __name__ == "__main__":
    worst, size, grads = main()
    print(f"prompt against tokens: largest difference {worst:.3g} of {size:.3g}")
    print("gradient norms:", ", ".join(f"{n} {g.float().norm():.3g}" for n, g in grads.items()))
