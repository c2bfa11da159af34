"""Measured cases of the mixer operators that follow the short convolution.

Three operators, each through the package's public calls:

  qknorm_fwd / qknorm_bwd   per-head norm of queries and keys with the position rotation in
                            the same pass, and its gradient
  linear_fwd / linear_bwd   linear attention with a decay per token and head over packed
                            sequences (prompts and training), and its gradient
  linear_update             its recurrent form for single tokens, on a pooled fp32 state

A case names the call and its sizes.  `run` computes the plain form (elementary torch
operations in fp32) or, with `own`, makes the package's calls; `exact` is the definition in
64 bits.

Sizes: rows and head counts of the package's q/k/v workload (16384 rows; q and k of 1024
channels as 8 heads of 128, v of 2048 as 16 heads of 128), its decode pool (512 slots, 256
rows), its ragged shape (4 x 777 rows) and a 64-row one, with odd ones in between.
"""
import math
import random

import torch

own = False

# ---------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------


def _norm(op, rows, hq, hk, dim, rot, mode, weights, interleaved, maxpos):
    return {"op": op, "rows": rows, "hq": hq, "hk": hk, "dim": dim, "rot": rot, "mode": mode,
            "weights": weights, "interleaved": interleaved, "maxpos": maxpos}


def _lin(op, total, nseq, hk, hv, kd, vd, states, slots, mix):
    # states: initial and final states in pool slots (forward), an initial state and its
    # gradient (backward).  mix: which mixture of lengths.
    return {"op": op, "total": total, "nseq": nseq, "hk": hk, "hv": hv, "kd": kd, "vd": vd,
            "states": states, "slots": slots, "mix": mix}


def _upd(rows, pads, slots, hk, hv, kd, vd):
    return {"op": "linear_update", "rows": rows, "pads": pads, "slots": slots, "hk": hk, "hv": hv,
            "kd": kd, "vd": vd}


def listed():
    return [
        # one decode step of a small batch: a call of a few microseconds, where latency counts
        dict(_norm("qknorm_fwd", 4, 8, 8, 128, 128, "rms", "f32", False, 40960), name="norm_decode4"),
        # the norm of a whole packed training batch or prompt
        dict(_norm("qknorm_fwd", 16384, 8, 8, 128, 128, "rms", "f32", False, 8192), name="norm_prompt"),
        # its gradient, with the weights' gradients
        dict(_norm("qknorm_bwd", 16384, 8, 8, 128, 128, "rms", "f32", False, 8192), name="norm_train"),
        # a ragged batch with odd heads, a partial rotation of neighbouring pairs, no weights
        dict(_norm("qknorm_bwd", 3108, 5, 3, 96, 32, "l2", "none", True, 777), name="norm_train_odd"),
        # the shortest prompt of one sequence: latency
        dict(_lin("linear_fwd", 64, 1, 8, 8, 128, 128, False, 0, 0), name="lin_short"),
        # a serving prefill: 16 sequences of mixed lengths, states read from and written to a pool
        dict(_lin("linear_fwd", 16384, 16, 8, 16, 128, 128, True, 64, 1), name="lin_prefill"),
        # a training batch of two long rows, v with twice the heads of q and k
        dict(_lin("linear_fwd", 16384, 2, 8, 16, 128, 128, False, 0, 0), name="lin_train_fwd"),
        # a small ragged batch with other head widths
        dict(_lin("linear_fwd", 3108, 7, 4, 4, 64, 96, True, 9, 2), name="lin_ragged"),
        # the gradient of the training batch
        dict(_lin("linear_bwd", 16384, 2, 8, 16, 128, 128, False, 0, 0), name="lin_train_bwd"),
        # the gradient of a ragged batch with initial states
        dict(_lin("linear_bwd", 3108, 7, 4, 4, 64, 96, True, 7, 2), name="lin_ragged_bwd"),
        # one token of one sequence
        dict(_upd(1, 0, 8, 8, 16, 128, 128), name="step1"),
        # a full decode batch out of a pool of 512 slots, a few of its rows padding
        dict(_upd(256, 5, 512, 8, 16, 128, 128), name="step256"),
    ]


def _log(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    n = min(hi, max(lo, n))
    return n + 1 if n == 3072 else n  # a multiple of the head widths no workload here has


def _heads(rng, widths):
    """(hk, hv, kd, vd) with at most 2048 channels of q, k and 4096 of v."""
    while True:
        hk, r = rng.choice([1, 2, 3, 4, 6, 8]), rng.choice([1, 1, 2, 4])
        kd, vd = rng.choice(widths[0]), rng.choice(widths[1])
        hv = hk * r
        if hk * kd <= 2048 and hv * vd <= 4096 and 3072 not in (hk * kd, hv * vd):
            return hk, hv, kd, vd


def draw(rng):
    op = rng.choice(["qknorm_fwd", "qknorm_bwd", "linear_fwd", "linear_bwd", "linear_update"])
    if op.startswith("qknorm"):
        while True:
            hq, hk = rng.choice([1, 2, 4, 5, 8, 12]), rng.choice([1, 2, 3, 4, 8])
            dim = rng.choice([32, 64, 80, 96, 128, 256])
            if (hq + hk) * dim <= 2048 and 3072 not in (hq * dim, hk * dim):
                break
        rot = rng.choice([0, 16, dim // 32 * 16, dim // 16 * 16])
        return _norm(op, _log(rng, 1, 16384), hq, hk, dim, rot, rng.choice(["rms", "l2"]),
                     rng.choice(["f32", "bf16", "none"]), rng.choice([False, True]),
                     rng.choice([777, 8192, 40960]))
    widths = ([32, 64, 96, 128], [32, 64, 96, 128, 256])
    hk, hv, kd, vd = _heads(rng, widths)
    if op == "linear_update":
        most = max(1, min(256, 256 * 16 * 128 * 128 // (hv * kd * vd)))
        rows = _log(rng, 1, most)
        return _upd(rows, rng.randint(0, rows // 8), rows + rng.randint(0, rows), hk, hv, kd, vd)
    while hk * kd + hv * vd > 1024 + 2048:
        hk, hv, kd, vd = _heads(rng, widths)
    total = _log(rng, 1, 16384)
    nseq = _log(rng, 1, min(64, total))
    states = rng.choice([False, True])
    return _lin(op, total, nseq, hk, hv, kd, vd, states,
                (nseq + rng.randint(0, 4) if op == "linear_fwd" else nseq) if states else 0,
                rng.randint(0, 5))


def _lengths(case):
    """Lengths of the packed sequences: equal ones (mix 0), else log-uniform over a 32-fold
    range with one empty and one single-token sequence where there are four or more."""
    total, nseq, mix = case["total"], case["nseq"], case["mix"]
    if nseq == 1:
        return [total]
    if mix == 0:
        return [total * (i + 1) // nseq - total * i // nseq for i in range(nseq)]
    rng = random.Random(mix)
    w = [32.0 ** rng.random() for _ in range(nseq)]
    fixed = {1: 0, nseq - 2: 1} if nseq >= 4 and total >= nseq else {}
    rest = total - sum(fixed.values())
    scale = rest / sum(x for i, x in enumerate(w) if i not in fixed)
    lens = [fixed.get(i, int(x * scale)) for i, x in enumerate(w)]
    lens[0] += total - sum(lens)
    return lens


# ---------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------


def prepare(case, seed):
    dev = torch.device("cuda", 0)
    gen = torch.Generator(device=dev).manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    def rand(*shape):
        return torch.rand(*shape, generator=gen, device=dev)

    def bf(x):
        return x.to(torch.bfloat16)

    s = {"case": case}
    if case["op"].startswith("qknorm"):
        rows, hq, hk, dim, rot = (case[n] for n in ("rows", "hq", "hk", "dim", "rot"))
        # q and k: the convolution's outputs, SiLU of roughly normal values
        s["q"] = bf(torch.nn.functional.silu(randn(rows, hq, dim)))
        s["k"] = bf(torch.nn.functional.silu(randn(rows, hk, dim)))
        wt = {"f32": torch.float32, "bf16": torch.bfloat16, "none": None}[case["weights"]]
        s["wq"] = None if wt is None else (1 + 0.2 * randn(dim)).to(wt)
        s["wk"] = None if wt is None else (1 + 0.2 * randn(dim)).to(wt)
        s["cos"] = s["sin"] = s["positions"] = None
        if rot:
            n = case["maxpos"]
            freq = 10000.0 ** (-torch.arange(rot // 2, device=dev, dtype=torch.float64) * 2 / rot)
            ang = torch.arange(n, device=dev, dtype=torch.float64)[:, None] * freq
            s["cos"], s["sin"] = ang.cos().float(), ang.sin().float()
            # rows of consecutive tokens from a random start, as sequences have them
            start = int(torch.randint(0, n, (1,), generator=gen, device=dev))
            s["positions"] = ((torch.arange(rows, device=dev) + start) % n).to(torch.int32)
        if case["op"] == "qknorm_bwd":
            s["dyq"], s["dyk"] = bf(randn(rows, hq, dim)), bf(randn(rows, hk, dim))
        return s

    hk, hv, kd, vd = (case[n] for n in ("hk", "hv", "kd", "vd"))
    rows = case["rows"] if case["op"] == "linear_update" else case["total"]
    norm = torch.nn.functional.normalize
    s["q"] = bf(norm(randn(rows, hk, kd), dim=-1) * kd ** 0.5)
    s["k"] = bf(norm(randn(rows, hk, kd), dim=-1))
    s["v"] = bf(torch.nn.functional.silu(randn(rows, hv, vd)))
    # log decays: heads remember from a few tokens to a few thousand, each token moves it
    reach = torch.exp(torch.linspace(0.0, -math.log(2048.0), hv, device=dev)) if hv > 1 else \
        torch.full((1,), 1 / 64, device=dev)
    s["g"] = -reach * torch.nn.functional.softplus(randn(rows, hv))
    if case["op"] == "linear_update":
        n, slots, pads = rows, case["slots"], case["pads"]
        s["state"] = randn(slots, hv, kd, vd)
        idx = torch.randperm(slots, generator=gen, device=dev)[:n].to(torch.int32)
        idx[n - pads:] = -1  # a padded batch: its last rows name no slot
        s["idx"] = idx
        s["o"] = torch.zeros(n, hv, vd, dtype=torch.bfloat16, device=dev)
        return s
    cu = [0]
    for n in _lengths(case):
        cu.append(cu[-1] + n)
    s["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
    s["idx"] = s["state"] = None
    if case["states"]:
        s["state"] = randn(case["slots"], hv, kd, vd)
        if case["op"] == "linear_fwd":
            s["idx"] = torch.randperm(case["slots"], generator=gen,
                                      device=dev)[:case["nseq"]].to(torch.int32)
            s["final"] = torch.zeros_like(s["state"])
    if case["op"] == "linear_bwd":
        s["do"] = bf(randn(rows, hv, vd))
    return s


# ---------------------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------------------

CHUNK = 64
EPS = 1e-6


def _rotate(u, cos, sin, rot, interleaved, sign):
    """u [rows, heads, dim], the first `rot` channels rotated by sign * angle."""
    if not rot:
        return u
    c, s = cos[:, None, :], sign * sin[:, None, :]
    head, rest = u[..., :rot], u[..., rot:]
    if interleaved:
        a, b = head[..., 0::2], head[..., 1::2]
        y = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    else:
        a, b = head[..., :rot // 2], head[..., rot // 2:]
        y = torch.cat((a * c - b * s, b * c + a * s), -1)
    return torch.cat((y, rest), -1)


def _norm_fwd(x, w, cos, sin, case):
    x = x.float()
    m = x.square().mean(-1, keepdim=True) if case["mode"] == "rms" else x.square().sum(-1, keepdim=True)
    u = x * torch.rsqrt(m + EPS)
    if w is not None:
        u = u * w.float()
    return _rotate(u, cos, sin, case["rot"], case["interleaved"], 1.0).to(torch.bfloat16)


def _norm_bwd(x, w, dy, cos, sin, case):
    x = x.float()
    rms = case["mode"] == "rms"
    m = x.square().mean(-1, keepdim=True) if rms else x.square().sum(-1, keepdim=True)
    r = torch.rsqrt(m + EPS)
    n = x * r
    du = _rotate(dy.float(), cos, sin, case["rot"], case["interleaved"], -1.0)
    dn = du if w is None else du * w.float()
    t = (dn * n).mean(-1, keepdim=True) if rms else (dn * n).sum(-1, keepdim=True)
    dx = r * (dn - n * t)
    dw = None if w is None else (du * n).sum((0, 1)).to(w.dtype)
    return dx.to(torch.bfloat16), dw


def _pairs(x):
    """T[..., i, j] = sum of x[..., m] over j < m <= i, and zero for j >= i; sums of one sign
    never cancel here, unlike differences of one running sum."""
    n = x.shape[-1]
    low = torch.ones(n, n, dtype=torch.bool, device=x.device).tril(-1)
    return (x[..., :, None] * low).cumsum(-2)


def _linear(q, k, v, g, cu, s0, scale):
    """o [total, hv, vd] and the final states, in chunks of CHUNK tokens; all fp32."""
    total, nseq, r = q.shape[0], cu.numel() - 1, v.shape[1] // q.shape[1]
    C, dev = CHUNK, q.device
    cu = cu.long()
    n = (cu[1:] - cu[:-1] + C - 1) // C
    ends = n.cumsum(0)
    c = torch.arange(total // C + nseq, device=dev)  # no fewer chunks than there can be
    seq = torch.searchsorted(ends, c, right=True).clamp(max=nseq - 1)
    row = (cu[seq] + (c - (ends - n)[seq]) * C)[:, None] + torch.arange(C, device=dev)
    ok = (row < cu[1:][seq][:, None]) & (c < ends[-1])[:, None]

    def cut(x):  # [total, h, ...] -> [chunks, h, C, ...], zeros in rows that are no token
        y = x[torch.where(ok, row, 0)]
        return torch.where(ok.view(*ok.shape, *[1] * (y.dim() - 2)), y, 0.0).transpose(1, 2)

    qc, kc = (cut(x).repeat_interleave(r, 1) for x in (q, k))
    vc, gc = cut(v), cut(g)
    t = _pairs(gc)
    low = torch.ones(C, C, dtype=torch.bool, device=dev).tril()
    o = (qc @ kc.transpose(-1, -2) * t.exp() * low) @ vc
    local = (kc * t[..., -1, :, None].exp()).transpose(-1, -2) @ vc
    whole = gc.sum(-1)  # [chunks, h]
    between = torch.nn.functional.pad(_pairs(whole.T)[:, :-1], (0, 0, 1, 0))
    same = (seq[:, None] == seq[None, :]) & (c[:, None] > c[None, :])
    mix = torch.where(same, between.exp(), 0.0)
    s_in = torch.einsum("hcj,jhkv->chkv", mix, local)
    if s0 is not None:
        s_in = s_in + (same.float() @ whole).exp()[..., None, None] * s0[seq]
    o = o + (qc * gc.cumsum(-1).exp()[..., None]) @ s_in
    out = torch.zeros(total + 1, v.shape[1], v.shape[2], device=dev)
    out = out.index_put((torch.where(ok, row, total),), scale * o.transpose(1, 2))[:total]
    last = (ends - 1).clamp(min=0)
    fin = whole[last].exp()[..., None, None] * s_in[last] + local[last]
    first = torch.zeros_like(fin) if s0 is None else s0
    return out, torch.where((n > 0)[:, None, None, None], fin, first)


def _plain(s):
    case = s["case"]
    op = case["op"]
    bf = torch.bfloat16
    if op.startswith("qknorm"):
        pos = s["positions"]
        cos, sin = (None, None) if pos is None else (s["cos"][pos], s["sin"][pos])
        if op == "qknorm_fwd":
            return [_norm_fwd(s["q"], s["wq"], cos, sin, case), _norm_fwd(s["k"], s["wk"], cos, sin, case)]
        dq, dwq = _norm_bwd(s["q"], s["wq"], s["dyq"], cos, sin, case)
        dk, dwk = _norm_bwd(s["k"], s["wk"], s["dyk"], cos, sin, case)
        return [dq, dk, dwq, dwk]
    scale = case["kd"] ** -0.5
    f = [s[n].float() for n in ("q", "k", "v", "g")]
    if op == "linear_update":
        n = case["rows"] - case["pads"]
        r = case["hv"] // case["hk"]
        q, k, v, g = (x[:n] for x in f)
        q, k = q.repeat_interleave(r, 1), k.repeat_interleave(r, 1)
        new = g.exp()[..., None, None] * s["state"][s["idx"][:n]] + k[..., None] * v[..., None, :]
        s["state"][s["idx"][:n]] = new
        s["o"][:n] = (scale * (q[..., None] * new).sum(-2)).to(bf)
        return [s["o"], s["state"]]
    if op == "linear_fwd":
        s0 = s["state"][s["idx"]] if case["states"] else None
        o, fin = _linear(*f, s["cu"], s0, scale)
        if not case["states"]:
            return [o.to(bf)]
        s["final"][s["idx"]] = fin
        return [o.to(bf), s["final"]]
    with torch.enable_grad():
        leaves = [x.clone().requires_grad_() for x in f]
        if case["states"]:
            leaves.append(s["state"].clone().requires_grad_())
        o, _ = _linear(*leaves[:4], s["cu"], leaves[4] if case["states"] else None, scale)
        grads = torch.autograd.grad(o, leaves, s["do"].float())
    return [x.to(bf) for x in grads[:3]] + list(grads[3:])


def _own(s):
    import depthwise_causal_short_gb300 as cc
    case = s["case"]
    op = case["op"]
    if op.startswith("qknorm"):
        kw = dict(wq=s["wq"], wk=s["wk"], cos=s["cos"], sin=s["sin"], positions=s["positions"],
                  mode=case["mode"], eps=EPS, interleaved=case["interleaved"])
        if op == "qknorm_fwd":
            return list(cc.cattn_qknorm_fwd(s["q"], s["k"], **kw))
        return list(cc.cattn_qknorm_bwd(s["q"], s["k"], s["dyq"], s["dyk"], **kw))
    if op == "linear_update":
        o, _ = cc.cattn_linear_update(s["q"], s["k"], s["v"], s["g"], s["state"], s["idx"],
                                      pad_rows=True, o=s["o"])
        return [o, s["state"]]
    if op == "linear_fwd":
        if not case["states"]:
            return [cc.cattn_linear_fwd(s["q"], s["k"], s["v"], s["g"], s["cu"])[0]]
        o, fin, _ = cc.cattn_linear_fwd(s["q"], s["k"], s["v"], s["g"], s["cu"],
                                        initial_state=s["state"], final_state=s["final"],
                                        state_indices=s["idx"])
        return [o, fin]
    dq, dk, dv, dg, ds = cc.cattn_linear_bwd(s["q"], s["k"], s["v"], s["g"], s["do"], s["cu"],
                                             initial_state=s["state"])
    return [dq, dk, dv, dg] + ([ds] if case["states"] else [])


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------------------
# the work a pass cannot do without
# ---------------------------------------------------------------------------------------


def work(case):
    op = case["op"]
    if op.startswith("qknorm"):
        rows, n = case["rows"], (case["hq"] + case["hk"]) * case["dim"]
        x = rows * n * 2
        table = min(rows, case["maxpos"]) * case["rot"] * 4 + (rows * 4 if case["rot"] else 0)
        w = {"f32": 8, "bf16": 4, "none": 0}[case["weights"]] * case["dim"]
        if op == "qknorm_fwd":
            return {"bytes": 2 * x + table + w, "flops": 7 * rows * n}
        return {"bytes": 3 * x + table + 2 * w, "flops": 14 * rows * n}
    hk, hv, kd, vd = (case[n] for n in ("hk", "hv", "kd", "vd"))
    state = hv * kd * vd * 4
    if op == "linear_update":
        n = case["rows"] - case["pads"]
        row = 2 * hk * kd * 2 + 2 * hv * vd * 2 + hv * 4
        return {"bytes": n * (2 * state + row) + case["rows"] * 4, "flops": 5 * n * hv * kd * vd}
    t, n = case["total"], case["nseq"]
    qk, v, g = t * hk * kd * 2, t * hv * vd * 2, t * hv * 4
    if op == "linear_fwd":
        # the recurrence: a product into the state and one out of it for each token and head
        return {"bytes": 2 * qk + 2 * v + g + (2 * n * state if case["states"] else 0) + 4 * (n + 1),
                "flops": 4 * t * hv * kd * vd}
    # its gradient: the state again, its gradient, and the products that give dq, dk and dv
    return {"bytes": 4 * qk + 3 * v + 2 * g + (2 * n * state if case["states"] else 0) + 4 * (n + 1),
            "flops": 10 * t * hv * kd * vd}


# ---------------------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------------------


def _exact_norm(s, case):
    dim, rot = case["dim"], case["rot"]
    outs, grads = [], []
    for side in "qk":
        x = s[side].double()
        rows, heads, _ = x.shape
        w = torch.ones(dim, device=x.device, dtype=torch.float64) if s["w" + side] is None else s["w" + side].double()
        # the rotation as one matrix for each row: y = R u
        R = torch.eye(dim, device=x.device, dtype=torch.float64).repeat(rows, 1, 1)
        for p in range(rot // 2):
            i, j = (2 * p, 2 * p + 1) if case["interleaved"] else (p, p + rot // 2)
            c, sn = (s[n].double()[s["positions"].long(), p] for n in ("cos", "sin"))
            R[:, i, i], R[:, i, j], R[:, j, i], R[:, j, j] = c, -sn, sn, c
        size = float(dim) if case["mode"] == "rms" else 1.0
        r = 1.0 / torch.sqrt((x * x).sum(-1) / size + EPS)
        if case["op"] == "qknorm_fwd":
            outs.append(torch.einsum("tij,thj->thi", R, x * r[..., None] * w))
            continue
        du = torch.einsum("tij,thi->thj", R, s["dy" + side].double())
        # dx_j = r w_j du_j - r^3 x_j / size * sum_i du_i w_i x_i
        dx = r[..., None] * w * du - (r ** 3 / size * (du * w * x).sum(-1))[..., None] * x
        outs.append(dx)
        grads.append(None if s["w" + side] is None else torch.einsum("thi,thi,th->i", du, x, r))
    return outs + grads


def _exact_update(s, case):
    n, hv, r = case["rows"] - case["pads"], case["hv"], case["hv"] // case["hk"]
    o, state = s["o"].double(), s["state"].double()
    for h in range(hv):
        at = s["idx"][:n].long()
        q, k = s["q"][:n, h // r].double(), s["k"][:n, h // r].double()
        new = state[at, h] * torch.exp(s["g"][:n, h].double())[:, None, None]
        new = new + torch.einsum("nk,nv->nkv", k, s["v"][:n, h].double())
        state[at, h] = new
        o[:n, h] = torch.einsum("nk,nkv->nv", q, new) / math.sqrt(case["kd"])
    return [o, state]


def _exact_linear(s, case):
    lens, hk, hv = _lengths(case), case["hk"], case["hv"]
    cost = sum(n * n for n in lens) * hv * (case["kd"] + case["vd"]) * (4 if case["op"] == "linear_fwd" else 8)
    if cost > 1.5e13:
        return None
    r, scale = hv // hk, case["kd"] ** -0.5
    q, k, v = (s[n].double() for n in "qkv")
    bwd = case["op"] == "linear_bwd"
    if bwd:
        do = s["do"].double()
        dq, dk, dv, dg = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v), torch.zeros_like(s["g"], dtype=torch.float64)
        ds = torch.zeros_like(s["state"], dtype=torch.float64) if case["states"] else None
    else:
        o = torch.zeros_like(v)
        fin = s["final"].double() if case["states"] else None
    a = 0
    for i, n in enumerate(lens):
        b = a + n
        at = None
        if case["states"]:
            at = i if s["idx"] is None else int(s["idx"][i])
        for h in range(hv):
            G = s["g"][a:b, h].double().cumsum(0)
            L = torch.exp((G[:, None] - G[None, :]).tril()).tril()
            E = torch.exp(G)[:, None]
            Q, K, V = q[a:b, h // r], k[a:b, h // r], v[a:b, h]
            S0 = None if at is None else s["state"][at, h].double()
            W = Q @ K.T * L
            if not bwd:
                y = W @ V
                if S0 is not None:
                    y = y + E * (Q @ S0)
                    if n:
                        fin[at, h] = torch.exp(G[-1]) * S0 + (K * torch.exp(G[-1] - G)[:, None]).T @ V
                    else:
                        fin[at, h] = S0
                o[a:b, h] = scale * y
                continue
            D = do[a:b, h]
            U = D @ V.T
            dv[a:b, h] = scale * (W.T @ D)
            W = W * U  # what each pair of tokens adds to the loss's change
            dg_t = W.sum(1) - W.sum(0)
            U = U * L
            dq[a:b, h // r] += scale * (U @ K)
            dk[a:b, h // r] += scale * (U.T @ Q)
            if S0 is not None:
                dq[a:b, h // r] += scale * E * (D @ S0.T)
                dg_t = dg_t + E[:, 0] * ((Q @ S0) * D).sum(1)
                ds[at, h] = scale * ((Q * E).T @ D)
            dg[a:b, h] = scale * dg_t.flip(0).cumsum(0).flip(0)
        a = b
    if bwd:
        return [dq, dk, dv, dg] + ([ds] if case["states"] else [])
    return [o] + ([fin] if case["states"] else [])


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("qknorm"):
        if case["rows"] * case["dim"] ** 2 > 4e8:
            half = case["rows"] // 2  # rows are independent but for the weights' sums: halves
            parts = []
            for lo, hi in ((0, half), (half, case["rows"])):
                t = {n: (x[lo:hi] if n in ("q", "k", "dyq", "dyk", "positions") and x is not None else x)
                     for n, x in s.items()}
                parts.append(_exact_norm(t, dict(case, rows=hi - lo)))
            return [torch.cat(p) if i < 2 else (None if p[0] is None else p[0] + p[1])
                    for i, p in enumerate(zip(*parts))]
        return _exact_norm(s, case)
    if case["op"] == "linear_update":
        return _exact_update(s, case)
    return _exact_linear(s, case)
