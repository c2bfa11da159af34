"""Measured cases of the mixer operators around the gated delta rule.

Operators, each through the package's public calls:

  delta_fwd / delta_bwd     the gated delta rule over packed sequences (prompts and training), a
                            decay and a step size for each token and value head, and its gradient
  delta_update              its recurrent form for single tokens, on a pooled fp32 state
  norm_fwd / norm_bwd       layer norm (or the norm by the root mean square) of a row or of each
                            head, with weight, bias and the gate silu(z) that such a mixer puts
                            on its outputs, and its gradient with the sums for weight and bias

    S_t = e^{g_t} S_{t-1} + k_t u_t^T,   u_t = beta_t (v_t - (e^{g_t} S_{t-1})^T k_t)
    o_t = scale q_t^T S_t
    y = ((x - mean) / sqrt(var + eps) * w + b) * silu(z)

A case names the call and its sizes.  `run` computes the plain form (elementary torch
operations in fp32) or, with `own`, makes the package's calls; `exact` is the definition in
64 bits.

Sizes: rows and head counts of the package's q/k/v workload (16384 rows; q and k of 1024
channels as 8 heads of 128, v of 2048 as 16 heads of 128), its decode pool (512 slots, 256
rows), its ragged shape (4 x 777 rows), its rows of 4096 channels and a 64-row call, with odd
ones in between.
"""
import math
import random

import torch

own = False

# ---------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------


def _delta_case(op, total, nseq, hk, hv, kd, vd, states, slots, mix):
    # states: initial and final states in pool slots (forward), an initial state and its
    # gradient (backward).  mix: which mixture of lengths.
    return {"op": op, "total": total, "nseq": nseq, "hk": hk, "hv": hv, "kd": kd, "vd": vd,
            "states": states, "slots": slots, "mix": mix}


def _update_case(rows, pads, slots, hk, hv, kd, vd):
    return {"op": "delta_update", "rows": rows, "pads": pads, "slots": slots, "hk": hk, "hv": hv,
            "kd": kd, "vd": vd}


def _norm_case(op, rows, heads, dim, mode, weights, bias, gate):
    return {"op": op, "rows": rows, "heads": heads, "dim": dim, "mode": mode, "weights": weights,
            "bias": bias, "gate": gate}


def listed():
    return [
        # the shortest prompt of one sequence: latency
        dict(_delta_case("delta_fwd", 64, 1, 8, 8, 128, 128, False, 0, 0), name="delta_short"),
        # a serving prefill: 16 sequences of mixed lengths, states read from and written to a pool
        dict(_delta_case("delta_fwd", 16384, 16, 8, 16, 128, 128, True, 64, 1), name="delta_prefill"),
        # a training batch of two long rows, v with twice the heads of q and k
        dict(_delta_case("delta_fwd", 16384, 2, 8, 16, 128, 128, False, 0, 0), name="delta_train_fwd"),
        # a small ragged batch with other head widths
        dict(_delta_case("delta_fwd", 3108, 7, 4, 4, 64, 96, True, 9, 2), name="delta_ragged"),
        # the gradient of the training batch
        dict(_delta_case("delta_bwd", 16384, 2, 8, 16, 128, 128, False, 0, 0), name="delta_train_bwd"),
        # the gradient of a ragged batch with initial states
        dict(_delta_case("delta_bwd", 3108, 7, 4, 4, 64, 96, True, 7, 2), name="delta_ragged_bwd"),
        # one token of one sequence
        dict(_update_case(1, 0, 8, 8, 16, 128, 128), name="delta_step1"),
        # a full decode batch out of a pool of 512 slots, a few of its rows padding
        dict(_update_case(256, 5, 512, 8, 16, 128, 128), name="delta_step256"),
        # the gated norm of the mixer's outputs in a decode step of a small batch: latency
        dict(_norm_case("norm_fwd", 4, 16, 128, "rms", "f32", False, True), name="norm_decode4"),
        # the same for a whole training batch, and its gradient
        dict(_norm_case("norm_fwd", 16384, 16, 128, "rms", "f32", False, True), name="norm_train"),
        dict(_norm_case("norm_bwd", 16384, 16, 128, "rms", "f32", False, True), name="norm_train_bwd"),
        # the gradient of the layer norm of whole rows ahead of a mixer, bf16 weight and bias
        dict(_norm_case("norm_bwd", 8192, 1, 4096, "layer", "bf16", True, False), name="norm_rows_bwd"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["delta_fwd", "delta_bwd", "delta_update", "norm_fwd", "norm_bwd"])
    if op.startswith("norm"):
        dim = 8 * _log(rng, 1, 1024)
        heads = rng.choice([1, 1, 2, 3, 5, 8, 16, 32]) if dim <= 512 else 1
        rows = _log(rng, 1, min(16384, 16384 * 2048 // (heads * dim)))
        weights = rng.choice(["f32", "bf16", "none"])
        return _norm_case(op, rows, heads, dim, rng.choice(["layer", "rms"]), weights,
                          weights != "none" and rng.choice([False, True]), rng.choice([False, True]))
    while True:
        hk, r = rng.choice([1, 2, 3, 4, 6, 8]), rng.choice([1, 1, 2, 3, 4])
        kd, vd = rng.choice([32, 40, 64, 96, 128]), rng.choice([32, 56, 64, 96, 128, 256])
        hv = hk * r
        if hk * kd <= 1024 and hv * vd <= 2048 and hv <= 16:
            break
    if op == "delta_update":
        rows = _log(rng, 1, max(1, min(256, 256 * 16 * 128 * 128 // (hv * kd * vd))))
        return _update_case(rows, rng.randint(0, rows // 8), rows + rng.randint(0, rows), hk, hv, kd, vd)
    total = _log(rng, 1, 16384)
    nseq = _log(rng, 1, min(64, total))
    states = rng.choice([False, True])
    return _delta_case(op, total, nseq, hk, hv, kd, vd, states,
                       (nseq + rng.randint(0, 4) if op == "delta_fwd" else nseq) if states else 0,
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

    def bf(x):
        return x.to(torch.bfloat16)

    s = {"case": case}
    if case["op"].startswith("norm"):
        rows, heads, dim = case["rows"], case["heads"], case["dim"]
        # rows with a mean of their own and channels of different sizes, as residual streams have
        x = randn(rows, heads, dim)
        s["x"] = bf(x * torch.exp(0.5 * randn(dim)) + 0.5 * randn(rows, heads, 1) + 0.2 * randn(dim))
        s["z"] = bf(randn(rows, heads, dim)) if case["gate"] else None
        wt = {"f32": torch.float32, "bf16": torch.bfloat16, "none": None}[case["weights"]]
        s["w"] = None if wt is None else (1 + 0.2 * randn(dim)).to(wt)
        s["b"] = (0.2 * randn(dim)).to(wt) if case["bias"] else None
        if case["op"] == "norm_bwd":
            s["dy"] = bf(randn(rows, heads, dim))
        return s

    hk, hv, kd, vd = (case[n] for n in ("hk", "hv", "kd", "vd"))
    rows = case["rows"] if case["op"] == "delta_update" else case["total"]
    silu, norm = torch.nn.functional.silu, torch.nn.functional.normalize
    # q, k, v: the convolution's outputs (SiLU of roughly normal values), q and k normalised, so
    # that the keys of different tokens are not orthogonal
    s["q"] = bf(norm(silu(randn(rows, hk, kd)), dim=-1) * kd ** 0.5)
    s["k"] = bf(norm(silu(randn(rows, hk, kd)), dim=-1))
    s["v"] = bf(silu(randn(rows, hv, vd)))
    # log decays: heads remember from a few tokens to a few thousand, each token moves it
    reach = torch.exp(torch.linspace(0.0, -math.log(2048.0), hv, device=dev)) if hv > 1 else \
        torch.full((1,), 1 / 64, device=dev)
    s["g"] = -reach * torch.nn.functional.softplus(randn(rows, hv))
    s["beta"] = torch.sigmoid(randn(rows, hv))
    if case["op"] == "delta_update":
        n, slots, pads = rows, case["slots"], case["pads"]
        s["state"] = randn(slots, hv, kd, vd)
        idx = torch.randperm(slots, generator=gen, device=dev)[:n].to(torch.int32)
        idx[n - pads:] = -1  # a padded batch: its last rows name no slot
        s["idx"] = idx
        s["o"] = torch.zeros(n, hv, vd, dtype=torch.bfloat16, device=dev)
        return s
    s["lens"] = _lengths(case)
    cu = [0]
    for n in s["lens"]:
        cu.append(cu[-1] + n)
    s["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
    s["idx"] = s["state"] = None
    if case["states"]:
        s["state"] = randn(case["slots"], hv, kd, vd)
        if case["op"] == "delta_fwd":
            s["idx"] = torch.randperm(case["slots"], generator=gen,
                                      device=dev)[:case["nseq"]].to(torch.int32)
            s["final"] = torch.zeros_like(s["state"])
    if case["op"] == "delta_bwd":
        s["do"] = bf(randn(rows, hv, vd))
    return s


# ---------------------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------------------

CHUNK = 64
EPS = 1e-6


def _pairs(x):
    """T[..., i, j] = sum of x[..., m] over j < m <= i, and zero for j >= i; sums of one sign
    never cancel here, unlike differences of one running sum."""
    n = x.shape[-1]
    low = torch.ones(n, n, dtype=torch.bool, device=x.device).tril(-1)
    return (x[..., :, None] * low).cumsum(-2)


def _inverse(a):
    """(1 + a)^-1 for strictly lower triangular a [..., CHUNK, CHUNK]: blocks of twice the size
    from blocks, 1 / [[A, 0], [B, C]] = [[1/A, 0], [-1/C B 1/A, 1/C]]."""
    i = torch.arange(CHUNK, device=a.device)
    t = torch.eye(CHUNK, device=a.device, dtype=a.dtype).expand_as(a)
    size = 1
    while size < CHUNK:
        off = (i[:, None] // (2 * size) == i[None, :] // (2 * size)) & (i[:, None] // size > i[None, :] // size)
        t = t - t @ (a * off) @ t
        size *= 2
    return t


def _delta(q, k, v, g, beta, lens, s0, scale):
    """o [total, hv, vd] and the final states, in chunks of CHUNK tokens; all fp32."""
    total, r, C, dev = q.shape[0], v.shape[1] // q.shape[1], CHUNK, q.device
    n = [-(-m // C) for m in lens]
    starts = [sum(lens[:i]) for i in range(len(lens))]
    # sequences by falling length: those that still run at a chunk position are the first ones
    order = sorted(range(len(lens)), key=lambda i: -n[i])
    at = [(i, j) for j in range(max(n)) for i in order if n[i] > j]
    row = torch.tensor([[starts[i] + j * C, starts[i] + lens[i]] for i, j in at], device=dev)
    row, end = row[:, :1] + torch.arange(C, device=dev), row[:, 1:]
    ok = row < end

    def cut(x):  # [total, h, ...] -> [chunks, h, C, ...], zeros in rows that are no token
        y = x[torch.where(ok, row, 0)]
        return torch.where(ok.view(*ok.shape, *[1] * (y.dim() - 2)), y, 0.0).transpose(1, 2)

    qc, kc = (cut(x).repeat_interleave(r, 1) for x in (q, k))
    vc, gc, bc = cut(v), cut(g), cut(beta)
    t = _pairs(gc)
    decay = t.exp().tril()
    front = gc.cumsum(-1).exp()[..., None]  # from before the chunk to each token
    back = t[..., -1, :, None].exp()        # from each token to the chunk's end
    inv = _inverse((kc @ kc.transpose(-1, -2) * decay * bc[..., None]).tril(-1)) * bc[..., None, :]
    u0, w = inv @ vc, inv @ (kc * front)
    kb = (kc * back).transpose(-1, -2)
    whole = gc.sum(-1).exp()[..., None, None]
    state = torch.zeros(len(lens), v.shape[1], q.shape[2], v.shape[2], device=dev) if s0 is None else s0
    state = state[torch.tensor(order, device=dev)]
    us, states, fin, a = [], [], [], 0
    for j in range(max(n)):
        m = sum(x > j for x in n)
        fin.append(state[m:])
        state = state[:m]
        b = a + m
        u = u0[a:b] - w[a:b] @ state
        us.append(u)
        states.append(state)
        state = whole[a:b] * state + kb[a:b] @ u
        a = b
    fin.append(state)
    u, s_in = torch.cat(us), torch.cat(states)
    o = (qc @ kc.transpose(-1, -2) * decay) @ u + (qc * front) @ s_in
    out = torch.zeros(total + 1, v.shape[1], v.shape[2], device=dev)
    out = out.index_put((torch.where(ok, row, total),), scale * o.transpose(1, 2))[:total]
    back_to = sorted(range(len(order)), key=lambda i: order[i])
    return out, torch.cat(fin[::-1])[torch.tensor(back_to, device=dev)]


def _norm_parts(s):
    case = s["case"]
    x = s["x"].float()
    if case["mode"] == "layer":
        x = x - x.mean(-1, keepdim=True)
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    n = x * r
    u = n if s["w"] is None else n * s["w"].float()
    if s["b"] is not None:
        u = u + s["b"].float()
    return n, r, u


def _norm_plain(s):
    case = s["case"]
    bf = torch.bfloat16
    n, r, u = _norm_parts(s)
    if case["op"] == "norm_fwd":
        if s["z"] is not None:
            z = s["z"].float()
            u = u * z * torch.sigmoid(z)
        return [u.to(bf)]
    du, dz = s["dy"].float(), None
    if s["z"] is not None:
        z = s["z"].float()
        sg = torch.sigmoid(z)
        dz = (du * u * sg * (1 + z * (1 - sg))).to(bf)
        du = du * z * sg
    dw = None if s["w"] is None else (du * n).sum((0, 1)).to(s["w"].dtype)
    db = None if s["b"] is None else du.sum((0, 1)).to(s["b"].dtype)
    dn = du if s["w"] is None else du * s["w"].float()
    dx = dn - n * (dn * n).mean(-1, keepdim=True)
    if case["mode"] == "layer":
        dx = dx - dn.mean(-1, keepdim=True)
    return [(r * dx).to(bf), dw, db, dz]


def _plain(s):
    case = s["case"]
    op = case["op"]
    bf = torch.bfloat16
    if op.startswith("norm"):
        return _norm_plain(s)
    scale = case["kd"] ** -0.5
    f = [s[n].float() for n in ("q", "k", "v", "g", "beta")]
    if op == "delta_update":
        n = case["rows"] - case["pads"]
        r = case["hv"] // case["hk"]
        q, k, v, g, beta = (x[:n] for x in f)
        q, k = q.repeat_interleave(r, 1), k.repeat_interleave(r, 1)
        old = g.exp()[..., None, None] * s["state"][s["idx"][:n]]
        u = beta[..., None] * (v - (k[..., None] * old).sum(-2))
        new = old + k[..., None] * u[..., None, :]
        s["state"][s["idx"][:n]] = new
        s["o"][:n] = (scale * (q[..., None] * new).sum(-2)).to(bf)
        return [s["o"], s["state"]]
    if op == "delta_fwd":
        s0 = s["state"][s["idx"]] if case["states"] else None
        o, fin = _delta(*f, s["lens"], s0, scale)
        if not case["states"]:
            return [o.to(bf)]
        s["final"][s["idx"]] = fin
        return [o.to(bf), s["final"]]
    with torch.enable_grad():
        leaves = [x.clone().requires_grad_() for x in f]
        if case["states"]:
            leaves.append(s["state"].clone().requires_grad_())
        o, _ = _delta(*leaves[:5], s["lens"], leaves[5] if case["states"] else None, scale)
        grads = torch.autograd.grad(o, leaves, s["do"].float())
    return [x.to(bf) for x in grads[:3]] + list(grads[3:])


def _own(s):
    import depthwise_causal_short_gb300 as cc
    case = s["case"]
    op = case["op"]
    if op.startswith("norm"):
        kw = dict(gate=s["z"], mode=case["mode"], eps=EPS)
        if op == "norm_fwd":
            return [cc.cattn_layernorm_fwd(s["x"], s["w"], s["b"], **kw)]
        return list(cc.cattn_layernorm_bwd(s["x"], s["dy"], s["w"], s["b"], **kw))
    args = [s[n] for n in ("q", "k", "v", "g", "beta")]
    if op == "delta_update":
        o, _ = cc.cattn_delta_update(*args, s["state"], s["idx"], pad_rows=True, o=s["o"])
        return [o, s["state"]]
    if op == "delta_fwd":
        if not case["states"]:
            return [cc.cattn_delta_fwd(*args, s["cu"])[0]]
        o, fin, _ = cc.cattn_delta_fwd(*args, s["cu"], initial_state=s["state"],
                                       final_state=s["final"], state_indices=s["idx"])
        return [o, fin]
    grads = cc.cattn_delta_bwd(*args, s["do"], s["cu"], initial_state=s["state"])
    return list(grads) if case["states"] else list(grads[:5])


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------------------
# the work a pass cannot do without
# ---------------------------------------------------------------------------------------


def work(case):
    op = case["op"]
    if op.startswith("norm"):
        n = case["rows"] * case["heads"] * case["dim"]
        w = {"f32": 4, "bf16": 2, "none": 0}[case["weights"]] * case["dim"] * (2 if case["bias"] else 1)
        if op == "norm_fwd":
            return {"bytes": n * 2 * (3 if case["gate"] else 2) + w, "flops": n * (12 if case["gate"] else 7)}
        return {"bytes": n * 2 * (5 if case["gate"] else 3) + 2 * w, "flops": n * (28 if case["gate"] else 16)}
    hk, hv, kd, vd = (case[n] for n in ("hk", "hv", "kd", "vd"))
    state = hv * kd * vd * 4
    if op == "delta_update":
        n = case["rows"] - case["pads"]
        row = 2 * hk * kd * 2 + 2 * hv * vd * 2 + 2 * hv * 4
        return {"bytes": n * (2 * state + row) + case["rows"] * 4, "flops": 7 * n * hv * kd * vd}
    t, n = case["total"], case["nseq"]
    qk, v, g = t * hk * kd * 2, t * hv * vd * 2, 2 * t * hv * 4
    if op == "delta_fwd":
        # the recurrence: a product out of the state and one into it for u, and one for o
        return {"bytes": 2 * qk + 2 * v + g + (2 * n * state if case["states"] else 0) + 4 * (n + 1),
                "flops": 6 * t * hv * kd * vd}
    # its gradient: the state again, its gradient, and the products that give dq, dk and dv
    return {"bytes": 4 * qk + 3 * v + 2 * g + (2 * n * state if case["states"] else 0) + 4 * (n + 1),
            "flops": 16 * t * hv * kd * vd}


# ---------------------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------------------


def _exact_norm(s):
    x, w, b, z, dy = (None if s.get(n) is None else s[n].double() for n in ("x", "w", "b", "z", "dy"))
    names = [(n, t) for n, t in (("x", x), ("w", w), ("b", b), ("z", z)) if t is not None]
    with torch.enable_grad():
        for _, t in names:
            t.requires_grad_()
        mean = x.sum(-1, keepdim=True) / x.shape[-1] if s["case"]["mode"] == "layer" else 0.0
        var = ((x - mean) ** 2).sum(-1, keepdim=True) / x.shape[-1]
        y = (x - mean) / torch.sqrt(var + EPS)
        y = y if w is None else y * w
        y = y if b is None else y + b
        y = y if z is None else y * (z / (1 + torch.exp(-z)))
        if dy is None:
            return [y.detach()]
        got = dict(zip((n for n, _ in names), torch.autograd.grad(y, [t for _, t in names], dy)))
    return [got.get(n) for n in ("x", "w", "b", "z")]


def _exact_update(s, case):
    n, hv, r = case["rows"] - case["pads"], case["hv"], case["hv"] // case["hk"]
    o, state = s["o"].double(), s["state"].double()
    at = s["idx"][:n].long()
    for h in range(hv):
        q, k = s["q"][:n, h // r].double(), s["k"][:n, h // r].double()
        old = state[at, h] * torch.exp(s["g"][:n, h].double())[:, None, None]
        miss = s["v"][:n, h].double() - torch.einsum("nk,nkv->nv", k, old)
        new = old + torch.einsum("nk,nv->nkv", k, miss * s["beta"][:n, h].double()[:, None])
        state[at, h] = new
        o[:n, h] = torch.einsum("nk,nkv->nv", q, new) / math.sqrt(case["kd"])
    return [o, state]


class _Steps:
    """The recurrence token by token, all sequences and heads at once.  Row t of the padded arrays
    holds token t of each sequence, the longest sequence first; the ones that still run are the
    first `live[t]`."""

    def __init__(self, s, case):
        lens = s["lens"]
        self.order = sorted(range(len(lens)), key=lambda i: -lens[i])
        self.lens, self.most = [lens[i] for i in self.order], max(lens)
        cu = s["cu"].tolist()
        dev = s["q"].device
        self.rows = torch.full((self.most, len(lens)), -1, device=dev)
        for j, i in enumerate(self.order):
            self.rows[:lens[i], j] = torch.arange(cu[i], cu[i + 1], device=dev)
        self.live = [sum(n > t for n in self.lens) for t in range(self.most)]
        r, hv = case["hv"] // case["hk"], case["hv"]
        f = {n: s[n].double() for n in ("q", "k", "v", "g", "beta", "do") if n in s}
        for n in ("q", "k"):
            f[n] = f[n].repeat_interleave(r, 1)
        f["q"] = f["q"] / math.sqrt(case["kd"])
        f["a"] = torch.exp(f["g"])
        self.f = f
        shape = (len(lens), hv, case["kd"], case["vd"])
        if case["states"]:
            slot = list(range(len(lens))) if s["idx"] is None else s["idx"].tolist()
            self.slots = torch.tensor([slot[i] for i in self.order], device=dev)
            self.first = s["state"].double()[self.slots]
        else:
            self.first = torch.zeros(shape, dtype=torch.float64, device=dev)

    def at(self, t):
        rows = self.rows[t, :self.live[t]]
        return rows, {n: x[rows] for n, x in self.f.items()}

    def step(self, state, x):
        """In place on the live part of the states; the decayed state, the miss and u."""
        old = state * x["a"][..., None, None]
        miss = x["v"] - torch.matmul(x["k"][..., None, :], old)[..., 0, :]
        u = miss * x["beta"][..., None]
        state.copy_(old).add_(x["k"][..., None] * u[..., None, :])
        return old, miss, u


SEGMENT = 128


def _exact_fwd(s, case):
    p = _Steps(s, case)
    o, state = p.f["v"].clone(), p.first.clone()
    for t in range(p.most):
        rows, x = p.at(t)
        live = state[:len(rows)]
        p.step(live, x)
        o[rows] = torch.matmul(x["q"][..., None, :], live)[..., 0, :]
    if not case["states"]:
        return [o]
    fin = s["final"].double()
    fin[p.slots] = state
    return [o, fin]


def _exact_bwd(s, case):
    p = _Steps(s, case)
    f = p.f
    dq, dk, dv, dg, db = (torch.zeros_like(f[n]) for n in ("q", "k", "v", "g", "beta"))
    state, kept = p.first.clone(), []
    for t in range(p.most):
        if t % SEGMENT == 0:
            kept.append(state[:p.live[t]].clone())
        rows, x = p.at(t)
        p.step(state[:len(rows)], x)
    D = torch.zeros_like(p.first)
    for c in reversed(range(len(kept))):
        run, before = kept.pop(), []
        for t in range(c * SEGMENT, min(p.most, (c + 1) * SEGMENT)):
            rows, x = p.at(t)
            run = run[:len(rows)].clone()
            before.append((rows, x, *p.step(run, x), run))
        while before:
            rows, x, old, miss, u, new = before.pop()
            d = D[:len(rows)]
            d += x["q"][..., None] * x["do"][..., None, :]
            dq[rows] = torch.matmul(new, x["do"][..., None])[..., 0]
            du = torch.matmul(x["k"][..., None, :], d)[..., 0, :]
            db[rows] = (du * miss).sum(-1)
            dz = du * x["beta"][..., None]
            dv[rows] = dz
            dk[rows] = torch.matmul(d, u[..., None])[..., 0] - torch.matmul(old, dz[..., None])[..., 0]
            d -= x["k"][..., None] * dz[..., None, :]
            dg[rows] = (d * old).sum((-1, -2))
            d *= x["a"][..., None, None]
    total, hk, r = dq.shape[0], case["hk"], case["hv"] // case["hk"]
    dq = dq.view(total, hk, r, -1).sum(2) / math.sqrt(case["kd"])
    dk = dk.view(total, hk, r, -1).sum(2)
    grads = [dq, dk, dv, dg, db]
    if case["states"]:
        ds = torch.zeros_like(D)
        ds[p.slots] = D
        grads.append(ds)
    return grads


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("norm"):
        return _exact_norm(s)
    if case["op"] == "delta_update":
        return _exact_update(s, case)
    return _exact_fwd(s, case) if case["op"] == "delta_fwd" else _exact_bwd(s, case)
