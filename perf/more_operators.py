"""Timed cases of the layer norm, of tokens sorted by expert and back, and of the matrix product with its epilogue.

Kinds of case (``kind``):

* ``ln``            s = x + residual; y = (s - mean(s)) / sqrt(var(s) + eps) * weight + bias; returns y and s;
* ``ln_bwd``        its gradients from the stored s, dy and the gradient ds that reaches s by the residual path: dx
                    (the residual's gradient too), dweight, dbias;
* ``dispatch``      from idx [T, k], the experts that each token picked (-1: a pick that was dropped): the picks' counts
                    and offsets per expert, the token of every sorted row (perm), the row of every pick (slot, -1 for
                    dropped ones), and the rows themselves, rows[slot[t, j]] = x[t].  Sorted by expert, then token,
                    then pick; entries of perm and rows past the last row stay as they were;
* ``dispatch_bwd``  dx[t] = sum_j drows[slot[t, j]] + add[t];
* ``combine``       y[t] = sum_j w[t, j] rows[slot[t, j]] + add[t];
* ``combine_bwd``   its gradients: drows[slot[t, j]] = w[t, j] dy[t], dw[t, j] = dy[t] . rows[slot[t, j]];
* ``linear``        pre = x weight^T + bias; y = act(pre) + residual; returns y, and pre where it is saved;
* ``linear_bwd``    its gradients from x, the saved pre and dy: dx, dweight, dbias.
"""
import math

import torch

own = False

EPS = 1e-5


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one generated token: the norm between two layers, all latency
        dict(name="ln_one_token", kind="ln", T=1, d=2048, x="bf16", res="bf16", out="bf16"),
        # odd row count and width, residual stream kept in fp32
        dict(name="ln_odd_f32_stream", kind="ln", T=6007, d=2501, x="bf16", res="f32", out="bf16"),
        # the norm of a training step over one batch
        dict(name="ln_training_backward", kind="ln_bwd", T=16384, d=4096, x="bf16"),
        # a decode batch on its way to the experts: launches and latency
        dict(name="dispatch_decode_batch", kind="dispatch", T=16, d=2048, k=8, E=256, x="bf16", rows="bf16", skew=False,
             drop=0.0),
        # a prompt with unevenly loaded experts, its residual stream in fp32
        dict(name="dispatch_prompt_skewed", kind="dispatch", T=4093, d=2048, k=8, E=256, x="f32", rows="bf16", skew=True,
             drop=0.0),
        # the same step's gradient in training
        dict(name="dispatch_training_backward", kind="dispatch_bwd", T=16384, d=2048, k=8, E=256, x="bf16", rows="bf16",
             skew=False, drop=0.0),
        # a prompt's expert outputs back in token order, on top of the residual; some picks went over a capacity
        dict(name="combine_prompt_dropped", kind="combine", T=4096, d=2048, k=8, E=256, x="bf16", rows="bf16", skew=True,
             drop=0.1),
        # its gradient in training
        dict(name="combine_training_backward", kind="combine_bwd", T=16384, d=2048, k=8, E=256, x="bf16", rows="bf16",
             skew=False, drop=0.0),
        # one generated token through a block's second product: reading 67 MB of weights
        dict(name="linear_one_token", kind="linear", T=1, k=8192, n=4096, act="none", bias="bf16", res="bf16", save=False),
        # a ragged prompt: no size is a multiple of a tile
        dict(name="linear_ragged_gelu", kind="linear", T=777, k=1000, n=2744, act="gelu", bias="f32", res=None, save=True),
        # forward of a training step's first product; pre is kept for the backward pass
        dict(name="linear_training_forward", kind="linear", T=8192, k=4096, n=16384, act="gelu", bias="bf16", res=None,
             save=True),
        # backward of a training step's first product
        dict(name="linear_training_backward", kind="linear_bwd", T=4096, k=4096, n=16384, act="gelu", bias="bf16",
             dy="bf16"),
    ]


def _log_size(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], spread over its logarithm."""
    while True:
        v = round(math.exp(rng.uniform(math.log(lo), math.log(hi + step))) / step) * step
        if lo <= v <= hi:
            return v


def draw(rng):
    kind = rng.choice(["ln", "ln_bwd", "dispatch", "dispatch_bwd", "combine", "combine_bwd", "linear", "linear",
                       "linear_bwd"])
    dt = ["bf16", "bf16", "f32"]
    if kind == "ln":
        return dict(kind=kind, T=_log_size(rng, 1, 16384), d=_log_size(rng, 256, 8192, rng.choice([1, 2, 8])),
                    x=rng.choice(dt), res=rng.choice(["bf16", "f32", None]), out=rng.choice(dt))
    if kind == "ln_bwd":
        return dict(kind=kind, T=_log_size(rng, 1, 16384), d=_log_size(rng, 256, 8192, rng.choice([1, 2, 8])),
                    x=rng.choice(dt))
    if kind.startswith("linear"):
        case = dict(kind=kind, T=_log_size(rng, 1, 8192 if kind == "linear" else 4096), k=_log_size(rng, 256, 4096, 8),
                    n=_log_size(rng, 256, 16384, 8), act=rng.choice(["none", "silu", "gelu"]),
                    bias=rng.choice(["bf16", "f32"]))
        if kind == "linear":
            return dict(case, res=rng.choice([None, "bf16", "f32"]), save=case["act"] != "none" and rng.random() < 0.5)
        return dict(case, dy=rng.choice(dt))
    E = rng.choice([8, 16, 60, 64, 128, 256])
    k = rng.choice([1, 2, 4, 6, 8])
    T = _log_size(rng, 1, 16384)
    return dict(kind=kind, T=T, d=_log_size(rng, 256, min(4096, 16384 * 8 * 2048 // (T * k)), rng.choice([1, 8, 8])),
                k=k, E=E, x=rng.choice(dt), rows="bf16" if rng.random() < 0.8 else "f32", skew=rng.random() < 0.5,
                drop=rng.choice([0.0, 0.0, 0.1]))


# ------------------------------------------------------------------ inputs
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _sorted_rows(idx, E):
    """Stable sort of the picks by expert: (counts, offsets, perm, slot)."""
    T, k = idx.shape
    e = idx.flatten().long()
    kept = (e >= 0).nonzero().flatten()
    order = kept[torch.argsort(e[kept], stable=True)]
    counts = torch.bincount(e[kept], minlength=E)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    slot = torch.full_like(e, -1)
    slot[order] = torch.arange(order.numel(), device=e.device)
    return counts.int(), offsets.int(), (order // k).int(), slot.view(T, k).int()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    kind, T = case["kind"], case["T"]

    def normal(*shape, scale=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)

    state = dict(case=dict(case))
    if kind in ("ln", "ln_bwd"):
        d = case["d"]
        state["weight"] = (1 + 0.1 * torch.randn(d, generator=gen, device="cuda")).to(torch.bfloat16)
        state["bias"] = normal(d, scale=0.1)
        # a residual stream: a few channels far larger than the rest, rows that are off centre, some of padding (zeros)
        channel = torch.where(torch.rand(d, generator=gen, device="cuda") < 0.005, 30.0, 1.0)
        live = (torch.rand(T, 1, generator=gen, device="cuda") >= 0.01).float()
        live[0] = 1.0
        s = (torch.randn(T, d, generator=gen, device="cuda") * channel + torch.randn(T, 1, generator=gen, device="cuda")) \
            * live
        if kind == "ln":
            if case["res"] is None:
                state.update(x=s.to(_DT[case["x"]]), res=None)
            else:
                state.update(x=(torch.randn(T, d, generator=gen, device="cuda") * 0.5 * live).to(_DT[case["x"]]),
                             res=s.to(_DT[case["res"]]))
        else:
            dt = _DT[case["x"]]
            state.update(s=s.to(dt), dy=normal(T, d, dtype=dt), ds=normal(T, d, dtype=dt))
        return state
    if kind.startswith("linear"):
        k, n = case["k"], case["n"]
        state["x"] = normal(T, k)
        state["weight"] = normal(n, k, scale=k ** -0.5)
        state["bias"] = normal(n, scale=0.5, dtype=_DT[case["bias"]])
        if kind == "linear":
            state["res"] = None if case["res"] is None else normal(T, n, scale=2.0, dtype=_DT[case["res"]])
        else:
            state["pre"] = None
            if case["act"] != "none":
                state["pre"] = (torch.matmul(state["x"], state["weight"].t()).float() + state["bias"].float()).to(
                    torch.bfloat16)
            state["dy"] = normal(T, n, dtype=_DT[case["dy"]])
        return state
    # each token's k different experts in ascending order, as a router gives them
    d, k, E = case["d"], case["k"], case["E"]
    logits = torch.randn(T, E, generator=gen, device="cuda")
    if case["skew"]:
        logits -= 1.2 * torch.log(torch.arange(1, E + 1, device="cuda").float())
    top, idx = logits.topk(k, dim=1)
    order = idx.argsort(1)
    idx, w = idx.gather(1, order).int(), torch.softmax(top, 1).gather(1, order)
    if case["drop"]:
        idx[torch.rand(T, k, generator=gen, device="cuda") < case["drop"]] = -1
    x_dt, rows_dt = _DT[case["x"]], _DT[case["rows"]]
    if kind == "dispatch":
        state.update(idx=idx, x=normal(T, d, dtype=x_dt), rows=torch.zeros(T * k, d, dtype=rows_dt, device="cuda"),
                     perm=torch.zeros(T * k, dtype=torch.int32, device="cuda"))
        return state
    state.update(slot=_sorted_rows(idx, E)[3].contiguous(), rows=normal(T * k, d, dtype=rows_dt))
    if kind != "dispatch_bwd":
        state["w"] = w.contiguous()
    if kind == "combine_bwd":
        state.update(dy=normal(T, d, dtype=x_dt), drows=torch.zeros(T * k, d, dtype=rows_dt, device="cuda"))
    else:
        state["add"] = normal(T, d, dtype=x_dt)
    return state


# ------------------------------------------------------------------ the plain forms, in 32 bits
def _act(g, act):
    if act == "none":
        return g
    if act == "silu":
        return g / (1 + torch.exp(-g))
    return 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g)))


def _act_grad(g, act):
    if act == "silu":
        p = 1 / (1 + torch.exp(-g))
        return p * (1 + g * (1 - p))
    t = torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g))
    return 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * g * g)


def _plain(state):
    case = state["case"]
    kind, T = case["kind"], case["T"]
    if kind == "ln":
        s = state["x"].float()
        if state["res"] is not None:
            s = s + state["res"].float()
        c = s - s.mean(-1, keepdim=True)
        y = c * torch.rsqrt((c * c).mean(-1, keepdim=True) + EPS) * state["weight"].float() + state["bias"].float()
        return {"y": y.to(_DT[case["out"]]), "s": s.to(state["x" if state["res"] is None else "res"].dtype)}
    if kind == "ln_bwd":
        s, w, dy = state["s"].float(), state["weight"].float(), state["dy"].float()
        c = s - s.mean(-1, keepdim=True)
        r = torch.rsqrt((c * c).mean(-1, keepdim=True) + EPS)
        n = c * r
        g = dy * w
        dx = r * (g - g.mean(-1, keepdim=True) - n * (g * n).mean(-1, keepdim=True)) + state["ds"].float()
        return {"dx": dx.to(state["s"].dtype), "dweight": (dy * n).sum(0).to(state["weight"].dtype),
                "dbias": dy.sum(0).to(state["weight"].dtype)}
    if kind == "linear":
        pre = state["x"].float() @ state["weight"].float().t() + state["bias"].float()
        y = _act(pre, case["act"])
        if state["res"] is not None:
            y = y + state["res"].float()
        out = {"y": y.to(torch.bfloat16 if state["res"] is None else state["res"].dtype)}
        if case["save"]:
            out["pre"] = pre.to(torch.bfloat16)
        return out
    if kind == "linear_bwd":
        dpre = state["dy"].float()
        if case["act"] != "none":
            dpre = dpre * _act_grad(state["pre"].float(), case["act"])
        return {"dx": (dpre @ state["weight"].float()).to(torch.bfloat16),
                "dweight": (dpre.t() @ state["x"].float()).to(torch.bfloat16),
                "dbias": dpre.sum(0).to(state["bias"].dtype)}
    k, E = case["k"], case["E"]
    if kind == "dispatch":
        e = state["idx"].flatten().long()
        hit = e.unsqueeze(1) == torch.arange(E, device=e.device)  # [T k, E]
        before = torch.cumsum(hit.int(), 0) - 1
        counts = hit.sum(0)
        offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
        there = e.clamp(min=0)
        slot = torch.where(e >= 0, offsets[there] + before.gather(1, there.unsqueeze(1)).squeeze(1), -1)
        pick = (e >= 0).nonzero().flatten()
        token = torch.div(pick, k, rounding_mode="floor")
        state["perm"][slot[pick]] = token.int()
        state["rows"][slot[pick]] = state["x"].to(state["rows"].dtype)[token]
        return {"counts": counts.int(), "offsets": offsets.int(), "perm": state["perm"], "slot": slot.view(T, k).int(),
                "rows": state["rows"]}
    slot = state["slot"].long()
    there, kept = slot.clamp(min=0), (slot >= 0).unsqueeze(-1)
    if kind == "combine_bwd":
        dy = state["dy"].float()
        drows, dw = state["drows"], torch.zeros(T, k, device=dy.device)
        for j in range(k):
            t = kept[:, j, 0].nonzero().flatten()
            drows[slot[t, j]] = (state["w"][t, j, None] * dy[t]).to(drows.dtype)
            dw[:, j] = torch.where(kept[:, j, 0], (dy * state["rows"][there[:, j]].float()).sum(-1), 0)
        return {"drows": drows, "dw": dw}
    y = torch.zeros(T, case["d"], device=slot.device)
    for j in range(k):
        v = state["rows"][there[:, j]].float()
        if kind == "combine":
            v = v * state["w"][:, j, None]
        y = y + torch.where(kept[:, j], v, 0)
    y = y + state["add"].float()
    return {"y" if kind == "combine" else "dx": y.to(state["add"].dtype)}


# ------------------------------------------------------------------ the framework's operators
_handles = {}


def _handle(case):
    """The handle that a program keeps for a layer of this shape."""
    import expert_routed_ffn_moe_gb300 as moe

    kind = case["kind"]
    key = ("ln", case["d"]) if kind.startswith("ln") else \
        (kind, case["T"], case["k"], case["n"], case["act"]) if kind.startswith("linear") else ("sort", case["E"], case["k"])
    if key not in _handles:
        if key[0] == "ln":
            _handles[key] = moe.LayerNorm(case["d"], eps=EPS)
        elif key[0] == "sort":
            _handles[key] = moe.TokenDispatch(case["E"], case["k"])
        else:
            _handles[key] = moe.Linear(case["k"], case["n"], max_tokens=case["T"], training=kind == "linear_bwd",
                                       activation={"none": moe.MOE_ACT_NONE, "silu": moe.MOE_ACT_SILU,
                                                   "gelu": moe.MOE_ACT_GELU}[case["act"]])
    return moe, _handles[key]


def _own(state):
    case = state["case"]
    kind = case["kind"]
    moe, op = _handle(case)
    if kind == "ln":
        y, s = op.forward(state["x"], state["res"], state["weight"], state["bias"],
                          y_dtype=moe.MOE_BF16 if case["out"] == "bf16" else moe.MOE_F32)
        return {"y": y, "s": s}
    if kind == "ln_bwd":
        dx, dweight, dbias = op.backward(state["s"], state["weight"], state["dy"], state["ds"])
        return {"dx": dx, "dweight": dweight, "dbias": dbias}
    if kind == "linear":
        y = op.forward(state["x"], state["weight"], state["bias"], state["res"], save=case["save"])
        return {"y": y[0], "pre": y[1]} if case["save"] else {"y": y}
    if kind == "linear_bwd":
        dx, dweight, dbias = op.backward(state["x"], state["pre"], state["weight"], state["bias"], state["dy"])
        return {"dx": dx, "dweight": dweight, "dbias": dbias}
    if kind == "dispatch":
        counts, offsets, perm, slot = op.sort(state["idx"], perm=state["perm"])
        rows = op.dispatch(state["x"], slot, rows=state["rows"])
        return {"counts": counts, "offsets": offsets, "perm": perm, "slot": slot, "rows": rows}
    if kind == "dispatch_bwd":
        return {"dx": op.dispatch_backward(state["rows"], state["slot"], add=state["add"])}
    if kind == "combine":
        return {"y": op.combine(state["rows"], state["slot"], state["w"], add=state["add"])}
    drows, dw = op.combine_backward(state["dy"], state["rows"], state["slot"], state["w"], drows=state["drows"])
    return {"drows": drows, "dw": dw}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ work and exact values
def work(case):
    kind, T = case["kind"], case["T"]
    size = {"bf16": 2, "f32": 4, None: 0}
    if kind == "ln":
        stream = size[case["x"]] if case["res"] is None else 2 * size[case["res"]]  # s, and the residual
        return {"bytes": T * case["d"] * (size[case["x"]] + stream + size[case["out"]]) + 4 * case["d"],
                "flops": 8 * T * case["d"]}
    if kind == "ln_bwd":
        return {"bytes": 4 * T * case["d"] * size[case["x"]] + 6 * case["d"], "flops": 16 * T * case["d"]}
    if kind.startswith("linear"):
        k, n, b = case["k"], case["n"], size[case["bias"]]
        if kind == "linear":
            y = 2 if case["res"] is None else 2 * size[case["res"]]
            return {"bytes": 2 * (T * k + n * k) + T * n * (y + (2 if case["save"] else 0)) + n * b, "flops": 2 * T * n * k}
        pre = 0 if case["act"] == "none" else 2
        return {"bytes": 4 * (T * k + n * k) + T * n * (size[case["dy"]] + pre) + n * b, "flops": 4 * T * n * k}
    rows, d, k = round(T * case["k"] * (1 - case["drop"])), case["d"], case["k"]
    x, r = T * d * size[case["x"]], rows * d * size[case["rows"]]
    if kind == "dispatch":
        return {"bytes": x + r + 4 * (2 * T * k + rows + 2 * case["E"] + 1), "flops": T * k}
    if kind == "combine_bwd":
        return {"bytes": x + 2 * r + 12 * T * k, "flops": 3 * rows * d}
    return {"bytes": 2 * x + r + (8 if kind == "combine" else 4) * T * k, "flops": 2 * rows * d}


def exact(case, seed):
    """From the definitions in 64 bits.  Where an output is rounded to fewer bits its value before that rounding."""
    st = prepare(case, seed)
    D = torch.float64
    kind, T = case["kind"], case["T"]
    if kind == "ln":
        s = st["x"].to(D) if st["res"] is None else st["x"].to(D) + st["res"].to(D)
        var, mean = torch.var_mean(s, dim=-1, correction=0, keepdim=True)
        return {"y": st["bias"].to(D) + st["weight"].to(D) * (s - mean) / (var + EPS).sqrt(), "s": s}
    if kind == "ln_bwd":
        s, w, dy = st["s"].to(D), st["weight"].to(D), st["dy"].to(D)
        var, mean = torch.var_mean(s, dim=-1, correction=0, keepdim=True)
        z = s - mean
        sd = (var + EPS).sqrt()
        g = dy * w
        proj = (g * z).sum(-1, keepdim=True) / case["d"]
        dx = (g - g.sum(-1, keepdim=True) / case["d"]) / sd - z * proj / sd ** 3 + st["ds"].to(D)
        return {"dx": dx, "dweight": (dy * z / sd).sum(0), "dbias": dy.sum(0)}
    if kind.startswith("linear"):
        act = case["act"]

        def phi(g):  # act(g) = g * phi(g): the logistic function of g, or of the tanh form's argument
            if act == "none":
                return torch.ones_like(g)
            return torch.sigmoid(g if act == "silu" else 2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3))

        x, w = st["x"].to(D), st["weight"].to(D)
        if kind == "linear":
            pre = torch.addmm(st["bias"].to(D), x, w.t())
            y = pre * phi(pre)
            out = {"y": y if st["res"] is None else y + st["res"].to(D)}
            if case["save"]:
                out["pre"] = pre
            return out
        dpre = st["dy"].to(D)
        if act != "none":
            g = st["pre"].to(D)
            p = phi(g)
            inner = 1.0 if act == "silu" else 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * g ** 2)
            dpre = dpre * (p + g * p * (1 - p) * inner)
        return {"dx": dpre @ w, "dweight": dpre.t() @ x, "dbias": dpre.sum(0)}
    k = case["k"]
    if kind == "dispatch":
        counts, offsets, perm, slot = _sorted_rows(st["idx"], case["E"])
        n = perm.numel()
        st["perm"][:n] = perm
        rows = st["rows"].to(D)
        rows[:n] = st["x"].to(D)[perm.long()]
        return {"counts": counts, "offsets": offsets, "perm": st["perm"], "slot": slot, "rows": rows}
    # the picks as (token, pick, row) triples
    t, j = (st["slot"] >= 0).nonzero(as_tuple=True)
    row = st["slot"][t, j].long()
    if kind == "combine_bwd":
        drows = st["drows"].to(D)
        dw = torch.zeros(T, k, dtype=D, device=drows.device)
        for part in range(0, t.numel(), 1 << 14):
            p = slice(part, part + (1 << 14))
            dy = st["dy"][t[p]].to(D)
            drows[row[p]] = dy * st["w"][t[p], j[p]].to(D).unsqueeze(1)
            dw[t[p], j[p]] = torch.einsum("nd,nd->n", dy, st["rows"][row[p]].to(D))
        return {"drows": drows, "dw": dw}
    y = st["add"].to(D)
    for part in range(0, t.numel(), 1 << 14):
        p = slice(part, part + (1 << 14))
        v = st["rows"][row[p]].to(D)
        if kind == "combine":
            v = v * st["w"][t[p], j[p]].to(D).unsqueeze(1)
        y.index_add_(0, t[p], v)
    return {"y" if kind == "combine" else "dx": y}
