"""Timed cases of the dense gated feed-forward block and the norm in front of it.

Kinds of case (``kind``):

* ``norm``      s = x + residual; y = s * rsqrt(mean(s^2) + eps) * weight; returns y and s.  ``out`` is y's form:
                "bf16", "f32", or "mx8" (e4m3 codes, one power-of-two scale per 32 columns);
* ``norm_bwd``  the gradients of that norm: from the stored s, dy and the gradient ds that reaches s by the
                residual path, dx (which is also the residual's gradient) and dweight;
* ``ffn``       y = down(act(gate(x)) * up(x)) in bf16; with ``save`` also the pre-activations [gate | up];
* ``ffn_bwd``   its gradients from x, the saved pre-activations and dy: dx, dgate_up, ddown;
* ``ffn_mx8``   the same block on mx8 rows and mx8 weights; act(gate) * up is itself held in mx8 between the two
                products, as the operator defines.

mx8: 32 neighbouring columns share the scale 2^e, e the smallest integer with max|v| <= 448 * 2^e (e >= -127), and
each value is stored as e4m3(v / 2^e), to the nearest, ties to even.  Scales are stored as bytes e + 127 in tiles of
128 rows x 4 groups (512 bytes): byte (row % 32) * 16 + (row / 32 % 4) * 4 + group % 4 of tile
(row / 128, group / 4); the bytes of rows and groups past the matrix are 0.
"""
import math

import torch

own = False

EPS = 1e-6


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one generated token: the norm between two layers' blocks, all latency
        dict(name="norm_one_token", kind="norm", T=1, d=2048, x="bf16", res="bf16", out="bf16"),
        # a prompt whose feed-forward block runs on 8-bit rows
        dict(name="norm_prompt_mx8", kind="norm", T=4096, d=2048, x="bf16", res="bf16", out="mx8"),
        # odd row count and width, residual stream kept in fp32
        dict(name="norm_odd_f32_stream", kind="norm", T=7001, d=1999, x="bf16", res="f32", out="bf16"),
        # the norm of a training step over one batch
        dict(name="norm_training_backward", kind="norm_bwd", T=16384, d=4096, x="bf16"),
        # one generated token through a dense layer's block: reading 100 MB of weights
        dict(name="ffn_one_token", kind="ffn", T=1, d=2048, I=8192, act="silu", save=False),
        # a small batch through a block of the shared expert's size: launches and latency
        dict(name="ffn_small_batch", kind="ffn", T=32, d=2048, I=512, act="silu", save=False),
        # a ragged prompt: no size is a multiple of a tile
        dict(name="ffn_ragged_gelu", kind="ffn", T=777, d=1000, I=2744, act="gelu", save=False),
        # forward of a training step; the pre-activations are kept for the backward pass
        dict(name="ffn_training_forward", kind="ffn", T=8192, d=4096, I=16384, act="silu", save=True),
        # backward of a small ragged micro-batch
        dict(name="ffn_small_backward", kind="ffn_bwd", T=501, d=2048, I=2048, act="gelu"),
        # backward of a training step
        dict(name="ffn_training_backward", kind="ffn_bwd", T=4096, d=4096, I=16384, act="silu"),
        # a decode batch on 8-bit weights: 200 MB of them
        dict(name="ffn_mx8_decode_batch", kind="ffn_mx8", T=9, d=4096, I=16384, act="silu"),
        # a long prompt on 8-bit weights
        dict(name="ffn_mx8_prompt", kind="ffn_mx8", T=8191, d=4096, I=16384, act="silu"),
    ]


def _log_size(rng, lo, hi, step):
    """A multiple of `step` in [lo, hi], spread over its logarithm."""
    while True:
        v = round(math.exp(rng.uniform(math.log(lo), math.log(hi + step))) / step) * step
        if lo <= v <= hi and v != 3072 and 2 * v != 3072:
            return v


def draw(rng):
    kind = rng.choice(["norm", "norm", "norm_bwd", "ffn", "ffn", "ffn_bwd", "ffn_mx8"])
    act = rng.choice(["silu", "gelu"])
    if kind == "norm":
        out = rng.choice(["bf16", "f32", "mx8"])
        d = _log_size(rng, 256, 8192, 32 if out == "mx8" else rng.choice([1, 8]))
        return dict(kind=kind, T=_log_size(rng, 1, 16384, 1), d=d, x=rng.choice(["bf16", "bf16", "f32"]), res=rng.choice(["bf16", "f32"]), out=out)
    if kind == "norm_bwd":
        return dict(kind=kind, T=_log_size(rng, 1, 16384, 1), d=_log_size(rng, 256, 8192, rng.choice([1, 8])),
                    x=rng.choice(["bf16", "f32"]))
    step = 32 if kind == "ffn_mx8" else 8
    case = dict(kind=kind, T=_log_size(rng, 1, 4096 if kind == "ffn_bwd" else 8192, 1),
                d=_log_size(rng, 256, 4096, step), I=_log_size(rng, 256, 16384, step), act=act)
    if kind == "ffn":
        case["save"] = rng.random() < 0.5
    return case


# ------------------------------------------------------------------ inputs
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _tile_scales(e):
    """Scale bytes [rows, groups] -> the stored tiles, padded with 0."""
    r, g = e.shape
    p = torch.zeros((r + 127) // 128 * 128, (g + 3) // 4 * 4, dtype=torch.uint8, device=e.device)
    p[:r, :g] = e
    return p.view(p.shape[0] // 128, 4, 32, p.shape[1] // 4, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)


def _untile_scales(s, rows, groups):
    R, G = (rows + 127) // 128, (groups + 3) // 4
    return s.view(R, G, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(R * 128, G * 4)[:rows, :groups]


def _group_exponent(amax):
    """Smallest e >= -127 with amax <= 448 * 2^e; amax == 0 gives -127."""
    m, e = torch.frexp(amax)  # amax = m * 2^e, 0.5 <= m < 1; 448 = 0.875 * 2^9
    e = e - 9 + (m > 0.875).to(e.dtype)
    return torch.where(amax > 0, e, torch.full_like(e, -127)).clamp(min=-127)


def _to_mx8(v):
    """fp32 [rows, cols] -> (codes as float8_e4m3fn [rows, cols], scale exponents [rows, cols / 32])."""
    r, c = v.shape
    g = v.view(r, c // 32, 32)
    e = _group_exponent(g.abs().amax(-1))
    q = torch.ldexp(g, -e.unsqueeze(-1)).to(torch.float8_e4m3fn)
    return q.view(r, c), e


def _from_mx8(codes, scales):
    r, c = codes.shape
    e = _untile_scales(scales, r, c // 32).to(torch.int32) - 127
    return torch.ldexp(codes.float().view(r, c // 32, 32), e.unsqueeze(-1)).view(r, c)


def _mx8_weights(rows, cols, gen):
    q, e = _to_mx8(torch.randn(rows, cols, generator=gen, device="cuda") * 0.02)
    return q, _tile_scales((e + 127).to(torch.uint8))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    kind, T, d = case["kind"], case["T"], case["d"]

    def normal(*shape, scale=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)

    state = dict(case=dict(case))
    if kind in ("norm", "norm_bwd"):
        state["weight"] = (1 + 0.1 * torch.randn(d, generator=gen, device="cuda")).to(torch.bfloat16)
        res_dtype = _DT[case["res"]] if kind == "norm" else _DT[case["x"]]
        # a residual stream: a few channels far larger than the rest, some rows of padding (zeros)
        channel = torch.where(torch.rand(d, generator=gen, device="cuda") < 0.005, 30.0, 1.0)
        live = (torch.rand(T, 1, generator=gen, device="cuda") >= 0.01).float()
        live[0] = 1.0
        res = (torch.randn(T, d, generator=gen, device="cuda") * channel * live).to(res_dtype)
        if kind == "norm":
            state.update(x=(torch.randn(T, d, generator=gen, device="cuda") * 0.5 * live).to(_DT[case["x"]]), res=res)
        else:
            state.update(s=res, dy=normal(T, d, dtype=res_dtype), ds=normal(T, d, dtype=res_dtype))
        return state
    I = case["I"]
    if kind == "ffn_mx8":
        x, e = _to_mx8(torch.randn(T, d, generator=gen, device="cuda"))
        state["x"] = (x, _tile_scales((e + 127).to(torch.uint8)))
        state["gate_up"] = _mx8_weights(2 * I, d, gen)
        state["down"] = _mx8_weights(d, I, gen)
        return state
    state["x"] = normal(T, d)
    state["gate_up"] = normal(2 * I, d, scale=0.02)
    state["down"] = normal(d, I, scale=0.02)
    if kind == "ffn_bwd":
        state["pre"] = torch.matmul(state["x"], state["gate_up"].t())
        state["dy"] = normal(T, d)
    return state


# ------------------------------------------------------------------ the plain forms, in 32 bits
def _act(g, act):
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
    kind = case["kind"]
    if kind == "norm":
        s = state["x"].float() + state["res"].float()
        y = s * torch.rsqrt((s * s).mean(-1, keepdim=True) + EPS) * state["weight"].float()
        kept = s.to(state["res"].dtype)
        if case["out"] != "mx8":
            return {"y": y.to(_DT[case["out"]]), "s": kept}
        codes, e = _to_mx8(y)
        return {"codes": codes, "scales": _tile_scales((e + 127).to(torch.uint8)).view(torch.float8_e8m0fnu), "s": kept}
    if kind == "norm_bwd":
        s, w, dy = state["s"].float(), state["weight"].float(), state["dy"].float()
        r = torch.rsqrt((s * s).mean(-1, keepdim=True) + EPS)
        n = s * r
        g = dy * w
        dx = r * (g - n * (g * n).mean(-1, keepdim=True)) + state["ds"].float()
        return {"dx": dx.to(state["s"].dtype), "dweight": (dy * n).sum(0).to(state["weight"].dtype)}
    act, I = case["act"], case["I"]
    if kind == "ffn_mx8":
        pre = _from_mx8(*state["x"]) @ _from_mx8(*state["gate_up"]).t()
        h, e = _to_mx8(_act(pre[:, :I], act) * pre[:, I:])
        h = torch.ldexp(h.float().view(*e.shape, 32), e.unsqueeze(-1)).view(-1, I)
        return {"y": (h @ _from_mx8(*state["down"]).t()).to(torch.bfloat16)}
    x, wgu, wd = state["x"].float(), state["gate_up"].float(), state["down"].float()
    if kind == "ffn":
        pre = x @ wgu.t()
        y = (_act(pre[:, :I], act) * pre[:, I:]) @ wd.t()
        out = {"y": y.to(torch.bfloat16)}
        if case["save"]:
            out["pre"] = pre.to(torch.bfloat16)
        return out
    g, u = state["pre"].float().split(I, 1)
    dy = state["dy"].float()
    dh = dy @ wd
    a = _act(g, act)
    dpre = torch.cat([dh * u * _act_grad(g, act), dh * a], 1)
    return {"dx": (dpre @ wgu).to(torch.bfloat16), "dgate_up": (dpre.t() @ x).to(torch.bfloat16),
            "ddown": (dy.t() @ (a * u)).to(torch.bfloat16)}


# ------------------------------------------------------------------ the framework's operators
_handles = {}


def _handle(case):
    """The handle that a program keeps for a layer of this shape."""
    import expert_routed_ffn_moe_gb300 as moe

    kind, T, d = case["kind"], case["T"], case["d"]
    key = (kind, T, d, case.get("I"), case.get("act"))
    if key not in _handles:
        if kind in ("norm", "norm_bwd"):
            _handles[key] = moe.AddNorm(d, eps=EPS)
        else:
            _handles[key] = moe.GatedFfn(d, case["I"], max_tokens=T, training=kind == "ffn_bwd",
                                         activation={"silu": moe.MOE_ACT_SILU, "gelu": moe.MOE_ACT_GELU}[case["act"]],
                                         weight_format=moe.MOE_W_MX8 if kind == "ffn_mx8" else moe.MOE_W_BF16)
    return moe, _handles[key]


def _own(state):
    case = state["case"]
    kind = case["kind"]
    moe, op = _handle(case)
    if kind == "norm":
        out = {"bf16": moe.MOE_BF16, "f32": moe.MOE_F32, "mx8": moe.MOE_MX8}[case["out"]]
        y, s = op.forward(state["x"], state["res"], state["weight"], y_dtype=out)
        if case["out"] != "mx8":
            return {"y": y, "s": s}
        return {"codes": y[0], "scales": y[1].view(torch.float8_e8m0fnu), "s": s}
    if kind == "norm_bwd":
        dx, dw = op.backward(state["s"], state["weight"], state["dy"], state["ds"])
        return {"dx": dx, "dweight": dw}
    if kind == "ffn_bwd":
        dx, dgu, dd = op.backward(state["x"], state["pre"], state["gate_up"], state["down"], state["dy"])
        return {"dx": dx, "dgate_up": dgu, "ddown": dd}
    if kind == "ffn" and case["save"]:
        y, pre = op.forward(state["x"], state["gate_up"], state["down"], save=True)
        return {"y": y, "pre": pre}
    return {"y": op.forward(state["x"], state["gate_up"], state["down"])}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ work and exact values
def work(case):
    kind, T, d = case["kind"], case["T"], case["d"]
    size = {"bf16": 2, "f32": 4, "mx8": 1 + 1 / 32}
    if kind == "norm":
        return {"bytes": T * d * (size[case["x"]] + 2 * size[case["res"]] + size[case["out"]]) + 2 * d, "flops": 5 * T * d}
    if kind == "norm_bwd":
        return {"bytes": 4 * T * d * size[case["x"]] + 4 * d, "flops": 12 * T * d}
    I = case["I"]
    if kind == "ffn_mx8":
        return {"bytes": (T * d + 3 * d * I) * size["mx8"] + 2 * T * d, "flops": 6 * T * d * I}
    if kind == "ffn":
        return {"bytes": 2 * (2 * T * d + 3 * d * I + (2 * T * I if case["save"] else 0)), "flops": 6 * T * d * I}
    return {"bytes": 2 * (3 * T * d + 6 * d * I + 2 * T * I), "flops": 12 * T * d * I}


def exact(case, seed):
    """From the definitions in 64 bits.  Where an output is rounded to fewer bits its value before that rounding."""
    st = prepare(case, seed)
    D = torch.float64
    kind = case["kind"]
    if kind == "norm":
        s = st["x"].to(D) + st["res"].to(D)
        y = st["weight"].to(D) * s / (s.pow(2).sum(-1, keepdim=True) / case["d"] + EPS).sqrt()
        if case["out"] != "mx8":
            return {"y": y, "s": s}
        groups = y.reshape(case["T"], -1, 32)
        top = groups.abs().max(-1).values
        e = torch.where(top > 0, torch.ceil(torch.log2(top / 448)), torch.full_like(top, -127)).clamp(min=-127)
        # codes: the quotients that are rounded to e4m3
        return {"codes": (groups / torch.exp2(e).unsqueeze(-1)).reshape(y.shape),
                "scales": torch.exp2(_tile_scales((e + 127).to(torch.uint8)).to(D) - 127), "s": s}
    if kind == "norm_bwd":
        s, w, dy = st["s"].to(D), st["weight"].to(D), st["dy"].to(D)
        v = s.pow(2).sum(-1, keepdim=True) / case["d"] + EPS
        proj = (dy * w * s).sum(-1, keepdim=True) / case["d"]
        return {"dx": dy * w / v.sqrt() - s * proj / v.pow(1.5) + st["ds"].to(D), "dweight": (dy * s / v.sqrt()).sum(0)}
    I = case["I"]
    silu = case["act"] == "silu"

    def phi(g):  # act(g) = g * phi(g): the logistic function of g, or of the tanh form's argument
        return torch.sigmoid(g if silu else 2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3))

    def wide(m):
        codes, scales = m
        r, c = codes.shape
        scale = torch.exp2(_untile_scales(scales, r, c // 32).to(D) - 127)
        return codes.float().to(D) * scale.repeat_interleave(32, 1)

    if kind == "ffn_mx8":
        wgu = wide(st["gate_up"])
        x = wide(st["x"])
        g, u = x @ wgu[:I].t(), x @ wgu[I:].t()
        del wgu
        h = (g * phi(g) * u).reshape(case["T"], -1, 32)
        top = h.abs().max(-1, keepdim=True).values
        unit = torch.exp2(torch.ceil(torch.log2(top / 448)).clamp(min=-127))
        h = ((h / unit).float().to(torch.float8_e4m3fn).float().to(D) * unit).reshape(case["T"], I)
        return {"y": h @ wide(st["down"]).t()}
    x, wgu, wd = (st[k].to(D) for k in ("x", "gate_up", "down"))
    if kind == "ffn":
        pre = torch.cat([x @ wgu[:I].t(), x @ wgu[I:].t()], 1)
        y = (pre[:, :I] * phi(pre[:, :I]) * pre[:, I:]) @ wd.t()
        return {"y": y, "pre": pre} if case["save"] else {"y": y}
    g, u = st["pre"][:, :I].to(D), st["pre"][:, I:].to(D)
    dy = st["dy"].to(D)
    p = phi(g)
    inner = torch.ones_like(g) if silu else 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * g ** 2)
    dh = dy @ wd
    dg, du = dh * u * (p + g * p * (1 - p) * inner), dh * g * p
    dx = dg @ wgu[:I] + du @ wgu[I:]
    return {"dx": dx, "dgate_up": torch.cat([dg.t() @ x, du.t() @ x]), "ddown": dy.t() @ (g * p * u)}
