"""Definitions in 64 bits of the layer norm, of tokens sorted by expert and back and of the product with its
epilogue, for the tests, with bounds on how far a right result may be from them.

Counted: one rounding to a type at half its step (bf16 2^-8, fp32 2^-24 of the value); an fp32 sum whose longest chain
of additions has D links at D * 2^-24 of the sum of magnitudes; rsqrt and quotients at 2^-22; the fast exponential and
division of the activations at 2^-18 of each term, as in ffn_case.
"""
import torch

import ffn_case as fc

D = torch.float64
U = 2.0 ** -24


def half_step(dtype):
    return fc.HALF if dtype == torch.bfloat16 else U


def act(g, name):
    return g if name == "none" else fc.act(g, name == "gelu")


def act_grad(g, name):
    return torch.ones_like(g) if name == "none" else fc.act_grad(g, name == "gelu")


# ------------------------------------------------------------------ layer norm
ROW = 40  # links of a row's sum: a thread's 16 values, two trees of 5 over 32, and the roundings of its terms


def _stats(s, eps):
    """c, rstd, the error of c and the relative error of rstd, for s known to fp32."""
    mean = s.mean(-1, keepdim=True)
    c = s - mean
    sd = (c.square().mean(-1, keepdim=True) + eps).sqrt()
    e_c = U * ((ROW + 2) * s.abs().mean(-1, keepdim=True) + s.abs() + c.abs())
    # mean(c^2): twice c's error times c, relative to sd^2, through the square root half of that
    rho = (e_c * c.abs() + e_c.square()).mean(-1, keepdim=True) / sd.square() + (ROW + 2) * U + 2.0 ** -22
    return c, 1 / sd, e_c, rho


def layer_norm(x, res, w, b, eps, s_dtype, y_dtype):
    """{name: (value, bound)} of s and y."""
    s = x.to(D) if res is None else x.to(D) + res.to(D)
    c, r, e_c, rho = _stats(s, eps)
    w = torch.ones_like(s[:1]) if w is None else w.to(D)
    b = torch.zeros_like(s[:1]) if b is None else b.to(D)
    y = c * r * w + b
    e = w.abs() * r * (e_c + c.abs() * rho) + 3 * U * ((c * r * w).abs() + b.abs())
    return {"s": (s, half_step(s_dtype) * s.abs()), "y": (y, half_step(y_dtype) * (y.abs() + e) + e + 1e-30)}


def layer_norm_backward(s, w, dy, ds, eps, w_dtype):
    """{name: (value, bound)} of dx, dweight and dbias."""
    dtype, T = s.dtype, s.shape[0]
    s, dy = s.to(D), dy.to(D)
    w = torch.ones_like(s[:1]) if w is None else w.to(D)
    c, r, e_c, rho = _stats(s, eps)
    n, g = c * r, dy * w
    e_n = r * e_c + n.abs() * (rho + 2 * U)
    gm, gnm = g.mean(-1, keepdim=True), (g * n).mean(-1, keepdim=True)
    e_gm = ROW * U * g.abs().mean(-1, keepdim=True)
    e_gnm = (g.abs() * e_n).mean(-1, keepdim=True) + (ROW + 4) * U * (g * n).abs().mean(-1, keepdim=True)
    dx = r * (g - gm - n * gnm)
    parts = g.abs() + gm.abs() + (n * gnm).abs()
    e = r * (e_gm + e_n * gnm.abs() + n.abs() * e_gnm + (rho + 6 * U) * parts)
    if ds is not None:
        dx = dx + ds.to(D)
        e = e + U * dx.abs()
    chain = T / 128 + 48  # a block's rows, 608 blocks by 32 threads, a tree of 5, four warps
    dw, db = (dy * n).sum(0), dy.sum(0)
    e_dw = (dy.abs() * e_n).sum(0) + chain * U * (dy * n).abs().sum(0)
    e_db = chain * U * dy.abs().sum(0)
    return {"dx": (dx, half_step(dtype) * (dx.abs() + e) + e + 1e-30),
            "dweight": (dw, half_step(w_dtype) * (dw.abs() + e_dw) + e_dw + 1e-30),
            "dbias": (db, half_step(w_dtype) * (db.abs() + e_db) + e_db + 1e-30)}


# ------------------------------------------------------------------ tokens sorted by expert
def sort(idx, E):
    """(counts, offsets, perm, slot) by a walk over the picks; ids outside 0 .. E - 1 are dropped."""
    T, k = idx.shape
    groups = [[] for _ in range(E)]
    for p, e in enumerate(idx.flatten().tolist()):
        if 0 <= e < E:
            groups[e].append(p)
    order = [p for g in groups for p in g]
    slot = torch.full((T * k,), -1, dtype=torch.int32)
    slot[torch.tensor(order, dtype=torch.long)] = torch.arange(len(order), dtype=torch.int32)
    counts = torch.tensor([len(g) for g in groups], dtype=torch.int32)
    offsets = torch.cat([torch.zeros(1, dtype=torch.int32), counts.cumsum(0).int()])
    perm = torch.tensor([p // k for p in order], dtype=torch.int32)
    return counts, offsets, perm, slot.view(T, k)


def picks(slot, n_rows):
    """(token, pick, row) of the picks that are not dropped."""
    t, j = ((slot >= 0) & (slot < n_rows)).nonzero(as_tuple=True)
    return t, j, slot[t, j].long()


def combine(rows, slot, w, add, y_dtype):
    """y and the bound of its error."""
    T, k = slot.shape
    t, j, r = picks(slot, rows.shape[0])
    v = rows[r].to(D)
    if w is not None:
        v = v * w[t, j].to(D).unsqueeze(1)
    y = torch.zeros(T, rows.shape[1], dtype=D, device=rows.device)
    mags = y.clone()
    y.index_add_(0, t, v)
    mags.index_add_(0, t, v.abs())
    if add is not None:
        y, mags = y + add.to(D), mags + add.to(D).abs()
    e = (k + 2) * U * mags
    return y, half_step(y_dtype) * (y.abs() + e) + e + 1e-30


def combine_dw(dy, rows, slot):
    """dw and the bound of its error."""
    t, j, r = picks(slot, rows.shape[0])
    a, b = dy[t].to(D), rows[r].to(D)
    dw = torch.zeros(slot.shape, dtype=D, device=rows.device)
    e = dw.clone()
    dw[t, j] = (a * b).sum(1)
    # a lane's columns one after another, a tree of 5, up to eight warps
    e[t, j] = (rows.shape[1] / 32 + 48) * U * (a * b).abs().sum(1)
    return dw, e + 1e-30


# ------------------------------------------------------------------ product with its epilogue
def linear(x, w, b, res, name, y_dtype):
    """{name: (value, bound)} of pre and y."""
    x, w = x.to(D), w.to(D)
    pre = x @ w.t()
    e = fc.product_bound(x, w, False)
    if b is not None:
        pre = pre + b.to(D)
        e = e + U * (pre.abs() + b.to(D).abs())
    y = act(pre, name)
    e_y = e if name == "none" else 1.2 * e + 2.0 ** -18 * y.abs()  # |act'| <= 1.13
    if res is not None:
        y = y + res.to(D)
        e_y = e_y + U * y.abs()
    return {"pre": (pre, fc.HALF * (pre.abs() + e) + e + 1e-30), "y": (y, half_step(y_dtype) * (y.abs() + e_y) + e_y + 1e-30)}


def linear_backward(x, pre, w, dy, name, b_dtype):
    """{name: (value, bound)} of dx, dweight and dbias."""
    rounded = name != "none" or dy.dtype != torch.bfloat16
    x, w, dy = x.to(D), w.to(D), dy.to(D)
    dpre, e = dy, torch.zeros_like(dy)
    if name != "none":
        da = act_grad(pre.to(D), name)
        dpre, e = dy * da, 2.0 ** -18 * dy.abs() * (1 + da.abs())  # (act' has terms up to about one that cancel)
    out = {"dx": (dpre @ w, fc.product_bound(dpre, w.t(), rounded) + e @ w.abs()),
           "dweight": (dpre.t() @ x, fc.product_bound(dpre.t(), x.t(), rounded) + e.t() @ x.abs())}
    out = {k: (v, fc.HALF * (v.abs() + s) + s + 1e-30) for k, (v, s) in out.items()}
    db = dpre.sum(0)
    # every 256th row in a thread, 32 threads, 8 blocks
    e_db = e.sum(0) + (dy.shape[0] / 256 + 48) * U * dpre.abs().sum(0)
    out["dbias"] = (db, half_step(b_dtype) * (db.abs() + e_db) + e_db + 1e-30)
    return out
