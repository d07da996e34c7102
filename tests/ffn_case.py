"""Definitions in 64 bits of the feed-forward block, its norm and the mx8 form,
for the tests, with bounds on how far a right result may be from them.

Rounding to bf16 is off by at most 2^-8 of the value (HALF), with a standard
deviation of at most 2^-8 / sqrt(3) of it; fp32 sums of K products by at most
K * 2^-24 of the sum of their magnitudes; the fast exponential and division of
the activations by ~2^-21, counted as 2^-18 of each term.  A sum over K
independently rounded bf16 terms t_i is then off by at most 6 standard
deviations, 6 * 2^-8 / sqrt(3) * sqrt(sum t_i^2).
"""
import math

import torch

D = torch.float64
HALF = 2.0 ** -8
SIX = 6 * HALF / math.sqrt(3)
C = math.sqrt(2 / math.pi)


def act(g, gelu):
    return g * torch.sigmoid(2 * C * (g + 0.044715 * g ** 3)) if gelu else g * torch.sigmoid(g)


def act_grad(g, gelu):
    # 0.5 (1 + tanh z) = sigmoid(2 z): the form whose far negative tail does not cancel
    s = torch.sigmoid(2 * C * (g + 0.044715 * g ** 3) if gelu else g)
    inner = 2 * C * (1 + 3 * 0.044715 * g * g) if gelu else 1.0
    return s * (1 + g * (1 - s) * inner)


def product_bound(a, b, rounded, extra=2.0 ** -18):
    """Bound on the error of a @ b.t() (before its own rounding) where a's entries were rounded to bf16
    (``rounded``) from values that are right to ``extra`` of their size."""
    k = a.shape[1]
    mags = a.abs() @ b.abs().t()
    e = (k * 2.0 ** -24 + (extra if rounded else 0)) * mags
    if rounded:
        e = e + SIX * (a.square() @ b.square().t()).sqrt()
    return e


def forward(x, gate_up, down, gelu):
    """pre, y and the bounds of their errors."""
    x, gate_up, down = x.to(D), gate_up.to(D), down.to(D)
    I = down.shape[1]
    pre = x @ gate_up.t()
    e_pre = product_bound(x, gate_up, False)
    g, u = pre[:, :I], pre[:, I:]
    h = act(g, gelu) * u
    e_h = 1.2 * (u.abs() * e_pre[:, :I] + act(g, gelu).abs() * e_pre[:, I:])  # |act'| <= 1.13
    y = h @ down.t()
    e_y = product_bound(h, down, True) + e_h @ down.abs().t()
    tiny = 1e-30
    return pre, HALF * pre.abs() + e_pre + tiny, y, HALF * y.abs() + e_y + tiny


def backward(x, pre, gate_up, down, dy, gelu):
    """{name: (value, bound)} of dx, dgate_up, ddown."""
    x, pre, gate_up, down, dy = (t.to(D) for t in (x, pre, gate_up, down, dy))
    I = down.shape[1]
    g, u = pre[:, :I], pre[:, I:]
    dh = dy @ down
    e_dh = product_bound(dy, down.t(), False)
    a, da = act(g, gelu), act_grad(g, gelu)
    dpre = torch.cat([dh * u * da, dh * a], 1)
    e_dpre = torch.cat([e_dh * (u * da).abs(), e_dh * a.abs()], 1)
    h = a * u
    out = {}
    for name, m, n, e in (("dx", dpre, gate_up.t(), e_dpre), ("dgate_up", dpre.t(), x.t(), e_dpre.t()),
                          ("ddown", None, None, None)):
        if name == "ddown":
            v, b = dy.t() @ h, product_bound(h.t(), dy.t(), True).t()
        else:
            v, b = m @ n.t(), product_bound(m, n, True) + e @ n.abs().t()
        out[name] = (v, HALF * v.abs() + b + 1e-30)
    return out


# ------------------------------------------------------------------ mx8
def scale_index(rows, cols, device="cpu"):
    """Position in the stored bytes of every (row, group)."""
    r = torch.arange(rows, device=device).view(-1, 1)
    g = torch.arange(cols // 32, device=device).view(1, -1)
    return ((r // 128) * ((cols + 127) // 128) + g // 4) * 512 + (r % 32) * 16 + (r // 32 % 4) * 4 + g % 4


def exponents(v):
    """The exponent of each group of 32 columns of v, from its definition."""
    top = v.to(D).reshape(v.shape[0], -1, 32).abs().max(-1).values
    e = torch.full_like(top, -127)
    ok = top > 0
    e[ok] = torch.ceil(torch.log2(top[ok] / 448))
    # log2 may be off by an ulp next to a power of two: settle by the definition itself
    e = torch.where(ok & (top <= 448 * torch.exp2(e - 1)), e - 1, e)
    e = torch.where(ok & (top > 448 * torch.exp2(e)), e + 1, e)
    return e.clamp(min=-127)


def quantize(v):
    """(codes as float8_e4m3fn, stored scale bytes) of a finite matrix."""
    rows, cols = v.shape
    e = exponents(v)
    q = (v.to(D).reshape(rows, -1, 32) / torch.exp2(e).unsqueeze(-1)).float().to(torch.float8_e4m3fn).view(rows, cols)
    s = torch.zeros((rows + 127) // 128 * ((cols + 127) // 128) * 512, dtype=torch.uint8, device=v.device)
    s[scale_index(rows, cols, v.device).view(-1)] = (e + 127).to(torch.uint8).view(-1)
    return q, s


def dequantize(codes, scales):
    rows, cols = codes.shape
    e = scales[scale_index(rows, cols, codes.device).view(-1)].view(rows, -1).to(D) - 127
    return codes.view(torch.float8_e4m3fn).float().to(D) * torch.exp2(e).repeat_interleave(32, 1)


def forward_mx(x, gate_up, down, gelu):
    """y and the bound of its error.  A value of h next to a rounding boundary may fall on its other side in
    fp32, one e4m3 step (2^-3 of it at most) away: so many that two standard deviations of one such step on
    every 16th term cover them, plus the largest single one."""
    x, gate_up, down = (dequantize(*t) for t in (x, gate_up, down))
    I = down.shape[1]
    pre = x @ gate_up.t()
    h = act(pre[:, :I], gelu) * pre[:, I:]
    h = dequantize(*quantize(h))
    y = h @ down.t()
    sq = (h.square() @ down.square().t()).sqrt()
    worst = h.abs().max(1, keepdim=True).values * down.abs().max(1).values.view(1, -1)
    return y, HALF * y.abs() + product_bound(h, down, False) + 2 * 2.0 ** -3 / 4 * sq + 2.0 ** -3 * worst + 1e-30


# ------------------------------------------------------------------ norm
def norm(x, res, w, eps):
    s = x.to(D) if res is None else x.to(D) + res.to(D)
    return s, s * torch.rsqrt(s.square().mean(-1, keepdim=True) + eps) * w.to(D)


def norm_backward(s, w, dy, ds, eps):
    s, w, dy = s.to(D), w.to(D), dy.to(D)
    r = torch.rsqrt(s.square().mean(-1, keepdim=True) + eps)
    n, g = s * r, dy * w
    dx = r * (g - n * (g * n).mean(-1, keepdim=True))
    if ds is not None:
        dx = dx + ds.to(D)
    return dx, (dy * n).sum(0)
