"""Data on which the mx8 block's pre-activations are exact in fp32, so that the
codes and scales of h are known but for values next to a rounding boundary, and
a bound on y narrow enough to tell whether h was held in mx8.

Operands are small integers times powers of two (exact in mx8), each group of 32
columns with a power of its own.  Every addend of a pre-activation is then a
multiple of one unit, and all of them together stay below 2^24 units: fp32 sums
in any order, and sums cut to 24 bits, are exact.

h = act(g) * u in fp32 is off by EPS(g) of its value: with z the argument of the
logistic function (g, or 2 sqrt(2 / pi) (g + 0.044715 g^3) from four roundings),
|z| 2^-22 from z's rounding, (2 + 1.2 |z|) 2^-23 from the fast exponential, 2^-22
from the fast division and four products: below 2^-20 + |z| 2^-21.

y = h down^T sums I terms in fp32, in which every addition loses at most 2^-23 of
the larger of the running sum and the addend; sums of terms of independent signs
stay within six standard deviations, 6 sqrt(sum of their squares).
"""
import math

import torch

import ffn_case as fc

D = fc.D


def integers(rows, cols, top, unit, gen, device):
    """Integers of [-top, top] times unit times 1, 2 or 4 for each group of 32 columns, in fp32."""
    v = torch.randint(-top, top + 1, (rows, cols), generator=gen, device=device).float()
    p = torch.randint(0, 3, (rows, cols // 32), generator=gen, device=device).float()
    return v * unit * torch.exp2(p).repeat_interleave(32, 1)


def operands(T, d, I, seed, device="cpu"):
    """x [T, d], gate_up [2I, d], down [d, I] in fp32, pre-activations of a size of about 2."""
    gen = torch.Generator(device=device).manual_seed(seed)
    unit = 2.0 ** -math.ceil(math.log2(math.sqrt(d) * 2.8))
    x = integers(T, d, 2, 1.0, gen, device)
    gu = integers(2 * I, d, 1, unit, gen, device)
    # an addend is at most (2 * 4) * (1 * 4) units
    assert d * 32 < 1 << 24
    return x, gu, integers(d, I, 4, 2.0 ** -5, gen, device)


def hidden(x, gate_up, gelu):
    """h in 64 bits, and the relative error that fp32 may bring."""
    pre = x.to(D) @ gate_up.to(D).t()
    I = pre.shape[1] // 2
    g, u = pre[:, :I], pre[:, I:]
    z = 2 * fc.C * (g + 0.044715 * g ** 3) if gelu else g
    return fc.act(g, gelu) * u, 2.0 ** -20 + z.abs() * 2.0 ** -21


def codes_of(v, e):
    """v rounded to e4m3 with the exponents e of its groups."""
    s = torch.exp2(e).repeat_interleave(32, 1)
    return (v / s).clamp(-448, 448).float().to(torch.float8_e4m3fn).float().to(D) * s


def forward(x, gate_up, down, gelu):
    """y and the bound of its error, from operands that are exact in mx8."""
    h, eps = hidden(x, gate_up, gelu)
    down = down.to(D)
    q = codes_of(h, fc.exponents(h))
    # how far the value that is stored may be from q: the ends of h's error interval, with the exponents of either end
    less, more = h * (1 - eps), h * (1 + eps)
    flip = torch.zeros_like(h)
    for e in (fc.exponents(less), fc.exponents(more)):
        for v in (less, more):
            flip = torch.maximum(flip, (codes_of(v, e) - q).abs())
    y = q @ down.t()
    I = h.shape[1]
    sums = 6 * (q.square() @ down.square().t()).sqrt()
    return y, fc.HALF * y.abs() + flip @ down.abs().t() + I * 2.0 ** -23 * sums + 1e-30


SHAPES = [(1, 2048, 512), (1, 4096, 8192), (17, 4096, 32), (48, 1024, 3008), (3, 160, 8992), (1, 32, 32), (2, 64, 96),
          (16, 256, 160), (33, 96, 2048), (64, 512, 224), (128, 256, 128), (129, 288, 384), (257, 1024, 992),
          (511, 160, 1568), (1000, 352, 2752), (33, 4096, 2752), (64, 1056, 10624), (700, 4128, 4096)]
