"""A pre-norm dense feed-forward block, trained for a few steps and then served.

    python examples/dense_block.py [--d 1024] [--inter 2816] [--tokens 512] [--steps 20]

Training: s = x + residual, y = norm(s), f = down(silu(gate(y)) * up(y)), fitted
to a teacher block of the same shape by plain gradient steps, with the backward
passes of both operators.  Serving: the trained weights are rounded to mx8 once,
and single tokens and a prompt go through norm (to mx8 rows) and the mx8 block.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import expert_routed_ffn_moe_gb300 as moe  # noqa: E402


def weights(d, inter, gen):
    def normal(*shape, scale):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(torch.bfloat16)

    return dict(norm=torch.ones(d, dtype=torch.bfloat16, device="cuda"), gate_up=normal(2 * inter, d, scale=d ** -0.5),
                down=normal(d, inter, scale=inter ** -0.5))


def train(d, inter, tokens, steps, lr=2.0, seed=0):
    """Loss of every step, and the trained weights."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    norm, ffn = moe.AddNorm(d), moe.GatedFfn(d, inter, max_tokens=tokens, training=True)
    teacher, w = weights(d, inter, gen), weights(d, inter, gen)
    master = {k: v.float() for k, v in w.items()}
    losses = []
    x = torch.randn(tokens, d, generator=gen, device="cuda").to(torch.bfloat16)
    res = torch.randn(tokens, d, generator=gen, device="cuda").to(torch.bfloat16)
    want = ffn.forward(norm.forward(x, res, teacher["norm"])[0], teacher["gate_up"], teacher["down"])
    for _ in range(steps):
        y, s = norm.forward(x, res, w["norm"])
        out, pre = ffn.forward(y, w["gate_up"], w["down"], save=True)
        diff = out.float() - want.float()
        losses.append(diff.square().mean())
        dout = (diff * (2.0 / tokens)).to(torch.bfloat16)  # gradient of d times the loss
        dy, dgate_up, ddown = ffn.backward(y, pre, w["gate_up"], w["down"], dout)
        _, dnorm = norm.backward(s, w["norm"], dy)
        for k, g in (("norm", dnorm), ("gate_up", dgate_up), ("down", ddown)):
            master[k] -= lr / d * g.float()
            w[k] = master[k].to(torch.bfloat16)
    status = ffn.status()  # (read once: that clears it)
    if status != moe.MOE_OK:
        raise RuntimeError(moe.moe_strerror(status))
    return [float(v) for v in losses], w


def serve(w, tokens, seed=1):
    """The block on mx8 weights for one token and for a prompt, beside the bf16 block: relative differences."""
    d, inter = w["down"].shape
    gen = torch.Generator(device="cuda").manual_seed(seed)
    norm = moe.AddNorm(d)
    mx = moe.GatedFfn(d, inter, max_tokens=tokens, weight_format=moe.MOE_W_MX8)
    bf = moe.GatedFfn(d, inter, max_tokens=tokens)
    gate_up, down = moe.moe_quantize_mx(w["gate_up"]), moe.moe_quantize_mx(w["down"])  # laid out once
    off = {}
    for n in (1, tokens):
        x = torch.randn(n, d, generator=gen, device="cuda").to(torch.bfloat16)
        res = torch.randn(n, d, generator=gen, device="cuda").to(torch.bfloat16)
        rows, s = norm.forward(x, res, w["norm"], y_dtype=moe.MOE_MX8)
        out = mx.forward(rows, gate_up, down)
        ref = bf.forward(norm.forward(x, res, w["norm"])[0], w["gate_up"], w["down"])
        off[n] = float((out.float() - ref.float()).norm() / ref.float().norm())
        norm.forward(out, s, w["norm"], s_out=s)  # the next block's norm, the residual stream updated in place
    if mx.status() != moe.MOE_OK or bf.status() != moe.MOE_OK:
        raise RuntimeError("a wait inside a kernel ran out")
    return off


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, default in (("d", 1024), ("inter", 2816), ("tokens", 512), ("steps", 20)):
        ap.add_argument("--" + name, type=int, default=default)
    a = ap.parse_args()
    moe.build()
    losses, w = train(a.d, a.inter, a.tokens, a.steps)
    print("loss: " + " ".join("%.4f" % v for v in losses))
    for n, v in serve(w, a.tokens).items():
        print(f"mx8 beside bf16, {n} token(s): relative difference {v:.3f}")


if __name__ == "__main__":
    main()
