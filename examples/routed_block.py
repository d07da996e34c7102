"""A pre-norm routed feed-forward block of the classic form (layer norm, experts with biases and gelu), trained.

    python examples/routed_block.py [--d 512] [--inter 1024] [--experts 8] [--top-k 2] [--tokens 512] [--steps 20]

Forward: s = x + residual, y = layer_norm(s); a router picks top_k experts per token; the tokens are sorted by
expert, each expert is two matrix products (bias and gelu in the first one's epilogue, bias in the second's) on its
slice of the rows, and the results come back in token order, weighted, on top of s.  Backward: the same steps in
reverse, each with its operator's gradient; the router's own gradient goes through the weights of the picks.  The
block is fitted to a teacher of the same shape by plain gradient steps.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import expert_routed_ffn_moe_gb300 as moe  # noqa: E402


def weights(d, inter, n_experts, gen):
    def normal(*shape, scale, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)

    return dict(norm_w=torch.ones(d, dtype=torch.bfloat16, device="cuda"), norm_b=normal(d, scale=0.1),
                router=normal(n_experts, d, scale=d ** -0.5, dtype=torch.float32),
                up=normal(n_experts, inter, d, scale=d ** -0.5), up_b=normal(n_experts, inter, scale=0.1),
                down=normal(n_experts, d, inter, scale=inter ** -0.5), down_b=normal(n_experts, d, scale=0.1))


class RoutedBlock:
    """The operators of one block; weights are passed to each call."""

    def __init__(self, d, inter, n_experts, top_k, tokens):
        self.norm = moe.LayerNorm(d)
        self.router = moe.MoeLayer(d, n_experts, 128, top_k, tokens, has_shared=False)  # (its routing alone is used)
        self.sort = moe.TokenDispatch(n_experts, top_k)
        # one context per product serves all experts, whose calls follow one another on the stream
        self.up = moe.Linear(d, inter, tokens * top_k, activation=moe.MOE_ACT_GELU, training=True)
        self.down = moe.Linear(inter, d, tokens * top_k, training=True)

    def forward(self, w, x, residual):
        """(out, saved): out = s + the experts' weighted sum."""
        y, s = self.norm.forward(x, residual, w["norm_w"], w["norm_b"])
        picks = self.router.route(y, w["router"], None)
        _, offsets, _, slot = self.sort.sort(picks["idx"])
        rows = self.sort.dispatch(y, slot)
        ends = offsets.tolist()  # (the host needs the slices' sizes)
        pre = torch.empty(rows.shape[0], w["up"].shape[1], dtype=torch.bfloat16, device=x.device)
        h, out_rows = torch.empty_like(pre), torch.empty_like(rows)
        for e in range(w["up"].shape[0]):
            at = slice(ends[e], ends[e + 1])
            self.up.forward(rows[at], w["up"][e], w["up_b"][e], y=h[at], pre=pre[at])
            self.down.forward(h[at], w["down"][e], w["down_b"][e], y=out_rows[at])
        out = self.sort.combine(out_rows, slot, picks["w"], add=s)
        return out, dict(y=y, s=s, idx=picks["idx"], pick_w=picks["w"], slot=slot, ends=ends, rows=rows, pre=pre, h=h,
                         out_rows=out_rows)

    def backward(self, w, saved, dout):
        """Gradients of the weights, and of x (and the residual) as "x"."""
        v, g = saved, {k: torch.empty_like(t) for k, t in w.items()}
        drows, dpick = self.sort.combine_backward(dout, v["out_rows"], v["slot"], v["pick_w"])
        dx_rows, dh = torch.empty_like(v["rows"]), torch.empty_like(v["h"])
        for e in range(w["up"].shape[0]):
            at = slice(v["ends"][e], v["ends"][e + 1])
            self.down.backward(v["h"][at], None, w["down"][e], w["down_b"][e], drows[at], dh[at], g["down"][e],
                               g["down_b"][e])
            self.up.backward(v["rows"][at], v["pre"][at], w["up"][e], w["up_b"][e], dh[at], dx_rows[at], g["up"][e],
                             g["up_b"][e])
        # the weights are the softmax of the picked logits
        dlogit = v["pick_w"] * (dpick - (v["pick_w"] * dpick).sum(1, keepdim=True))
        dlogits = torch.zeros(dlogit.shape[0], w["router"].shape[0], device=dlogit.device)
        dlogits.scatter_(1, v["idx"].long(), dlogit)
        g["router"] = dlogits.t() @ v["y"].float()
        dy = self.sort.dispatch_backward(dx_rows, v["slot"], add=(dlogits @ w["router"]).to(torch.bfloat16))
        g["x"], g["norm_w"], g["norm_b"] = self.norm.backward(v["s"], w["norm_w"], dy, dout)
        return g

    def check(self):
        for op in (self.router, self.up, self.down):
            status = op.status()
            if status != moe.MOE_OK:
                raise RuntimeError(moe.moe_strerror(status))


def train(d, inter, n_experts, top_k, tokens, steps, lr=1.0, seed=0):
    """Loss of every step."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    block = RoutedBlock(d, inter, n_experts, top_k, tokens)
    teacher, w = weights(d, inter, n_experts, gen), weights(d, inter, n_experts, gen)
    master = {k: t.float() for k, t in w.items()}
    losses = []
    for _ in range(steps):
        x = torch.randn(tokens, d, generator=gen, device="cuda").to(torch.bfloat16)
        res = torch.randn(tokens, d, generator=gen, device="cuda").to(torch.bfloat16)
        want, _ = block.forward(teacher, x, res)
        out, saved = block.forward(w, x, res)
        diff = out.float() - want.float()
        losses.append(diff.square().mean())
        grads = block.backward(w, saved, (diff * (2.0 / tokens)).to(torch.bfloat16))
        for k in w:
            master[k] -= lr / d * grads[k].float()
            w[k] = master[k].to(w[k].dtype)
    block.check()
    return [float(v) for v in losses]


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, default in (("d", 512), ("inter", 1024), ("experts", 8), ("top-k", 2), ("tokens", 512), ("steps", 20)):
        ap.add_argument("--" + name, type=int, default=default)
    a = ap.parse_args()
    moe.build()
    losses = train(a.d, a.inter, a.experts, a.top_k, a.tokens, a.steps)
    print("loss: " + " ".join("%.4f" % v for v in losses))


if __name__ == "__main__":
    main()
