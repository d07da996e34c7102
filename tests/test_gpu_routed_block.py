"""Layer norm, routing, sorted tokens, the experts' products and the way back, as a block uses them together."""
import importlib.util
import os

import pytest
import torch

import expert_routed_ffn_moe_gb300 as moe
import ops_case as oc

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "routed_block.py")
    spec = importlib.util.spec_from_file_location("routed_block", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def reference(w, x, res, idx):
    """out in 64 bits with these picks."""
    s = x + res
    y = torch.nn.functional.layer_norm(s, s.shape[-1:], w["norm_w"], w["norm_b"], 1e-5)
    pick = torch.softmax((y @ w["router"].t()).gather(1, idx), 1)
    out = s
    for j in range(idx.shape[1]):
        for e in range(w["up"].shape[0]):
            t = (idx[:, j] == e).nonzero().flatten()
            h = oc.act(y[t] @ w["up"][e].t() + w["up_b"][e], "gelu")
            out = out.index_add(0, t, pick[t, j, None] * (h @ w["down"][e].t() + w["down_b"][e]))
    return out


@pytest.mark.parametrize("tokens,experts,top_k", [(1, 4, 2), (37, 8, 3), (300, 5, 2), (200, 200, 1)])
def test_block_and_gradients_match_the_definition(example, tokens, experts, top_k):
    d, inter = 256, 328
    gen = torch.Generator(device="cuda").manual_seed(tokens)
    w = example.weights(d, inter, experts, gen)
    block = example.RoutedBlock(d, inter, experts, top_k, tokens)
    x, res, dout = (torch.randn(tokens, d, generator=gen, device="cuda").to(torch.bfloat16) for _ in range(3))
    out, saved = block.forward(w, x, res)
    grads = block.backward(w, saved, dout)
    block.check()
    leaves = {k: t.to(oc.D).requires_grad_() for k, t in w.items()}
    xd = x.to(oc.D).requires_grad_()
    want = reference(leaves, xd, res.to(oc.D), saved["idx"].long())
    leaves["x"] = xd
    # The results differ from the definition by the roundings to bf16 on the way (some twelve, each of a relative root mean
    # square of 2^-8 / sqrt(3), doubled at most by the activation's and the norm's slopes): sqrt(12) * 2 * 0.0023 = 0.016.
    def near(got, value, name):
        off = (got.to(oc.D) - value).norm() / value.norm().clamp(min=1e-3)
        assert off < 0.02, (name, float(off))

    near(out, want.detach(), "out")
    for (name, _), g in zip(leaves.items(), torch.autograd.grad(want, list(leaves.values()), dout.to(oc.D))):
        near(grads[name], g, name)


def test_two_steps_run(example):
    losses = example.train(256, 136, 6, 2, 50, 2)
    assert len(losses) == 2 and all(v == v and v < 1e4 for v in losses)


def test_dense_block_of_two_products_in_a_graph():
    # layer norm, product with gelu, product with the residual, and back, captured and replayed on new data
    T, d, inter = 130, 264, 520
    gen = torch.Generator(device="cuda").manual_seed(1)
    n = lambda *s, scale=1.0: (torch.randn(*s, generator=gen, device="cuda") * scale).to(torch.bfloat16)  # noqa: E731
    norm, up = moe.LayerNorm(d), moe.Linear(d, inter, T, activation=moe.MOE_ACT_GELU, training=True)
    down = moe.Linear(inter, d, T, training=True)
    x, nw, nb = n(T, d), n(d), n(d)
    uw, ub, dw, db = n(inter, d, scale=d ** -0.5), n(inter), n(d, inter, scale=inter ** -0.5), n(d)
    dout = n(T, d)

    def step():
        y, s = norm.forward(x, None, nw, nb)
        h, pre = up.forward(y, uw, ub, save=True)
        out = down.forward(h, dw, db, s)
        dh, gdw, gdb = down.backward(h, None, dw, db, dout)
        dy, guw, gub = up.backward(y, pre, uw, ub, dh)
        return [out, gdw, gdb, guw, gub, *norm.backward(s, nw, dy, dout)]

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    x.copy_(n(T, d))
    dout.copy_(n(T, d))
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(got, step()))
    assert up.status() == moe.MOE_OK and down.status() == moe.MOE_OK
