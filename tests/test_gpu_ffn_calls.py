"""Calls of the feed-forward block and the norm in unusual order or company."""
import importlib.util
import os
import threading

import pytest
import torch

import expert_routed_ffn_moe_gb300 as moe
import ffn_case as fc
from test_gpu_ffn import BF, gen, near, norm_bound, normal

pytestmark = pytest.mark.gpu


def test_no_rows_and_dx_alone():
    # (frozen weights: only the input's gradient is wanted, and an empty tensor has no address)
    d, I = 64, 48
    z = lambda *s: torch.empty(*s, dtype=BF, device="cuda")  # noqa: E731
    op = moe.GatedFfn(d, I, 8, training=True)
    gu, dn, w = z(2 * I, d).normal_(), z(d, I).normal_(), z(d).normal_()
    dx, dgu, dd = op.backward(z(0, d), z(0, 2 * I), gu, dn, z(0, d), None, False, False)
    assert dx.shape == (0, d) and dgu is None and dd is None
    moe.moe_add_norm_backward(z(0, d), w, z(0, d), None, 1e-6, z(0, d), None, None)
    with pytest.raises(moe.MoeError) as e:  # with rows it stays an error to want nothing
        op.backward(z(2, d), z(2, 2 * I), gu, dn, z(2, d), False, False, False)
    assert e.value.code == moe.MOE_ERR_ARG


def test_functions_take_a_stream():
    g = gen(40)
    x, w = normal(g, 20, 256), normal(g, 256)
    y0, s0 = moe.AddNorm(256).forward(x, x, w)
    dx0, dw0 = moe.AddNorm(256).backward(s0, w, x)
    y, s, dx, dw = (torch.empty_like(t) for t in (y0, s0, dx0, dw0))
    ws = torch.empty(moe.lib().moe_add_norm_workspace(256), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    moe.moe_add_norm(x, x, w, 1e-6, s, y, stream=side)
    moe.moe_add_norm_backward(s, w, x, None, 1e-6, dx, dw, ws, stream=side)
    torch.cuda.synchronize()
    for a, b in zip((y, s, dx, dw), (y0, s0, dx0, dw0)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("what,widths", [("forward", (12301, 16301)), ("backward", (6201, 8001))])
def test_widths_of_one_kernel_from_several_threads(what, widths):
    # both widths of a pair run on the same kernel and need different amounts of shared memory, above 48 KB
    g = gen(41)
    failed, rounds = [], 1500

    def work(d):
        try:
            op, st = moe.AddNorm(d), torch.cuda.Stream()
            with torch.cuda.stream(st):
                x, w = normal(g, 3, d), normal(g, d)
                call = (lambda: op.forward(x, x, w)) if what == "forward" else (lambda: op.backward(x, w, x))
                want = [t.clone() for t in call()]
                start.wait()
                for _ in range(rounds):
                    got = call()
                assert all(torch.equal(a, b) for a, b in zip(got, want))
        except Exception as e:
            failed.append(repr(e))
            start.abort()

    start = threading.Barrier(len(widths))
    threads = [threading.Thread(target=work, args=(d,)) for d in widths]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed


@pytest.mark.parametrize("rows,cols", [(5, 64), (130, 160)])
def test_quantize_into_one_given_output(rows, cols):
    v = normal(gen(42), rows, cols)
    codes, scales = moe.moe_quantize_mx(v)
    c, s = torch.zeros_like(codes), torch.zeros_like(scales)
    got = moe.moe_quantize_mx(v, codes=c)
    assert got[0] is c and torch.equal(c.view(torch.uint8), codes.view(torch.uint8)) and torch.equal(got[1], scales)
    got = moe.moe_quantize_mx(v, scales=s)
    assert got[1] is s and torch.equal(s, scales) and torch.equal(got[0].view(torch.uint8), codes.view(torch.uint8))


def test_example_names_a_wait_that_ran_out(monkeypatch):
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "dense_block.py")
    spec = importlib.util.spec_from_file_location("dense_block", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    left = [moe.MOE_ERR_TIMEOUT]  # (reading the status clears it)
    monkeypatch.setattr(moe.GatedFfn, "status", lambda self: left.pop() if left else moe.MOE_OK)
    with pytest.raises(RuntimeError, match=moe.moe_strerror(moe.MOE_ERR_TIMEOUT)):
        ex.train(64, 64, 8, 1)


@pytest.mark.parametrize("T", [1, 24])
def test_wait_limit_does_not_count_the_kernel_before(T):
    # The block before ends with one long tile on a few SMs (8 columns, 2^20 neurons: ~1 ms) and lets what follows
    # start beside it; the limit is far above what the small block itself takes and below that.
    g = gen(43)
    long_d, long_I, d, I = 8, 1 << 20, 256, 512
    slow = moe.GatedFfn(long_d, long_I, 100, training=True)
    a = normal(g, 100, long_d), normal(g, 2 * long_I, long_d), normal(g, long_d, long_I, scale=2.0 ** -10)
    ffn = moe.GatedFfn(d, I, T, training=True)
    x, dy = normal(g, T, d), normal(g, T, d)
    gu, dn = normal(g, 2 * I, d, scale=0.06), normal(g, d, I, scale=0.04)
    want, pre = ffn.forward(x, gu, dn, save=True)
    grads = ffn.backward(x, pre, gu, dn, dy)
    y = torch.empty_like(want)
    outs = [torch.empty_like(t) for t in grads]
    slow_y = torch.empty_like(a[0])
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    slow.forward(*a, y=slow_y)
    torch.cuda.synchronize()
    begin.record()
    slow.forward(*a, y=slow_y)
    end.record()
    torch.cuda.synchronize()
    took = begin.elapsed_time(end)
    assert took > 0.6, f"the block before took {took} ms"
    moe.moe_ffn_set_spin_limit(ffn.ctx, 200_000)
    for _ in range(3):
        y.zero_()
        torch.cuda.synchronize()
        slow.forward(*a, y=slow_y)
        ffn.forward(x, gu, dn, y=y)
        assert ffn.status() == moe.MOE_OK
        assert torch.equal(y, want)
        slow.forward(*a, y=slow_y)
        ffn.backward(x, pre, gu, dn, dy, *outs)
        assert ffn.status() == moe.MOE_OK
        assert all(torch.equal(p, q) for p, q in zip(outs, grads))
    assert slow.status() == moe.MOE_OK


# ------------------------------------------------------------------ few tokens: norm -> block -> norm ...
def chain_of(T, d, I, mx, seed, layers=3):
    """A chain of `layers` norms and blocks on fixed inputs, and its definition in steps."""
    g = gen(seed)
    x, res = normal(g, T, d), normal(g, T, d)
    w = [normal(g, d) for _ in range(layers + 1)]
    gu = [normal(g, 2 * I, d, scale=d ** -0.5) for _ in range(layers)]
    dn = [normal(g, d, I, scale=I ** -0.5) for _ in range(layers)]
    if mx:
        gu, dn = [moe.moe_quantize_mx(t) for t in gu], [moe.moe_quantize_mx(t) for t in dn]
    op = moe.AddNorm(d)
    ffn = moe.GatedFfn(d, I, max(T, 8), weight_format=moe.MOE_W_MX8 if mx else moe.MOE_W_BF16)
    form = moe.MOE_MX8 if mx else moe.MOE_BF16

    def run():
        steps, s, out = [], res, x
        for i in range(layers):
            rows, s = op.forward(out, s, w[i], y_dtype=form)
            out = ffn.forward(rows, gu[i], dn[i])
            steps.append((rows, s, out))
        steps.append(op.forward(out, s, w[layers]))
        return steps

    def check(steps):  # each step from the inputs that it had
        s, out = res, x
        for i in range(layers):
            rows, s1, out1 = steps[i]
            s0, y0 = fc.norm(out, s, w[i], 1e-6)
            near(s1, s0, fc.HALF * s0.abs(), f"s {i}")
            if mx:
                y, b = fc.forward_mx(rows, gu[i], dn[i], False)
            else:
                near(rows, y0, norm_bound(y0, fc.HALF), f"norm {i}")
                _, _, y, b = fc.forward(rows, gu[i], dn[i], False)
            near(out1, y, b, f"block {i}")
            s, out = s1, out1
        y0 = fc.norm(out, s, w[layers], 1e-6)[1]
        near(steps[layers][0], y0, norm_bound(y0, fc.HALF), "last norm")

    return run, check, (x, res), ffn


def flat(t):
    return [q for p in t for q in flat(p)] if isinstance(t, (list, tuple)) else [t]


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("T,d,I", [(1, 2048, 8192), (1, 1024, 2816), (9, 512, 1024), (17, 2048, 512), (40, 4096, 2752)])
def test_few_tokens_in_a_graph_between_norms(T, d, I, mx):
    run, check, inputs, ffn = chain_of(T, d, I, mx, 44)
    eager = run()
    check(eager)
    eager = [t.view(torch.uint8).clone() for t in flat(eager)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    got = [t.view(torch.uint8) for t in flat(got)]
    for _ in range(5):
        for t in got:
            t.zero_()
        graph.replay()
        graph.replay()  # (back to back: the first of a replay follows the last of the one before)
        for a, b in zip(got, eager):
            assert torch.equal(a, b)
    # other inputs through the same graph
    for t in inputs:
        t.copy_(normal(gen(45), *t.shape))
    graph.replay()
    for a, b in zip(got, flat(run())):
        assert torch.equal(a, b.view(torch.uint8))
    assert ffn.status() == moe.MOE_OK


@pytest.mark.parametrize("T", [1, 16, 33])
def test_few_tokens_read_weights_that_the_kernel_before_wrote(T):
    # (the second product asks for its weights before the first has ended)
    g = gen(46)
    d, I = (4096, 2752) if T > 32 else (1024, 2048)
    op, ffn = moe.AddNorm(d), moe.GatedFfn(d, I, T, training=True)
    sets = [(normal(g, T, d), normal(g, 2 * I, d, scale=d ** -0.5), normal(g, d, I, scale=I ** -0.5), normal(g, d))
            for _ in range(2)]
    res = normal(g, T, d)
    want = []
    for x, gu, dn, w in sets:
        y, s = op.forward(x, res, w)
        out, pre = ffn.forward(y, gu, dn, save=True)
        want.append([t.clone() for t in (out, pre) + ffn.backward(y, pre, gu, dn, x)])
        torch.cuda.synchronize()
    x, gu, dn, w = (torch.empty_like(t) for t in sets[0])
    got = []
    for i in range(20):
        for to, t in zip((x, gu, dn, w), sets[i % 2]):
            to.copy_(t)
        y, s = op.forward(x, res, w)
        out, pre = ffn.forward(y, gu, dn, save=True)
        got.append((out, pre) + ffn.backward(y, pre, gu, dn, x))
    for i, r in enumerate(got):
        for a, b in zip(r, want[i % 2]):
            assert torch.equal(a, b)
    assert ffn.status() == moe.MOE_OK


@pytest.mark.parametrize("mx", [False, True])
def test_few_tokens_beside_other_work(mx):
    # two chains on two streams, each with a context of its own
    chains = [chain_of(T, 1024, 2816, mx, 47 + T) for T in (1, 12)]
    want = [[t.view(torch.uint8).clone() for t in flat(run())] for run, *_ in chains]
    streams = [torch.cuda.Stream() for _ in chains]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, (run, *_) in enumerate(chains):
            with torch.cuda.stream(streams[i]):
                got[i].append(run())
    torch.cuda.synchronize()
    for i in range(2):
        for r in got[i]:
            for a, b in zip(flat(r), want[i]):
                assert torch.equal(a.view(torch.uint8), b)
        assert chains[i][3].status() == moe.MOE_OK
