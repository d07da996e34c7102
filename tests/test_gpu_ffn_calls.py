"""Calls of the feed-forward block and the norm in unusual order or company."""
import importlib.util
import os
import threading

import pytest
import torch

import expert_routed_ffn_moe_gb300 as moe
from test_gpu_ffn import BF, gen, normal

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
