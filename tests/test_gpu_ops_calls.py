"""Calls of the layer norm, the token sort and the product in unusual company."""
import threading

import pytest
import torch

import expert_routed_ffn_moe_gb300 as moe
from test_gpu_ffn import BF, F32, gen, normal

pytestmark = pytest.mark.gpu


def test_calls_side_by_side_from_several_threads():
    # each thread its own stream, sizes and contexts; kernels, their limits of shared memory and counters are shared
    failed, rounds = [], 200

    def work(i):
        try:
            g = gen(i)
            with torch.cuda.stream(torch.cuda.Stream()):
                d, E, k, T = (1999, 2048, 4096, 301)[i], (64, 600, 8, 1000)[i], (8, 2, 4, 1)[i], (100, 500, 1500, 9)[i]
                norm, sort = moe.LayerNorm(d), moe.TokenDispatch(E, k)
                lin = moe.Linear(256, 264, T, activation=moe.MOE_ACT_GELU, training=True)
                x, w = normal(g, T, d, dtype=F32 if i == 2 else BF), normal(g, d)
                idx = torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
                pw = torch.rand(T, k, generator=g, device="cuda")
                lx, lw, lb = normal(g, T, 256), normal(g, 264, 256, scale=0.06), normal(g, 264)

                def step():
                    y, s = norm.forward(x, x, w)
                    counts, offsets, perm, slot = sort.sort(idx)
                    rows = sort.dispatch(x, slot)
                    z, pre = lin.forward(lx, lw, lb, save=True)
                    return [y, s, *norm.backward(s, w, x), counts, offsets, perm, slot, rows,
                            sort.combine(rows, slot, pw, add=x), *sort.combine_backward(x, rows, slot, pw), z, pre,
                            *lin.backward(lx, pre, lw, lb, z)]

                want = [t.clone() for t in step()]
                start.wait()
                for _ in range(rounds):
                    got = step()
                torch.cuda.current_stream().synchronize()
                assert all(torch.equal(a, b) for a, b in zip(got, want)) and lin.status() == moe.MOE_OK
        except Exception as e:
            failed.append(repr(e))
            start.abort()

    start = threading.Barrier(4)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed


@pytest.mark.parametrize("T", [1, 3, 20, 200])
def test_a_waits_limit_does_not_count_the_kernel_before(T):
    # The product before ends with one long tile on a few SMs (8 outputs, 2^21 inputs) and lets what follows start beside
    # it; the limit is far above what the small product itself takes and below that.
    g = gen(T)
    slow = moe.Linear(1 << 21, 8, 100)
    a = normal(g, 100, 1 << 21), normal(g, 8, 1 << 21)
    lin = moe.Linear(256, 512, T, training=True)
    x, w, b, dy = normal(g, T, 256), normal(g, 512, 256), normal(g, 512), normal(g, T, 512)
    want = [lin.forward(x, w, b), *lin.backward(x, None, w, b, dy)]
    outs = [torch.empty_like(t) for t in want]
    slow_y = torch.empty(100, 8, dtype=BF, device="cuda")
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    slow.forward(*a, y=slow_y)
    torch.cuda.synchronize()
    begin.record()
    slow.forward(*a, y=slow_y)
    end.record()
    torch.cuda.synchronize()
    limit = int(begin.elapsed_time(end) * 1e6 / 4)  # ns
    assert limit > 50_000  # (the small products take some 20 us at most)
    moe.moe_linear_set_spin_limit(lin.ctx, limit)
    for _ in range(5):
        slow.forward(*a, y=slow_y)
        lin.forward(x, w, b, y=outs[0])
        slow.forward(*a, y=slow_y)
        lin.backward(x, None, w, b, dy, *outs[1:])
    assert lin.status() == moe.MOE_OK and slow.status() == moe.MOE_OK
    assert all(torch.equal(p, q) for p, q in zip(outs, want))


def test_an_output_of_one_call_is_the_next_ones_input_without_a_wait():
    # kernels come up while the one before still runs: every first read must follow it
    g = gen(9)
    T, d, k = 300, 512, 4
    norm, sort, lin = moe.LayerNorm(d), moe.TokenDispatch(32, k), moe.Linear(d, d, T * k, training=True)
    x, w = normal(g, T, d), normal(g, d)
    lw, lb = normal(g, d, d, scale=d ** -0.5), normal(g, d)
    pw = torch.rand(T, k, generator=g, device="cuda")
    idx = torch.randint(-1, 32, (T, k), generator=g, device="cuda", dtype=torch.int32)

    def chain(wait):
        h, out = x, []
        for _ in range(6):
            h, s = norm.forward(h, x, w)
            wait()
            _, _, _, slot = sort.sort(idx)
            wait()
            rows = sort.dispatch(h, slot, rows=torch.zeros(T * k, d, dtype=BF, device="cuda"))
            wait()
            rows = lin.forward(rows, lw, lb)
            wait()
            h = sort.combine(rows, slot, pw, add=s)
            wait()
            dr, dw = sort.combine_backward(h, rows, slot, pw, drows=torch.zeros_like(rows))
            wait()
            dx, gw, gb = lin.backward(rows, None, lw, lb, dr)
            wait()
            out += [h, dw, dx, gw, gb, *norm.backward(s, w, sort.dispatch_backward(dx, slot))]
            wait()
            # one token through the same weights, straight after they were written
            lw.copy_(lw * 0.5 + gw * 1e-3)
            out.append(lin.forward(h[:1], lw, lb))
            wait()
        return out

    before = lw.clone()
    want = [t.clone() for t in chain(torch.cuda.synchronize)]
    lw.copy_(before)
    got = chain(lambda: None)
    bits = {1: torch.uint8, 2: torch.int16, 4: torch.int32}  # (values that have grown past the type's range among them)
    assert all(torch.equal(*(t.view(bits[t.element_size()]) for t in pair)) for pair in zip(got, want))
