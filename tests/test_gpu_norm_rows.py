"""The norm and its gradients over more rows than blocks fit on the device, so
that every block walks several, against their definitions in 64 bits."""
import pytest
import torch

import expert_routed_ffn_moe_gb300 as moe
import ffn_case as fc
import test_gpu_ffn as base
from test_gpu_ffn import BF, F32, gen, near, normal

pytestmark = pytest.mark.gpu

# (T, d): at least three rows for every block (or warp, below 512 columns) that an SM of 2048 threads can hold
ROWS = [(30011, 75), (30011, 256), (29999, 301), (30011, 500), (30011, 504), (7507, 999), (7507, 1000), (7507, 1999), (7503, 2048),
        (3701, 4001), (3701, 4096), (1901, 5001), (1901, 8192), (941, 9001), (941, 12288), (941, 16383), (941, 16384)]


def threads_per_row(d):
    chunks = d // 8 if d % 8 == 0 else (d + 7) // 8 + 1
    return 32 if chunks <= 64 else 128 if chunks <= 256 else 256 if chunks <= 512 else 512 if chunks <= 1024 else 1024


@pytest.mark.parametrize("T,d", ROWS)
def test_blocks_walk_several_rows(T, d):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert T > 3 * sms * (2048 // threads_per_row(d))


@pytest.mark.parametrize("T,d", ROWS)
@pytest.mark.parametrize("xt,st,yt", [(BF, BF, BF), (BF, F32, BF), (F32, F32, F32), (F32, BF, F32)])
def test_norm_of_many_rows(T, d, xt, st, yt):
    base.test_norm_matches_definition(T, d, xt, st, yt)


@pytest.mark.parametrize("T,d", [(30011, 96), (30011, 512), (7507, 1024), (7503, 2080), (3701, 4096), (1901, 8192),
                                 (941, 16384)])
@pytest.mark.parametrize("st", [BF, F32])
def test_norm_to_mx8_of_many_rows(T, d, st):
    base.test_norm_to_mx8(T, d, st)


@pytest.mark.parametrize("T,d", ROWS)
@pytest.mark.parametrize("dt", [BF, F32])
def test_norm_backward_of_many_rows(T, d, dt):
    base.test_norm_backward_matches_formula(T, d, dt, dt == BF)


@pytest.mark.parametrize("T,d", ROWS)
@pytest.mark.parametrize("dt", [BF, F32])
def test_no_row_is_missing_from_the_weights_gradient(T, d, dt):
    # dy * n of every row is positive and about 1, so that a row left out or added twice is 1 / T of the sum.  With fp32
    # weights the result carries no rounding of its own.  The sum has at most T / 152 additions in a thread (a block or
    # more on each of 152 SMs), 4 over a block's warps, 38 over partial rows and 5 over a warp, each off by 2^-24 of the
    # sum, and n is right to 2^-20: T = 30011 gives 1.6e-5, half of a row's 3.3e-5.
    g = gen(T + d)
    sign = torch.where(torch.rand(T, d, generator=g, device="cuda") < 0.5, -1.0, 1.0)
    s, dy = sign.to(dt), sign.to(dt)
    w = normal(g, d, dtype=F32)
    _, dw = moe.AddNorm(d).backward(s, w, dy)
    dw0 = fc.norm_backward(s, w, dy, None, 1e-6)[1]
    tol = 2.0 ** -20 + (T / 152 + 50) * 2.0 ** -24
    assert tol * T < 0.5
    near(dw, dw0, tol * dw0, "dweight")
