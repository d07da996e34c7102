"""Calls of the feed-forward block and the norm in unusual order or company."""
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
