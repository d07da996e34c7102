"""The mx8 block on data that determines the codes and scales of h (ffn_mx_case.py)."""
import pytest
import torch

import expert_routed_ffn_moe_gb300 as moe
import ffn_case as fc
import ffn_mx_case as mc
from test_gpu_ffn import ACTS, near

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,d,I", mc.SHAPES)
@pytest.mark.parametrize("name", sorted(ACTS))
def test_h_is_held_in_mx8(T, d, I, name):
    x, gu, dn = mc.operands(T, d, I, T + d + I, "cuda")
    q = [moe.moe_quantize_mx(t) for t in (x, gu, dn)]
    for (codes, scales), t in zip(q, (x, gu, dn)):
        assert torch.equal(fc.dequantize(codes, scales), t.to(mc.D))
    op = moe.GatedFfn(d, I, T + 3, activation=ACTS[name], weight_format=moe.MOE_W_MX8)
    y = op.forward(*q)
    assert op.status() == moe.MOE_OK
    near(y, *mc.forward(x, gu, dn, name == "gelu"), "y")
    # the scales of rows and groups that a larger call left in the workspace reach no row of a smaller one
    if T > 1:
        y1 = op.forward((q[0][0][:1].contiguous(), moe.moe_quantize_mx(x[:1].contiguous())[1]), q[1], q[2])
        near(y1, *mc.forward(x[:1], gu, dn, name == "gelu"), "y of one row")
    assert op.status() == moe.MOE_OK
