"""Backward calls without rows (no GPU: they launch nothing)."""
import ctypes

import pytest

import expert_routed_ffn_moe_gb300 as moe


@pytest.mark.parametrize("ws", [None, ctypes.c_void_p(16)])
def test_no_rows_with_dx_alone(ws):
    # the dx of no rows is an empty tensor, whose address is NULL
    moe.build()
    L, a, B = moe.lib(), ctypes.c_void_p(16), moe.MOE_BF16
    assert L.moe_add_norm_backward(None, a, None, None, B, B, 0, 64, 1e-6, None, None, ws, None) == moe.MOE_OK
    assert L.moe_add_norm_backward(a, a, a, None, B, B, 1, 64, 1e-6, None, None, ws, None) == moe.MOE_ERR_ARG
