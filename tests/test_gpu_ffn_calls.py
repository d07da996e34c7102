"""Calls of the feed-forward block and the norm in unusual order or company."""
import pytest
import torch

import expert_routed_ffn_moe_gb300 as moe
from test_gpu_ffn import BF

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
