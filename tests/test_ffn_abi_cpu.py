"""Host-side checks of the feed-forward block's and the norm's entry points, and
the mx8 definitions that the tests use (no GPU)."""
import ctypes
import os
import re

import pytest
import torch

import expert_routed_ffn_moe_gb300 as moe
import ffn_case as fc


@pytest.fixture(scope="module")
def lib():
    moe.build()
    return moe.lib()


def test_binding_config_matches_header():
    hdr = open(moe.HEADER).read()
    body = re.search(r"typedef struct moe_ffn_config \{(.*?)\} moe_ffn_config;", hdr, re.S).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    assert [n for n, _ in moe.moe_ffn_config._fields_] == re.findall(r"\bint\s+(\w+)\s*;", body)
    for name in ("MOE_MX8", "MOE_W_MX8", "MOE_ACT_SILU", "MOE_ACT_GELU"):
        assert int(re.search(rf"#define {name} (\d+)", hdr).group(1)) == getattr(moe, name)


@pytest.mark.parametrize("kw,code", [
    (dict(d=0), moe.MOE_ERR_ARG), (dict(inter=-8), moe.MOE_ERR_ARG), (dict(max_tokens=0), moe.MOE_ERR_ARG),
    (dict(activation=2), moe.MOE_ERR_ARG), (dict(weight_format=moe.MOE_W_Q4G64), moe.MOE_ERR_ARG),
    (dict(training=2), moe.MOE_ERR_ARG), (dict(d=68), moe.MOE_ERR_UNSUPPORTED), (dict(inter=4), moe.MOE_ERR_UNSUPPORTED),
    (dict(weight_format=moe.MOE_W_MX8, d=72), moe.MOE_ERR_UNSUPPORTED),
    (dict(weight_format=moe.MOE_W_MX8, training=1), moe.MOE_ERR_UNSUPPORTED),
    (dict(max_tokens=1 << 30), moe.MOE_ERR_UNSUPPORTED),
])
def test_init_rejects_bad_configs_before_any_device_call(lib, kw, code):
    base = dict(d=64, inter=64, max_tokens=8, activation=0, weight_format=0, training=0)
    base.update(kw)
    h = ctypes.c_void_p()
    assert lib.moe_ffn_init(ctypes.byref(moe.moe_ffn_config(**base)), ctypes.byref(h)) == code
    assert not h.value


def test_null_and_bad_arguments(lib):
    h = ctypes.c_void_p()
    p = ctypes.c_void_p
    assert lib.moe_ffn_init(None, ctypes.byref(h)) == moe.MOE_ERR_ARG
    assert lib.moe_ffn_init(ctypes.byref(moe.moe_ffn_config(64, 64, 8, 0, 0, 0)), None) == moe.MOE_ERR_ARG
    assert lib.moe_ffn_forward(None, *[None] * 2, 1, *[None] * 7) == moe.MOE_ERR_ARG
    assert lib.moe_ffn_backward(None, None, None, 1, *[None] * 7) == moe.MOE_ERR_ARG
    assert lib.moe_ffn_status(None) == moe.MOE_ERR_ARG and lib.moe_ffn_launch_count(None) == 0
    lib.moe_ffn_destroy(None)
    B, F, M = moe.MOE_BF16, moe.MOE_F32, moe.MOE_MX8
    a = p(16)  # never dereferenced: the checks below answer first

    def norm(x=a, xt=B, st=B, w=a, wt=B, T=1, d=64, eps=1e-6, y=a, yt=B, ys=None):
        return lib.moe_add_norm(x, xt, None, st, w, wt, T, d, eps, None, y, yt, ys, None)

    assert norm(T=0) == moe.MOE_OK
    for kw in (dict(x=None), dict(w=None), dict(y=None), dict(xt=M), dict(st=9), dict(wt=M), dict(yt=3), dict(T=-1),
               dict(d=0), dict(eps=-1.0), dict(eps=float("nan")), dict(yt=M), dict(ys=a)):
        assert norm(**kw) == moe.MOE_ERR_ARG, kw
    assert norm(d=16385) == moe.MOE_ERR_UNSUPPORTED and norm(d=40, yt=M, ys=a) == moe.MOE_ERR_UNSUPPORTED
    assert norm(x=p(8)) == moe.MOE_ERR_ALIGN and norm(y=p(20)) == moe.MOE_ERR_ALIGN

    def grad(s=a, w=a, dy=a, dt=B, wt=B, T=1, d=64, eps=1e-6, dx=a, dw=a, ws=a):
        return lib.moe_add_norm_backward(s, w, dy, None, dt, wt, T, d, eps, dx, dw, ws, None)

    for kw in (dict(s=None), dict(w=None), dict(dy=None), dict(dt=M), dict(wt=5), dict(T=-1), dict(d=-2),
               dict(dx=None, dw=None), dict(ws=None)):
        assert grad(**kw) == moe.MOE_ERR_ARG, kw
    assert grad(d=20000) == moe.MOE_ERR_UNSUPPORTED and grad(dw=p(2)) == moe.MOE_ERR_ALIGN
    assert grad(T=0, dw=None) == moe.MOE_OK
    assert lib.moe_quantize_mx(a, M, 1, 32, a, a, None) == moe.MOE_ERR_ARG
    assert lib.moe_quantize_mx(a, F, 1, 40, a, a, None) == moe.MOE_ERR_UNSUPPORTED
    assert lib.moe_quantize_mx(a, F, 1, 32, None, a, None) == moe.MOE_ERR_ARG
    assert lib.moe_quantize_mx(a, F, 0, 32, None, None, None) == moe.MOE_OK


def test_scale_layout(lib):
    for rows, cols in ((1, 32), (128, 128), (129, 160), (300, 544)):
        n = moe.moe_mx_scale_bytes(rows, cols)
        at = fc.scale_index(rows, cols)
        assert n == -(-rows // 128) * -(-cols // 128) * 512
        assert at.max() < n and at.unique().numel() == at.numel()
    assert moe.moe_mx_scale_bytes(0, 64) == 0
    assert fc.scale_index(40, 160)[33, 4] == 512 + 1 * 16 + 1 * 4  # second tile, row 33, its first group


def test_mx8_definition():
    v = torch.zeros(1, 96)
    v[0, 3], v[0, 40], v[0, 41] = 448.0, -449.0, 1.0
    codes, scales = fc.quantize(v)
    assert [int(scales[i]) - 127 for i in (0, 1, 2)] == [0, 1, -127]
    back = fc.dequantize(codes, scales)
    assert back[0, 3] == 448 and back[0, 40] == -448 and back[0, 41] == 1 and not back[0, 64:].any()


@pytest.mark.parametrize("rows", [(1 << 30) + 1, (1 << 31) - 128, (1 << 31) - 1])
def test_more_rows_than_the_kernels_count_are_refused(lib, rows):
    a, B = ctypes.c_void_p(16), moe.MOE_BF16  # never dereferenced
    assert lib.moe_add_norm(a, B, None, B, a, B, rows, 1, 1e-6, None, a, B, None, None) == moe.MOE_ERR_UNSUPPORTED
    assert lib.moe_add_norm_backward(a, a, a, None, B, B, rows, 1, 1e-6, a, a, a, None) == moe.MOE_ERR_UNSUPPORTED
    assert lib.moe_quantize_mx(a, B, rows, 32, a, a, None) == moe.MOE_ERR_UNSUPPORTED


def test_sizes_past_an_int_are_refused_before_the_call():
    # (the C entries take ints: 2^32 + 1 rows would arrive there as one)
    t = torch.empty((1 << 32) + 1, 32, dtype=torch.bfloat16, device="meta")
    w = torch.empty(32, dtype=torch.bfloat16, device="meta")
    for call in (lambda: moe.moe_quantize_mx(t), lambda: moe.AddNorm(32).forward(t, None, w),
                 lambda: moe.AddNorm(32).backward(t, w, t)):
        with pytest.raises(ValueError, match="than an int holds"):
            call()
