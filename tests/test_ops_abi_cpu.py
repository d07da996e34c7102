"""Host-side checks of the layer norm's, the token sort's and the product's entry points, and the definitions that their
GPU tests use (no GPU)."""
import ctypes
import re

import pytest
import torch

import expert_routed_ffn_moe_gb300 as moe
import ops_case as oc

B, F, M = moe.MOE_BF16, moe.MOE_F32, moe.MOE_MX8
P = ctypes.c_void_p
A = P(16)  # never dereferenced: the checks answer first
OK, ARG, ALIGN, UNSUP = moe.MOE_OK, moe.MOE_ERR_ARG, moe.MOE_ERR_ALIGN, moe.MOE_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    moe.build()
    return moe.lib()


def test_binding_config_matches_header():
    hdr = open(moe.HEADER).read()
    body = re.search(r"typedef struct moe_linear_config \{(.*?)\} moe_linear_config;", hdr, re.S).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    assert [n for n, _ in moe.moe_linear_config._fields_] == re.findall(r"\bint\s+(\w+)\s*;", body)
    assert int(re.search(r"#define MOE_ACT_NONE (\d+)", hdr).group(1)) == moe.MOE_ACT_NONE


@pytest.mark.parametrize("kw,code", [
    (dict(in_features=0), ARG), (dict(out_features=-8), ARG), (dict(max_tokens=0), ARG), (dict(activation=3), ARG),
    (dict(training=2), ARG), (dict(in_features=68), UNSUP), (dict(out_features=4), UNSUP),
    (dict(in_features=(1 << 24) + 8), UNSUP), (dict(max_tokens=1 << 30), UNSUP),
])
def test_linear_init_rejects_bad_configs_before_any_device_call(lib, kw, code):
    h = P()
    c = moe.moe_linear_config(**dict(dict(in_features=64, out_features=64, max_tokens=8, activation=2, training=0), **kw))
    assert lib.moe_linear_init(ctypes.byref(c), ctypes.byref(h)) == code and not h.value
    assert lib.moe_linear_init(None, ctypes.byref(h)) == ARG and lib.moe_linear_init(ctypes.byref(c), None) == ARG


def test_linear_without_a_context(lib):
    assert lib.moe_linear_forward(None, A, 1, A, A, B, None, A, B, None, None) == ARG
    assert lib.moe_linear_backward(None, A, A, 1, A, A, B, A, A, A, B, None) == ARG
    assert lib.moe_linear_status(None) == ARG and lib.moe_linear_launch_count(None) == 0
    assert lib.moe_linear_set_spin_limit(None, 0) == ARG and lib.moe_linear_inject_stall(None, 1) == ARG
    lib.moe_linear_destroy(None)


def test_layer_norm_arguments(lib):
    def norm(x=A, xt=B, st=B, w=A, b=A, wt=B, T=1, d=64, eps=1e-6, y=A, yt=B):
        return lib.moe_layer_norm(x, xt, None, st, w, b, wt, T, d, eps, None, y, yt, None)

    assert norm(T=0) == OK
    for kw in (dict(x=None), dict(y=None), dict(xt=M), dict(st=9), dict(wt=M), dict(yt=M), dict(T=-1), dict(d=0),
               dict(eps=-1.0), dict(eps=float("nan"))):
        assert norm(**kw) == ARG, kw
    assert norm(d=16385) == UNSUP and norm(d=16378) == UNSUP and norm(d=16383) == UNSUP and norm(T=(1 << 30) + 1) == UNSUP
    for kw in (dict(x=P(8)), dict(w=P(20)), dict(b=P(2)), dict(y=P(24))):
        assert norm(**kw) == ALIGN, kw

    def grad(s=A, w=A, dy=A, dt=B, wt=B, T=1, d=64, eps=1e-6, dx=A, dw=A, db=A, ws=A):
        return lib.moe_layer_norm_backward(s, w, dy, None, dt, wt, T, d, eps, dx, dw, db, ws, None)

    for kw in (dict(s=None), dict(dy=None), dict(dt=M), dict(wt=5), dict(T=-1), dict(d=-2), dict(dx=None, dw=None, db=None),
               dict(ws=None), dict(ws=None, dw=None), dict(ws=None, db=None), dict(eps=-1.0)):
        assert grad(**kw) == ARG, kw
    assert grad(d=20000) == UNSUP and grad(dw=P(2)) == ALIGN and grad(T=0, dw=None, db=None) == OK
    assert lib.moe_layer_norm_workspace(0) == 0 and lib.moe_layer_norm_workspace(10) % 80 == 0


def test_token_sort_arguments(lib):
    def sort(idx=A, T=1, k=8, E=64, out=A):
        return lib.moe_sort_tokens(idx, T, k, E, out, out, out, out, None)

    for kw in (dict(idx=None), dict(T=-1), dict(k=0), dict(E=0)):
        assert sort(**kw) == ARG, kw
    for kw in (dict(k=33), dict(E=1025), dict(T=1 << 28)):
        assert sort(**kw) == UNSUP, kw
    assert sort(idx=P(4)) == ALIGN and sort(out=P(8)) == ALIGN
    assert lib.moe_sort_tokens(None, 0, 8, 64, None, None, None, None, None) == OK

    def dispatch(x=A, xt=B, slot=A, T=1, k=8, d=64, rows=A, rt=B, n=8):
        return lib.moe_dispatch(x, xt, slot, T, k, d, rows, rt, n, None)

    def combine(x=A, xt=B, slot=A, T=1, k=8, d=64, rows=A, rt=B, n=8):
        return lib.moe_combine(rows, rt, n, slot, A, T, k, d, A, x, xt, None)

    def grad(x=A, xt=B, slot=A, T=1, k=8, d=64, rows=A, rt=B, n=8, w=A, drows=A, dw=A):
        return lib.moe_combine_backward(x, xt, rows, rt, n, slot, w, T, k, d, drows, dw, None)

    for f in (dispatch, combine, grad):
        for kw in (dict(x=None), dict(slot=None), dict(rows=None), dict(xt=M), dict(rt=7), dict(T=-1), dict(k=0), dict(d=0),
                   dict(n=-1)):
            assert f(**kw) == ARG, (f, kw)
        for kw in (dict(k=33), dict(T=1 << 28), dict(T=1 << 20, k=1, d=1 << 20), dict(d=(1 << 24) + 1)):
            assert f(**kw) == UNSUP, (f, kw)
        for kw in (dict(x=P(8)), dict(slot=P(4)), dict(rows=P(24))):
            assert f(**kw) == ALIGN, (f, kw)
        assert f(T=0) == OK
    assert dispatch(n=0, rows=None) == OK
    assert grad(w=None) == ARG and grad(drows=None, dw=None) == ARG


def test_sizes_past_an_int_and_bad_handles_are_refused_before_the_call():
    t = torch.empty((1 << 32) + 1, 32, dtype=torch.bfloat16, device="meta")
    i = torch.empty((1 << 32) + 1, 4, dtype=torch.int32, device="meta")
    w = torch.empty(32, dtype=torch.bfloat16, device="meta")
    op = moe.TokenDispatch(8, 4)
    for call in (lambda: moe.LayerNorm(32).forward(t, None, w), lambda: moe.LayerNorm(32).backward(t, w, t),
                 lambda: op.dispatch(t, i), lambda: op.combine(t, i)):
        with pytest.raises(ValueError, match="than an int holds"):
            call()
    for bad in ((0, 4), (1025, 4), (8, 0), (8, 33)):
        with pytest.raises(ValueError, match="must be 1 to"):
            moe.TokenDispatch(*bad)


def test_sort_definition_on_a_case_worked_by_hand():
    idx = torch.tensor([[1, 0], [2, 1], [-1, 1], [1, 1]], dtype=torch.int32)
    counts, offsets, perm, slot = oc.sort(idx, 3)
    assert counts.tolist() == [1, 5, 1] and offsets.tolist() == [0, 1, 6, 7]
    assert perm.tolist() == [0, 0, 1, 2, 3, 3, 1] and slot.tolist() == [[1, 0], [6, 2], [-1, 3], [4, 5]]


@pytest.mark.parametrize("name", ["none", "silu", "gelu"])
def test_definitions_agree_with_automatic_differentiation(name):
    g = torch.Generator().manual_seed(1)
    n = lambda *s: torch.randn(*s, generator=g, dtype=oc.D)  # noqa: E731
    x, w, b, dy = n(5, 12).requires_grad_(), n(7, 12).requires_grad_(), n(7).requires_grad_(), n(5, 7)
    pre = x @ w.t() + b
    y = {"none": lambda v: v, "silu": torch.nn.functional.silu,
         "gelu": lambda v: torch.nn.functional.gelu(v, approximate="tanh")}[name](pre)
    want = torch.autograd.grad(y, (x, w, b), dy)
    assert torch.allclose(oc.linear(x, w, b, None, name, torch.float32)["y"][0], y)
    got = oc.linear_backward(x, pre, w, dy, name, torch.float32)
    assert all(torch.allclose(got[k][0], v) for k, v in zip(("dx", "dweight", "dbias"), want))
    s, lw, lb, dy = n(5, 12).requires_grad_(), n(12).requires_grad_(), n(12).requires_grad_(), n(5, 12)
    y = torch.nn.functional.layer_norm(s, (12,), lw, lb, 1e-5)
    want = torch.autograd.grad(y, (s, lw, lb), dy)
    assert torch.allclose(oc.layer_norm(s, None, lw, lb, 1e-5, torch.float32, torch.float32)["y"][0], y)
    got = oc.layer_norm_backward(s, lw, dy, None, 1e-5, torch.float32)
    assert all(torch.allclose(got[k][0], v) for k, v in zip(("dx", "dweight", "dbias"), want))
