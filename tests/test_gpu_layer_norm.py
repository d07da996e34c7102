"""The layer norm and its gradients against their definitions in 64 bits (bounds: ops_case.py)."""
import pytest
import torch

import expert_routed_ffn_moe_gb300 as moe
import ops_case as oc
from test_gpu_ffn import BF, F32, gen, near, normal

pytestmark = pytest.mark.gpu
EPS = 1e-5
SIZES = [(1, 2048), (1, 1), (3, 7), (5, 8), (130, 31), (64, 96), (257, 255), (33, 1000), (300, 512), (300, 513),
         (17, 1999), (9, 2056), (700, 1024), (40, 4096), (7, 5001), (3, 8192), (2, 9001), (9, 16377), (2, 16384)]


def rows(g, T, d, dtype=BF):
    """Rows off centre, with a few large channels; one of padding and one of equal values where there are more."""
    v = torch.randn(T, d, generator=g, device="cuda") * torch.where(
        torch.rand(d, generator=g, device="cuda") < 0.01, 20.0, 1.0) + 3 * torch.randn(T, 1, generator=g, device="cuda")
    if T > 2:
        v[1], v[2] = 0, 1.5
    return v.to(dtype)


@pytest.mark.parametrize("T,d", SIZES)
@pytest.mark.parametrize("xt,st,yt,wt", [(BF, BF, BF, BF), (BF, F32, BF, F32), (F32, F32, F32, BF), (F32, BF, F32, F32)])
def test_matches_definition(T, d, xt, st, yt, wt):
    g = gen(T * 100003 + d)
    x, res = normal(g, T, d, dtype=xt), rows(g, T, d, st)
    if T > 2:
        x[1], x[2] = 0, 0
    w, b = normal(g, d, dtype=wt), normal(g, d, dtype=wt)
    y, s = moe.LayerNorm(d, EPS).forward(x, res, w, b, y_dtype=moe.MOE_BF16 if yt == BF else moe.MOE_F32)
    assert y.dtype == yt and s.dtype == st
    want = oc.layer_norm(x, res, w, b, EPS, st, yt)
    near(s, *want["s"], "s")
    near(y, *want["y"], "y")


@pytest.mark.parametrize("T,d", SIZES)
@pytest.mark.parametrize("dt,wt,with_ds", [(BF, BF, True), (F32, F32, True), (BF, F32, False), (F32, BF, False)])
def test_gradients_match_definition(T, d, dt, wt, with_ds):
    g = gen(T * 100003 + d + 1)
    s, dy = rows(g, T, d, dt), normal(g, T, d, dtype=dt)
    ds = normal(g, T, d, dtype=dt) if with_ds else None
    w = normal(g, d, dtype=wt)
    got = moe.LayerNorm(d, EPS).backward(s, w, dy, ds)
    want = oc.layer_norm_backward(s, w, dy, ds, EPS, wt)
    for v, name in zip(got, ("dx", "dweight", "dbias")):
        near(v, *want[name], name)


@pytest.mark.parametrize("T,d,dt", [(5000, 640, BF), (2000, 2051, F32), (1300, 4096, BF), (900, 6000, F32), (400, 12288, BF),
                                    (6007, 129, BF), (3001, 1021, BF), (1201, 4087, F32), (700, 8190, BF), (500, 16377, F32)])
def test_blocks_that_walk_several_rows(T, d, dt):
    g = gen(T + d)
    s, dy, ds = rows(g, T, d, dt), normal(g, T, d, dtype=dt), normal(g, T, d, dtype=dt)
    w, b = normal(g, d), normal(g, d)
    op = moe.LayerNorm(d, EPS)
    y, kept = op.forward(s, ds, w, b, y_dtype=moe.MOE_F32)
    want = oc.layer_norm(s, ds, w, b, EPS, dt, F32)
    near(kept, *want["s"], "s")
    near(y, *want["y"], "y")
    got = op.backward(s, w, dy, ds)
    want = oc.layer_norm_backward(s, w, dy, ds, EPS, BF)
    for v, name in zip(got, ("dx", "dweight", "dbias")):
        near(v, *want[name], name)
    again = op.backward(s, w, dy, ds)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


def test_gradients_match_differences():
    T, d = 6, 40
    g = gen(9)
    x, w, b, dy = (normal(g, *sh, dtype=F32) for sh in ((T, d), (d,), (d,), (T, d)))
    op = moe.LayerNorm(d, EPS)
    dx, dw, db = op.backward(x, w, dy)

    def loss(x, w, b):
        return (oc.layer_norm(x, None, w, b, EPS, F32, F32)["y"][0] * dy.to(oc.D)).sum()

    for t, grad, at in ((0, dx, (2, 7)), (0, dx, (5, 39)), (1, dw, (3,)), (2, db, (39,))):
        h = 1e-4
        args = [v.to(oc.D) for v in (x, w, b)]
        args[t][at] += h
        up = loss(*args)
        args[t][at] -= 2 * h
        slope = float((up - loss(*args)) / (2 * h))
        # the difference is off by h^2 / 6 of a third derivative, below 1e-6 here; fp32 by some 1e-5 of terms near one
        assert abs(slope - float(grad[at])) < 1e-4


def test_options_in_place_and_offsets_past_31_bits():
    g = gen(5)
    x, w, b = rows(g, 30, 520), normal(g, 520), normal(g, 520)
    op = moe.LayerNorm(520, EPS)
    y, s = op.forward(x, None, w, b)
    assert s is x
    near(y, *oc.layer_norm(x, None, w, b, EPS, BF, BF)["y"], "no residual")
    copy = torch.empty_like(x)
    assert op.forward(x, None, w, b, s_out=copy)[1] is copy and torch.equal(copy, x)
    near(op.forward(x, None, None, None)[0], *oc.layer_norm(x, None, None, None, EPS, BF, BF)["y"], "no weight")
    near(op.forward(x, None, w)[0], *oc.layer_norm(x, None, w, None, EPS, BF, BF)["y"], "no bias")
    near(op.forward(x, None, None, b)[0], *oc.layer_norm(x, None, None, b, EPS, BF, BF)["y"], "bias alone")
    got = op.backward(x, None, y)
    for v, name in zip(got, ("dx", "dweight", "dbias")):
        near(v, *oc.layer_norm_backward(x, None, y, None, EPS, F32)[name], name)
    # s over the residual, y over x, dx over dy
    L, B, F, p = moe.lib(), moe.MOE_BF16, moe.MOE_F32, lambda t: t.data_ptr()
    for d in (520, 519):
        x, res, w, b = rows(g, 30, d), rows(g, 30, d, F32), normal(g, d), normal(g, d)
        want = oc.layer_norm(x, res, w, b, EPS, F32, BF)
        xx, rr = x.clone(), res.clone()
        assert L.moe_layer_norm(p(xx), B, p(rr), F, p(w), p(b), B, 30, d, EPS, p(rr), p(xx), B, None) == moe.MOE_OK
        near(rr, *want["s"], "s in place")
        near(xx, *want["y"], "y in place")
        dy = x.clone()
        assert L.moe_layer_norm_backward(p(x), p(w), p(dy), None, B, B, 30, d, EPS, p(dy), None, None, None,
                                         None) == moe.MOE_OK
        near(dy, *oc.layer_norm_backward(x, w, x, None, EPS, BF)["dx"], "dx over dy")
    T, d = 140001, 16377
    x = torch.zeros(T, d, dtype=BF, device="cuda")
    x[-1] = normal(g, d)
    w, b = normal(g, d), torch.zeros(d, dtype=BF, device="cuda")
    y, _ = moe.LayerNorm(d, EPS).forward(x, None, w, b)
    near(y[-1:], *oc.layer_norm(x[-1:], None, w, b, EPS, BF, BF)["y"], "last row")
    assert not y[:1000].any()


def test_wanted_gradients_do_not_change_one_another():
    g = gen(8)
    T, d = 200, 3000
    s, dy, w = rows(g, T, d), normal(g, T, d), normal(g, d)
    L, B, p = moe.lib(), moe.MOE_BF16, lambda t: None if t is None else t.data_ptr()
    all_ = moe.LayerNorm(d, EPS).backward(s, w, dy)
    ws = torch.empty(L.moe_layer_norm_workspace(d), dtype=torch.uint8, device="cuda")
    for want in ((1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 0, 1), (0, 1, 1)):
        out = [torch.empty_like(t) if k else None for t, k in zip(all_, want)]
        assert L.moe_layer_norm_backward(p(s), p(w), p(dy), None, B, B, T, d, EPS, *map(p, out), p(ws), None) == moe.MOE_OK
        for a, b in zip(out, all_):
            assert a is None or torch.equal(a, b)


def test_nan_and_infinity_stay_in_their_rows():
    g = gen(6)
    for d in (256, 255):
        x, w = normal(g, 6, d), normal(g, d)
        x[2, 7], x[4, 9] = float("nan"), float("inf")
        y, _ = moe.LayerNorm(d).forward(x, None, w)
        bad = torch.isnan(y)
        assert bad[2].all() and bad[4].any() and not bad[[0, 1, 3, 5]].any()
        dx, _, _ = moe.LayerNorm(d).backward(x, w, x)
        bad = torch.isnan(dx)
        assert bad[2].all() and not bad[[0, 1, 3, 5]].any()


def test_no_rows_streams_and_graphs():
    g = gen(7)
    d = 264
    op = moe.LayerNorm(d, EPS)
    w, b = normal(g, d), normal(g, d)
    z = torch.empty(0, d, dtype=BF, device="cuda")
    y, _ = op.forward(z, z, w, b)
    dx, dw, db = op.backward(z, w, z)
    assert y.shape == dx.shape == (0, d) and not dw.any() and not db.any()
    x, res = normal(g, 50, d), normal(g, 50, d)
    y0, s0 = op.forward(x, res, w, b)
    g0 = op.backward(s0, w, x, res)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y1, s1 = op.forward(x, res, w, b, stream=side)
    g1 = op.backward(s1, w, x, res, stream=side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y2, s2 = op.forward(x, res, w, b)
        g2 = op.backward(s2, w, x, res)
    x.copy_(normal(g, 50, d))
    graph.replay()
    y3, s3 = op.forward(x, res, w, b)
    g3 = op.backward(s3, w, x, res)
    for a, c in zip((y1, s1, *g1), (y0, s0, *g0)):
        assert torch.equal(a, c)
    for a, c in zip((y2, s2, *g2), (y3, s3, *g3)):
        assert torch.equal(a, c)
