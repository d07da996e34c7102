"""The dense gated feed-forward block, its gradients, its mx8 form and the norm
in front of it, against their definitions in 64 bits (bounds: ffn_case.py)."""
import pytest
import torch

import expert_routed_ffn_moe_gb300 as moe
import ffn_case as fc

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
ACTS = {"silu": moe.MOE_ACT_SILU, "gelu": moe.MOE_ACT_GELU}


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape, scale=1.0, dtype=BF):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def near(got, want, bound, what):
    got = got.to(fc.D)
    assert got.shape == want.shape, what
    bad = ~((got - want).abs() <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} values off, worst "
                           f"{float(((got - want).abs() / bound).max()):.2f} of its bound, first at "
                           f"{bad.nonzero()[0].tolist()}")


# ------------------------------------------------------------------ norm
def norm_bound(y, extra=0.0):
    return (2.0 ** -20 + extra) * y.abs() + 1e-30  # fp32: a sum of d squares, rsqrt, three products


@pytest.mark.parametrize("T,d", [(1, 2048), (1, 1), (3, 7), (5, 8), (130, 31), (64, 96), (257, 255), (33, 1000),
                                 (17, 1999), (9, 2056), (40, 4096), (7, 5001), (3, 8192), (2, 9000), (2, 16383),
                                 (2, 16384)])
@pytest.mark.parametrize("xt,st,yt", [(BF, BF, BF), (BF, F32, BF), (F32, F32, F32), (F32, BF, F32)])
def test_norm_matches_definition(T, d, xt, st, yt):
    g = gen(T * 100003 + d)
    x, res = normal(g, T, d, dtype=xt), normal(g, T, d, scale=3, dtype=st)
    w = normal(g, d, dtype=BF if d % 2 else F32)
    if T > 2:
        x[1], res[1] = 0, 0  # a row of padding
    y, s = moe.AddNorm(d, 1e-5).forward(x, res, w, y_dtype=moe.MOE_BF16 if yt == BF else moe.MOE_F32)
    s0, y0 = fc.norm(x, res, w, 1e-5)
    near(s, s0, (fc.HALF if st == BF else 2.0 ** -24) * s0.abs(), "s")
    near(y, y0, norm_bound(y0, fc.HALF if yt == BF else 0.0), "y")


def test_norm_without_residual_in_place_and_large_rows():
    g = gen(5)
    x, w = normal(g, 30, 520), normal(g, 520)
    op = moe.AddNorm(520)
    y, s = op.forward(x, None, w)
    assert torch.equal(s, x)
    near(y, fc.norm(x, None, w, 1e-6)[1], norm_bound(fc.norm(x, None, w, 1e-6)[1], fc.HALF), "y")
    res = normal(g, 30, 520, dtype=F32)
    s0, y0 = fc.norm(x, res, w, 1e-6)
    xx = x.clone()
    moe.moe_add_norm(xx, res, w, 1e-6, res, xx)  # y over x, s over the residual
    near(res, s0, 2.0 ** -24 * s0.abs(), "s in place")
    near(xx, y0, norm_bound(y0, fc.HALF), "y in place")
    # element offsets past 2^31
    T, d = 140001, 16383
    x = torch.zeros(T, d, dtype=BF, device="cuda")
    x[-1] = normal(g, d)
    w = normal(g, d)
    y, s = moe.AddNorm(d).forward(x, None, w)
    near(y[-1:], fc.norm(x[-1:], None, w, 1e-6)[1], norm_bound(fc.norm(x[-1:], None, w, 1e-6)[1], fc.HALF), "last row")
    assert not y[:1000].any()


def test_norm_nan_and_infinity_stay_in_their_rows():
    g = gen(6)
    x, w = normal(g, 6, 256), normal(g, 256)
    x[2, 7], x[4, 9] = float("nan"), float("inf")
    y, _ = moe.AddNorm(256).forward(x, None, w)
    bad = torch.isnan(y)
    assert bad[2].all() and bad[4, 9] and not bad[[0, 1, 3, 5]].any()
    (codes, scales), _ = moe.AddNorm(256).forward(x, None, w, y_dtype=moe.MOE_MX8)
    at = fc.scale_index(6, 256, "cuda")
    assert (scales[at[2]] == 255).all() and scales[at[4, 0]] == 255 and not (scales[at[[0, 1, 3, 5]]] == 255).any()
    near(fc.dequantize(codes, scales)[[0, 1, 3, 5]], y[[0, 1, 3, 5]].to(fc.D),
         0.08 * y[[0, 1, 3, 5]].to(fc.D).abs() + 0.01, "rows beside them")


@pytest.mark.parametrize("T,d", [(1, 2048), (1, 32), (5, 160), (127, 256), (128, 384), (129, 1024), (300, 2080),
                                 (4, 4096), (3, 16384)])
@pytest.mark.parametrize("st", [BF, F32])
def test_norm_to_mx8(T, d, st):
    g = gen(T + d)
    x, res, w = normal(g, T, d), normal(g, T, d, dtype=st), normal(g, d)
    if T > 2:
        x[1], res[1] = 0, 0
        x[2, :32], res[2, :32] = 0, 0  # a group of zeros
    (codes, scales), _ = moe.AddNorm(d).forward(x, res, w, y_dtype=moe.MOE_MX8)
    y0 = fc.norm(x, res, w, 1e-6)[1]
    e = fc.exponents(y0)
    at = fc.scale_index(T, d, "cuda")
    got_e = scales[at.view(-1)].view(T, -1).to(fc.D) - 127
    top = y0.reshape(T, -1, 32).abs().max(-1).values
    clear = (top == 0) | ((torch.log2(top / 448) - torch.log2(top / 448).round()).abs() > 1e-5)
    assert torch.equal(got_e[clear], e[clear])
    rest = torch.ones_like(scales, dtype=torch.bool)
    rest[at.view(-1)] = False
    assert not scales[rest].any()  # bytes past the matrix
    unit = torch.exp2(torch.maximum(got_e, e)).repeat_interleave(32, 1)
    near(fc.dequantize(codes, scales), y0, (2.0 ** -4 + 2.0 ** -20) * y0.abs() + 2.0 ** -10 * unit, "values")


@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 64), (128, 128), (130, 160), (1000, 544), (64, 8192)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_quantize_is_exact(rows, cols, dtype):
    g = gen(rows + cols)
    v = torch.randn(rows, cols, generator=g, device="cuda")
    v = (v * torch.exp2(torch.randint(-140, 100, (rows, 1), generator=g, device="cuda").float())).to(dtype)
    v.view(-1)[:32] = 0
    v.view(-1)[5] = 448.0
    v.view(-1)[-1] = 1.76 * 2.0 ** 8
    codes, scales = moe.moe_quantize_mx(v)
    q, s = fc.quantize(v)
    assert torch.equal(codes.view(torch.uint8), q.view(torch.uint8))
    assert torch.equal(scales, s)


@pytest.mark.parametrize("T,d", [(1, 2048), (1, 1), (3, 7), (700, 31), (64, 96), (257, 255), (33, 1000), (1300, 256),
                                 (17, 1999), (40, 4096), (7, 5001), (3, 8192), (2, 16383), (2, 16384)])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("with_ds", [True, False])
def test_norm_backward_matches_formula(T, d, dt, with_ds):
    g = gen(T * 7 + d)
    s, dy = normal(g, T, d, scale=2, dtype=dt), normal(g, T, d, dtype=dt)
    ds = normal(g, T, d, dtype=dt) if with_ds else None
    w = normal(g, d, dtype=dt)
    if T > 2:
        s[1] = 0
    dx, dw = moe.AddNorm(d, 1e-4).backward(s, w, dy, ds)
    dx0, dw0 = fc.norm_backward(s, w, dy, ds, 1e-4)
    r = torch.rsqrt(s.to(fc.D).square().mean(-1, keepdim=True) + 1e-4)
    n, gg = s.to(fc.D) * r, dy.to(fc.D) * w.to(fc.D)
    # fp32: terms of either sum are right to 2^-20, the mean to 2^-20 of its terms' magnitudes
    terms = r * (gg.abs() + n.abs() * (gg * n).abs().mean(-1, keepdim=True)) + (ds.to(fc.D).abs() if with_ds else 0)
    rnd = fc.HALF if dt == BF else 2.0 ** -24
    near(dx, dx0, rnd * dx0.abs() + 2.0 ** -20 * terms + 1e-30, "dx")
    near(dw, dw0, rnd * dw0.abs() + (2.0 ** -20 + T * 2.0 ** -24) * (dy.to(fc.D) * n).abs().sum(0) + 1e-30, "dweight")


@pytest.mark.parametrize("d", [64, 75, 301, 999])
def test_norm_backward_nan_stays_in_its_row(d):
    # (rows of odd width share 16-byte windows with their neighbours)
    g = gen(13)
    T = 9
    s, dy, ds, w = (normal(g, *sh, dtype=F32) for sh in ((T, d), (T, d), (T, d), (d,)))
    clean, _ = moe.AddNorm(d).backward(s, w, dy, ds)
    for bad in (float("nan"), float("inf")):
        s2, dy2 = s.clone(), dy.clone()
        s2[3, 0], dy2[5, d - 1] = bad, bad
        dx, dw = moe.AddNorm(d).backward(s2, w, dy2, ds)
        keep = [0, 1, 2, 4, 6, 7, 8]
        assert torch.equal(dx[keep], clean[keep])
        assert not torch.isfinite(dx[3]).all() and not torch.isfinite(dx[5]).all() and not torch.isfinite(dw).all()


def test_norm_backward_against_differences_and_repeatable():
    g = gen(11)
    T, d = 50, 104
    s, dy, w, ds = (normal(g, *sh, dtype=F32) for sh in ((T, d), (T, d), (d,), (T, d)))
    op = moe.AddNorm(d, 1e-3)
    dx, dw = op.backward(s, w, dy, ds)
    dx2, dw2 = op.backward(s, w, dy, ds)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)

    def loss(s, w):
        return float((fc.norm(s, None, w, 1e-3)[1] * dy.to(fc.D)).sum() + (s * ds.to(fc.D)).sum())

    h = 1e-5
    for name, grad, base in (("s", dx, s), ("w", dw, w)):
        v = torch.randn(base.shape, generator=g, device="cuda", dtype=fc.D)
        plus, minus = base.to(fc.D) + h * v, base.to(fc.D) - h * v
        a, b = (plus, w.to(fc.D)) if name == "s" else (s.to(fc.D), plus)
        c, e = (minus, w.to(fc.D)) if name == "s" else (s.to(fc.D), minus)
        want = (loss(a, b) - loss(c, e)) / (2 * h)
        # third-order remainder h^2, rounding 1e-16 / h, and 2^-20 of the gradient's magnitudes
        tol = (1e-7 + 2.0 ** -20) * float((grad.to(fc.D) * v).abs().sum())
        assert abs(float((grad.to(fc.D) * v).sum()) - want) <= tol


# ------------------------------------------------------------------ feed-forward block
SHAPES = [(1, 2048, 512), (1, 4096, 8192), (5, 1000, 5000), (40, 2048, 3000), (64, 8, 4096), (17, 4096, 8),
          (3, 136, 9000), (62, 640, 640), (63, 2048, 200), (1, 8, 8), (2, 16, 24), (3, 64, 72), (7, 200, 136),
          (8, 512, 1000), (9, 2048, 2048),
          (16, 256, 128), (17, 520, 264), (32, 2048, 512), (33, 72, 2000), (64, 1024, 640), (100, 256, 8),
          (127, 128, 256), (128, 256, 128), (129, 264, 384), (200, 8, 520), (255, 640, 768), (256, 512, 256),
          (257, 1000, 1000), (385, 2048, 136), (511, 136, 1544), (640, 1536, 1024), (1000, 328, 2744), (1537, 512, 512),
          (3000, 1024, 1032), (2049, 2048, 264)]


@pytest.mark.parametrize("T,d,I", SHAPES)
@pytest.mark.parametrize("name", ["silu", "gelu"])
def test_forward_matches_definition(T, d, I, name):
    g = gen(T + 1000 * d + I)
    x, gu, dn = normal(g, T, d), normal(g, 2 * I, d, scale=d ** -0.5), normal(g, d, I, scale=I ** -0.5)
    op = moe.GatedFfn(d, I, T, activation=ACTS[name])
    y, pre = op.forward(x, gu, dn, save=True)
    y2 = op.forward(x, gu, dn)
    assert op.status() == moe.MOE_OK
    pre0, e_pre, y0, e_y = fc.forward(x, gu, dn, name == "gelu")
    near(pre, pre0, e_pre, "pre")
    near(y, y0, e_y, "y")
    near(y2, y0, e_y, "y without pre")


@pytest.mark.parametrize("T,d,I", SHAPES)
@pytest.mark.parametrize("name", ["silu", "gelu"])
def test_backward_matches_formula(T, d, I, name):
    g = gen(T + 3000 * d + I)
    x, gu, dn = normal(g, T, d), normal(g, 2 * I, d, scale=d ** -0.5), normal(g, d, I, scale=I ** -0.5)
    pre, dy = normal(g, T, 2 * I, scale=2), normal(g, T, d)
    op = moe.GatedFfn(d, I, T + 5, activation=ACTS[name], training=True)
    got = dict(zip(("dx", "dgate_up", "ddown"), op.backward(x, pre, gu, dn, dy)))
    assert op.status() == moe.MOE_OK
    for k, (v, b) in fc.backward(x, pre, gu, dn, dy, name == "gelu").items():
        near(got[k], v, b, k)
    for k, skip in (("dx", (None, False, False)), ("dgate_up", (False, None, False)), ("ddown", (False, False, None))):
        only = dict(zip(("dx", "dgate_up", "ddown"), op.backward(x, pre, gu, dn, dy, *skip)))
        assert torch.equal(only.pop(k), got[k]) and all(v is None for v in only.values())


@pytest.mark.parametrize("name", ["silu", "gelu"])
def test_backward_against_differences(name):
    g = gen(21)
    T, d, I = 24, 64, 48
    x, gu, dn = normal(g, T, d), normal(g, 2 * I, d, scale=d ** -0.5), normal(g, d, I, scale=I ** -0.5)
    dy = normal(g, T, d)
    op = moe.GatedFfn(d, I, T, activation=ACTS[name], training=True)
    y, pre = op.forward(x, gu, dn, save=True)
    grads = op.backward(x, pre, gu, dn, dy)
    base = [t.to(fc.D) for t in (x, gu, dn)]

    def loss(x, gu, dn):
        p = x @ gu.t()
        return float(((fc.act(p[:, :I], name == "gelu") * p[:, I:]) @ dn.t() * dy.to(fc.D)).sum())

    h = 1e-5
    for k in range(3):
        for _ in range(4):
            v = torch.randn(base[k].shape, generator=g, device="cuda", dtype=fc.D)
            plus, minus = list(base), list(base)
            plus[k], minus[k] = base[k] + h * v, base[k] - h * v
            want = (loss(*plus) - loss(*minus)) / (2 * h)
            # roundings to bf16 of pre (twice: gate and up), dpre or h, and the gradient: each moves every term of
            # the gradient by HALF of it at most; the terms add up like independent ones
            tol = 6 * 4 * fc.HALF * float((grads[k].to(fc.D) * v).square().sum().sqrt()) + 1e-6
            assert abs(float((grads[k].to(fc.D) * v).sum()) - want) <= tol, (k, want)


@pytest.mark.parametrize("T,d,I", [(1, 2048, 512), (1, 4096, 8192), (17, 4096, 32), (48, 1024, 3008), (3, 160, 8992),
                                   (1, 32, 32), (2, 64, 96), (9, 1024, 2048), (16, 256, 160),
                                   (33, 96, 2048), (64, 512, 224), (128, 256, 128), (129, 288, 384), (257, 1024, 992),
                                   (511, 160, 1568), (1000, 352, 2752), (2000, 256, 4128), (2000, 4096, 256),
                                   (700, 4128, 4096)])
@pytest.mark.parametrize("name", ["silu", "gelu"])
def test_mx8_forward_matches_definition(T, d, I, name):
    g = gen(T + 5000 * d + I)
    x = moe.moe_quantize_mx(normal(g, T, d, dtype=F32))
    gu = moe.moe_quantize_mx(normal(g, 2 * I, d, scale=d ** -0.5))
    dn = moe.moe_quantize_mx(normal(g, d, I, scale=I ** -0.5))
    op = moe.GatedFfn(d, I, T + 3, activation=ACTS[name], weight_format=moe.MOE_W_MX8)
    y = op.forward(x, gu, dn)
    assert op.status() == moe.MOE_OK
    y0, b = fc.forward_mx(x, gu, dn, name == "gelu")
    near(y, y0, b, "y")


@pytest.mark.parametrize("T,d,I", [(33, 4096, 2752), (64, 1056, 10624), (50, 11264, 1024)])
def test_mx8_few_tokens_and_large_weights(T, d, I):
    test_mx8_forward_matches_definition(T, d, I, "silu")


def test_saturated_activations_stay_finite():
    # gates far outside the range in which exp() is finite, and the ends of bf16
    vals = torch.tensor([-3e38, -1e19, -1e4, -200.0, -90.0, -10.0, -1e-30, 0.0, 1e-30, 10.0, 90.0, 200.0, 1e4],
                        device="cuda")
    I = 16
    pre = torch.zeros(len(vals), 2 * I, dtype=BF, device="cuda")
    pre[:, :I] = vals.to(BF).view(-1, 1)
    pre[:, I:] = 0.5
    g = gen(3)
    x, dy = normal(g, len(vals), 16), normal(g, len(vals), 16)
    gu, dn = normal(g, 2 * I, 16), normal(g, 16, I)
    for name in ACTS:
        op = moe.GatedFfn(16, I, 64, activation=ACTS[name], training=True)
        keep = vals.abs() < (1e30 if name == "silu" else 1e6)  # the formula in 64 bits overflows past that
        got = dict(zip(("dx", "dgate_up", "ddown"), op.backward(x, pre, gu, dn, dy)))
        assert torch.isfinite(got["dx"]).all()
        want = fc.backward(x[keep], pre[keep], gu, dn, dy[keep], name == "gelu")["dx"]
        near(got["dx"][keep], *want, "dx")


def test_nan_stays_in_its_row():
    g = gen(8)
    for T in (5, 300):
        x, gu, dn = normal(g, T, 256), normal(g, 512, 256, scale=0.06), normal(g, 256, 256, scale=0.06)
        clean = moe.GatedFfn(256, 256, T).forward(x, gu, dn)
        x[3, 17] = float("nan")
        y = moe.GatedFfn(256, 256, T).forward(x, gu, dn)
        assert torch.isnan(y[3]).all()
        y[3] = clean[3]
        assert torch.equal(y, clean)


def test_stream_graph_and_reuse():
    g = gen(9)
    T, d, I = 70, 512, 384
    op, nm = moe.GatedFfn(d, I, 512, training=True), moe.AddNorm(d)
    x, res, w = normal(g, T, d), normal(g, T, d), normal(g, d)
    gu, dn, dy = normal(g, 2 * I, d, scale=0.05), normal(g, d, I, scale=0.05), normal(g, T, d)

    def step():
        y, s = nm.forward(x, res, w)
        out, pre = op.forward(y, gu, dn, save=True)
        dxn, dgu, dd = op.backward(y, pre, gu, dn, dy)
        dx, dw = nm.backward(s, w, dxn, dy)
        return out, pre, dgu, dd, dx, dw

    want = [t.clone() for t in step()]
    other = normal(g, 500, d)
    op.forward(other, gu, dn)  # leaves other values in the workspace
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for a, b in zip(step(), want):
            assert torch.equal(a, b)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(2):
        for t in got:
            t.zero_()
        graph.replay()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    assert op.status() == moe.MOE_OK and moe.moe_ffn_launch_count(op.ctx) > 0


def shifted(t):
    """A copy of t that begins 16 bytes past a 32-byte boundary."""
    n = 16 // t.element_size()
    buf = torch.empty(t.numel() + n, dtype=t.dtype, device=t.device)[n:].view(t.shape)
    assert buf.data_ptr() % 32 == 16
    return buf.copy_(t)


@pytest.mark.parametrize("T", [3, 300, 700])
def test_tensors_at_16_bytes_give_the_same(T):
    d, I = 256, 544
    g = gen(T)
    x, gu, dn = normal(g, T, d), normal(g, 2 * I, d, scale=0.05), normal(g, d, I, scale=0.05)
    dy, w = normal(g, T, d), normal(g, d)
    ffn, mx = moe.GatedFfn(d, I, T, training=True), moe.GatedFfn(d, I, T, weight_format=moe.MOE_W_MX8)
    y0, pre0 = ffn.forward(x, gu, dn, save=True)
    grads0 = ffn.backward(x, pre0, gu, dn, dy)
    sx, sgu, sdn, sdy = (shifted(t) for t in (x, gu, dn, dy))
    y, pre = shifted(torch.zeros_like(y0)), shifted(torch.zeros_like(pre0))
    for out in ((y, pre), (y, torch.zeros_like(pre0)), (torch.zeros_like(y0), pre)):
        got = ffn.forward(sx, sgu, sdn, y=out[0], pre=out[1])
        assert torch.equal(got[0], y0) and torch.equal(got[1], pre0)
    outs = [shifted(torch.zeros_like(t)) for t in grads0]
    for a, b in zip(ffn.backward(sx, pre, sgu, sdn, sdy, *outs), grads0):
        assert torch.equal(a, b)
    q = [moe.moe_quantize_mx(t) for t in (x, gu, dn)]
    y0 = mx.forward(*q)
    sq = [(shifted(c), shifted(s)) for c, s in (moe.moe_quantize_mx(shifted(t)) for t in (x, gu, dn))]
    assert torch.equal(mx.forward(*sq, y=shifted(torch.zeros_like(y0))), y0)
    op = moe.AddNorm(d)
    for a, b in zip(op.forward(sx, sdy, shifted(w)), op.forward(x, dy, w)):
        assert torch.equal(a, b)
    for a, b in zip(op.backward(sx, shifted(w), sdy), op.backward(x, w, dy)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("what", ["norm", "norm_mx8", "norm_backward", "quantize", "ffn", "ffn_save", "ffn_backward"])
def test_results_on_another_stream_are_not_in_memory_still_read(what):
    # A tensor is let go while the present stream has yet to read it: its memory is the present stream's to give out
    # again, and a call on another stream must not write there now.
    g = gen(21)
    T, d, I = 64, 256, 512
    x, gu, dn, w = normal(g, T, d), normal(g, 2 * I, d, scale=0.06), normal(g, d, I, scale=0.04), normal(g, d)
    op, ffn = moe.AddNorm(d), moe.GatedFfn(d, I, T, training=True)
    y, pre = ffn.forward(x, gu, dn, save=True)
    side = torch.cuda.Stream()
    call = {"norm": lambda st: op.forward(x, x, w, stream=st),
            "norm_mx8": lambda st: op.forward(x, None, w, y_dtype=moe.MOE_MX8, stream=st),
            "norm_backward": lambda st: op.backward(x, w, x, stream=st),
            "quantize": lambda st: moe.moe_quantize_mx(x, stream=st),
            "ffn": lambda st: ffn.forward(x, gu, dn, stream=st),
            "ffn_save": lambda st: ffn.forward(x, gu, dn, save=True, stream=st),
            "ffn_backward": lambda st: ffn.backward(x, pre, gu, dn, x, stream=st)}[what]

    def flat(r):
        return [t for q in (r if isinstance(r, tuple) else (r,)) for t in (q if isinstance(q, tuple) else (q,))]

    want = [t.view(torch.uint8).clone() for t in flat(call(None))]
    old = [torch.full_like(t, 7) for t in want]
    keep = [torch.empty_like(t) for t in want]
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)  # ~50 ms
    for k, o in zip(keep, old):
        k.copy_(o)
    del old, o
    got = flat(call(side))
    torch.cuda.synchronize()
    for k, t, want_t in zip(keep, got, want):
        assert bool((k == 7).all())
        assert torch.equal(t.view(torch.uint8), want_t)


def test_norm_backward_of_one_object_on_two_streams():
    g = gen(22)
    T, d = 20000, 1024
    op, w = moe.AddNorm(d), normal(g, d)
    s, dy = [normal(g, T, d) for _ in range(2)], normal(g, T, d)
    want = [op.backward(t, w, dy)[1] for t in s]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):  # the calls overlap
        got = [op.backward(t, w, dy, stream=st)[1] for t, st in zip(s, streams)]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_offsets_past_32_bits():
    # pre has 2.3e9 elements, h 1.15e9
    g = gen(10)
    T, d, I = 70001, 64, 16384
    x, gu, dn = normal(g, T, d), normal(g, 2 * I, d, scale=0.1), normal(g, d, I, scale=0.01)
    op = moe.GatedFfn(d, I, T, training=True)
    y, pre = op.forward(x, gu, dn, save=True)
    dy = normal(g, T, d)
    (dx,) = op.backward(x, pre, gu, dn, dy, None, False, False)[:1]
    assert op.status() == moe.MOE_OK
    rows = slice(T - 40, T)
    pre0, e_pre, y0, e_y = fc.forward(x[rows], gu, dn, False)
    near(pre[rows], pre0, e_pre, "pre")
    near(y[rows], y0, e_y, "y")
    near(dx[rows], *fc.backward(x[rows], pre[rows], gu, dn, dy[rows], False)["dx"], "dx")


@pytest.mark.parametrize("d,I", [(1032, 10856), (11200, 1000), (4096, 2752)])
@pytest.mark.parametrize("T", [33, 47, 64])
def test_few_tokens_and_large_weights(T, d, I):
    # weights large enough to be streamed up to 64 tokens; clusters of 1 to 8 CTAs
    g = gen(T * 7 + d)
    x, gu, dn, dy = normal(g, T, d), normal(g, 2 * I, d, scale=0.02), normal(g, d, I, scale=0.02), normal(g, T, d)
    op = moe.GatedFfn(d, I, T, training=True)
    y, pre = op.forward(x, gu, dn, save=True)
    pre0, e_pre, y0, e_y = fc.forward(x, gu, dn, False)
    near(pre, pre0, e_pre, "pre")
    near(y, y0, e_y, "y")
    got = op.backward(x, pre, gu, dn, dy)
    want = fc.backward(x, pre, gu, dn, dy, False)
    for name, t in zip(("dx", "dgate_up", "ddown"), got):
        near(t, *want[name], name)
    assert torch.equal(op.backward(x, pre, gu, dn, dy, None, False, False)[0], got[0])
    assert op.status() == moe.MOE_OK


def test_few_tokens_and_large_weights_wait_that_runs_out():
    g = gen(31)
    T, d, I = 40, 4096, 2752
    x, gu, dn = normal(g, T, d), normal(g, 2 * I, d, scale=0.02), normal(g, d, I, scale=0.02)
    op = moe.GatedFfn(d, I, T, training=True)
    want, pre = op.forward(x, gu, dn, save=True)
    moe.moe_ffn_set_spin_limit(op.ctx, 20_000_000)
    moe.moe_ffn_inject_stall(op.ctx, True)
    op.forward(x, gu, dn)
    assert op.status() == moe.MOE_ERR_TIMEOUT
    op.backward(x, pre, gu, dn, x)
    assert op.status() == moe.MOE_ERR_TIMEOUT
    moe.moe_ffn_inject_stall(op.ctx, False)
    moe.moe_ffn_set_spin_limit(op.ctx, 0)
    assert torch.equal(op.forward(x, gu, dn), want) and op.status() == moe.MOE_OK


@pytest.mark.parametrize("T", [9, 700])
def test_wait_that_runs_out_is_reported_and_recovered(T):
    g = gen(12)
    d, I = 256, 520
    x, gu, dn = normal(g, T, d), normal(g, 2 * I, d, scale=0.06), normal(g, d, I, scale=0.04)
    op = moe.GatedFfn(d, I, T, training=True)
    want, pre = op.forward(x, gu, dn, save=True)
    moe.moe_ffn_set_spin_limit(op.ctx, 20_000_000)
    moe.moe_ffn_inject_stall(op.ctx, True)
    op.forward(x, gu, dn)
    assert op.status() == moe.MOE_ERR_TIMEOUT and op.status() == moe.MOE_OK
    op.backward(x, pre, gu, dn, x)
    assert op.status() == moe.MOE_ERR_TIMEOUT
    moe.moe_ffn_inject_stall(op.ctx, False)
    moe.moe_ffn_set_spin_limit(op.ctx, 0)
    for _ in range(3):
        assert torch.equal(op.forward(x, gu, dn), want) and op.status() == moe.MOE_OK
    with pytest.raises(moe.MoeError):
        moe.moe_ffn_set_spin_limit(op.ctx, -1)


def test_no_rows():
    d, I = 64, 48
    op, nm = moe.GatedFfn(d, I, 8, training=True), moe.AddNorm(d)
    z = lambda *s: torch.empty(*s, dtype=BF, device="cuda")  # noqa: E731
    gu, dn, w = z(2 * I, d).normal_(), z(d, I).normal_(), z(d).normal_()
    y, s = nm.forward(z(0, d), z(0, d), w)
    assert y.shape == (0, d) and s.shape == (0, d)
    y, pre = op.forward(z(0, d), gu, dn, save=True)
    assert y.shape == (0, d) and pre.shape == (0, 2 * I)
    dx, dgu, dd = op.backward(z(0, d), z(0, 2 * I), gu, dn, z(0, d))
    assert dx.shape == (0, d) and not dgu.any() and not dd.any()
    dx, dw = nm.backward(z(0, d), w, z(0, d))
    assert dx.shape == (0, d) and not dw.any()


def test_refusals():
    op = moe.GatedFfn(64, 32, 8)
    z = lambda *s, dtype=BF: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    x, gu, dn = z(4, 64), z(64, 64), z(64, 32)
    for bad in (lambda: op.forward(x.float(), gu, dn), lambda: op.forward(z(4, 128)[:, ::2], gu, dn),
                lambda: op.forward(z(4, 32), gu, dn), lambda: op.forward(x, z(32, 64), dn),
                lambda: op.forward(x.cpu(), gu, dn), lambda: op.forward(x, gu, dn, y=z(5, 64)),
                lambda: moe.AddNorm(64).forward(z(4, 32), None, z(32)), lambda: moe.AddNorm(64).forward(x, None, z(32)),
                lambda: moe.AddNorm(64).forward(x, x.half(), z(64)),
                lambda: moe.AddNorm(64).forward(x, None, z(64), y_dtype=7),
                lambda: moe.GatedFfn(64, 32, 8, weight_format=moe.MOE_W_MX8).forward(x, gu, dn)):
        with pytest.raises(ValueError):
            bad()
    for bad, code in ((lambda: op.forward(z(9, 64), gu, dn), moe.MOE_ERR_ARG),
                      (lambda: op.backward(x, z(4, 64), gu, dn, x), moe.MOE_ERR_UNSUPPORTED),
                      (lambda: op.forward(z(4 * 64 + 1)[1:].view(4, 64), gu, dn), moe.MOE_ERR_ALIGN),
                      (lambda: moe.AddNorm(20000).forward(z(1, 20000), None, z(20000)), moe.MOE_ERR_UNSUPPORTED),
                      (lambda: moe.AddNorm(40).forward(z(1, 40), None, z(40), y_dtype=moe.MOE_MX8),
                       moe.MOE_ERR_UNSUPPORTED),
                      (lambda: moe.moe_quantize_mx(z(4, 32, dtype=F32).view(2, 64)[:, :40].contiguous()),
                       moe.MOE_ERR_UNSUPPORTED)):
        with pytest.raises((moe.MoeError, ValueError)) as e:
            bad()
        assert getattr(e.value, "code", code) == code
