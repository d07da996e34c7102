"""The product with bias, activation and residual, and its gradients, against the definitions in 64 bits (bounds:
ops_case.py)."""
import pytest
import torch

import expert_routed_ffn_moe_gb300 as moe
import ops_case as oc
from test_gpu_ffn import BF, F32, gen, near, normal

pytestmark = pytest.mark.gpu
ACTS = {"none": moe.MOE_ACT_NONE, "silu": moe.MOE_ACT_SILU, "gelu": moe.MOE_ACT_GELU}


def operands(g, T, k, n, bias=BF, res=None):
    x, w = normal(g, T, k), normal(g, n, k, scale=k ** -0.5)
    return x, w, None if bias is None else normal(g, n, dtype=bias), None if res is None else normal(g, T, n, scale=2, dtype=res)


# few tokens as a weight stream; one tile and split ones; several tiles per pair of CTAs; no multiple of a tile
SIZES = [(1, 8, 8), (1, 2048, 4096), (1, 8200, 1000), (2, 64, 136), (3, 520, 2400), (4, 4096, 3000), (4, 16, 17000), (5, 264, 1000), (8, 4096, 4096), (12, 2048, 4104), (13, 1024, 776), (16, 256, 1000), (17, 72, 128), (31, 1000, 264), (33, 512, 64),
         (48, 4096, 4096), (64, 4104, 4096), (40, 128, 8200), (50, 8200, 136), (65, 256, 512), (128, 4096, 4096), (200, 1024, 768), (200, 1000, 5000), (300, 136, 2744), (777, 1000, 2744),
         (1025, 264, 8), (2500, 512, 4352)]


@pytest.mark.parametrize("T,k,n", SIZES)
@pytest.mark.parametrize("act,bias,res,y", [("none", None, None, BF), ("gelu", BF, None, BF), ("silu", F32, BF, BF),
                                            ("none", BF, F32, F32), ("gelu", F32, None, F32)])
def test_matches_definition(T, k, n, act, bias, res, y):
    x, w, b, r = operands(gen(T + k * 7 + n), T, k, n, bias, res)
    op = moe.Linear(k, n, T, activation=ACTS[act])
    want = oc.linear(x, w, b, r, act, y)
    got, pre = op.forward(x, w, b, r, y_dtype=y, save=True)
    assert got.dtype == y and pre.dtype == BF
    near(got, *want["y"], "y")
    near(pre, *want["pre"], "pre")
    assert torch.equal(op.forward(x, w, b, r, y_dtype=y), got)  # pre does not change y
    assert op.status() == moe.MOE_OK


@pytest.mark.parametrize("T,k,n", SIZES)
@pytest.mark.parametrize("act,bias,dyt", [("none", BF, BF), ("gelu", F32, BF), ("silu", BF, F32), ("none", F32, F32)])
def test_gradients_match_definition(T, k, n, act, bias, dyt):
    g = gen(T + k * 7 + n + 1)
    x, w, b, _ = operands(g, T, k, n, bias)
    pre, dy = normal(g, T, n), normal(g, T, n, dtype=dyt)
    op = moe.Linear(k, n, T, activation=ACTS[act], training=True)
    got = op.backward(x, pre, w, b, dy)
    want = oc.linear_backward(x, pre, w, dy, act, bias)
    for v, name in zip(got, ("dx", "dweight", "dbias")):
        near(v, *want[name], name)
    for i in range(3):  # one at a time, and all but one
        one = op.backward(x, pre, w, b, dy, *[None if j == i else False for j in range(3)])
        two = op.backward(x, pre, w, b, dy, *[False if j == i else None for j in range(3)])
        assert all((a is None) == (j != i) for j, a in enumerate(one)) and torch.equal(one[i], got[i])
        assert all(a is None if j == i else torch.equal(a, got[j]) for j, a in enumerate(two))
    assert op.status() == moe.MOE_OK


def test_gradients_match_differences():
    T, k, n = 3, 16, 24
    g = gen(4)
    x, w, b, _ = operands(g, T, k, n, F32)
    dy = normal(g, T, n)
    op = moe.Linear(k, n, T, activation=moe.MOE_ACT_GELU, training=True)
    _, pre = op.forward(x, w, b, save=True)
    got = op.backward(x, pre, w, b, dy)

    def loss(x, w, b):
        return (oc.linear(x, w, b, None, "gelu", F32)["y"][0] * dy.to(oc.D)).sum()

    for t, at in ((0, (1, 3)), (0, (2, 15)), (1, (23, 0)), (1, (5, 9)), (2, (7,))):
        h = 1e-4
        args = [v.to(oc.D) for v in (x, w, b)]
        args[t][at] += h
        up = loss(*args)
        args[t][at] -= 2 * h
        slope = float((up - loss(*args)) / (2 * h))
        # pre, dpre and the gradient are rounded to bf16: three times 2^-8 of terms, whose sums stay below 8 here
        assert abs(slope - float(got[t][at])) < 3 * 8 * 2.0 ** -8


def test_in_place_unaligned_tensors_and_no_rows():
    g = gen(6)
    T, k, n = 100, 136, 264
    x, w, b, r = operands(g, T, k, n, BF, F32)
    op = moe.Linear(k, n, T, activation=moe.MOE_ACT_SILU, training=True)
    want = op.forward(x, w, b, r)
    over = r.clone()
    assert op.forward(x, w, b, over, y=over) is over and torch.equal(over, want)

    def shifted(t):  # the same values 16 bytes past a 32-byte boundary
        v = torch.empty(t.numel() + 16 // t.element_size(), dtype=t.dtype, device="cuda")[16 // t.element_size():]
        v = v.view(t.shape)
        return v.copy_(t)

    for T in (1, 20, 100):
        for rr in (r[:T], r[:T].to(BF)):
            y, pre = op.forward(x[:T], w, b, rr, save=True)
            ys, ps = shifted(torch.zeros_like(y)), shifted(torch.zeros_like(pre))
            op.forward(shifted(x[:T]), shifted(w), shifted(b), shifted(rr), y=ys, pre=ps)
            assert torch.equal(ys, y) and torch.equal(ps, pre)
        dy = normal(g, T, n)
        got = op.backward(x[:T], pre, w, b, dy)
        outs = [shifted(torch.zeros_like(t)) for t in got]
        op.backward(shifted(x[:T]), shifted(pre), shifted(w), shifted(b), shifted(dy), *outs)
        assert all(torch.equal(a, c) for a, c in zip(outs, got))
    z = lambda *s: torch.empty(*s, dtype=BF, device="cuda")  # noqa: E731
    assert op.forward(z(0, k), w, b).shape == (0, n)
    dx, dw, db = op.backward(z(0, k), z(0, n), w, b, z(0, n))
    assert dx.shape == (0, k) and not dw.any() and not db.any()
    assert op.status() == moe.MOE_OK


@pytest.mark.parametrize("T", [1, 40, 700])
def test_streams_graphs_and_rows_behind_the_last(T):
    g = gen(T)
    k, n = 512, 1032
    x, w, b, r = operands(g, T, k, n, BF, BF)
    dy = normal(g, T, n)
    op = moe.Linear(k, n, T + 5, activation=moe.MOE_ACT_GELU, training=True)

    def step(stream=None):
        y, pre = op.forward(x, w, b, r, save=True, stream=stream)
        return [y, pre, *op.backward(x, pre, w, b, dy, stream=stream)]

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(got, want))
    big = torch.full((T + 5, n), 3.0, dtype=BF, device="cuda")
    op.forward(x, w, b, r, y=big[:T])
    assert torch.equal(big[:T], want[0]) and (big[T:] == 3).all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    w.copy_(normal(g, n, k, scale=0.05))  # written on the same stream just before: the kernels' first reads follow it
    graph.replay()
    assert all(torch.equal(a, c) for a, c in zip(got, step()))
    assert op.status() == moe.MOE_OK


@pytest.mark.parametrize("T", [1, 7, 300])
def test_a_wait_that_runs_out_is_reported(T):
    g = gen(1)
    x, w, b, _ = operands(g, T, 256, 512)
    op = moe.Linear(256, 512, T, training=True)
    want = op.forward(x, w, b)
    moe.moe_linear_set_spin_limit(op.ctx, 1_000_000)
    moe.moe_linear_inject_stall(op.ctx, True)
    op.forward(x, w, b)
    assert op.status() == moe.MOE_ERR_TIMEOUT and op.status() == moe.MOE_OK
    moe.moe_linear_inject_stall(op.ctx, False)
    moe.moe_linear_set_spin_limit(op.ctx, 0)
    assert torch.equal(op.forward(x, w, b), want) and op.status() == moe.MOE_OK


def test_launch_count_and_errors():
    op = moe.Linear(64, 64, 8)
    x, w = normal(gen(0), 8, 64), normal(gen(0), 64, 64)
    op.forward(x, w)
    assert moe.moe_linear_launch_count(op.ctx) == 1
    with pytest.raises(moe.MoeError) as e:
        op.backward(x, None, w, None, x)
    assert e.value.code == moe.MOE_ERR_UNSUPPORTED
    with pytest.raises(moe.MoeError) as e:
        op.forward(normal(gen(0), 9, 64), w)
    assert e.value.code == moe.MOE_ERR_ARG
    op = moe.Linear(64, 64, 8, activation=moe.MOE_ACT_GELU, training=True)
    with pytest.raises(moe.MoeError) as e:  # an activation's gradient needs pre
        op.backward(x, None, w, None, x)
    assert e.value.code == moe.MOE_ERR_ARG


# a stream's kinds, split and unsplit tiles, and many tiles of a short reduction per pair of CTAs
SOME = [(1, 64, 200), (9, 64, 200), (70, 4096, 264), (300, 136, 520), (2100, 72, 5000)]


@pytest.mark.parametrize("T,k,n", SOME)
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_a_value_beyond_the_range_stays_alone(T, k, n, act):
    x, w, b, r = operands(gen(T + n), T, k, n, F32, F32)
    op = moe.Linear(k, n, T, activation=ACTS[act], training=True)
    want = oc.linear(x, w, b, r, act, F32)["y"]
    pre = op.forward(x, w, b, r, save=True, y_dtype=F32)[1]
    cols = torch.tensor([0, 3, 6, 17, 33, 66, 134, 199])
    far = torch.tensor([float("nan"), float("inf"), 1e30, -1e30, float("nan"), 3e38, -3e38, float("inf")], device="cuda")
    b[cols] = far
    got = op.forward(x, w, b, r, y_dtype=F32)
    others = torch.ones(n, dtype=torch.bool)
    others[cols] = False
    # A value's last bits may follow its neighbour, with which it shares a reciprocal: the logistic function is then off by
    # the rounding of the two denominators' product (2^-24), the reciprocal's last place (2^-23) and that of the product
    # with the other denominator (2^-24); times the value once more 2^-24: 2.5 * 2^-23 < 2^-21, within the bound.
    near(got[:, others], *(v[:, others] for v in want), "y")
    far_y = torch.where(far < 0, 0.0, far) + r[:, cols]  # act is the value itself, or 0
    off = torch.where(far_y.isfinite() & (far > 0), 2.0 ** -21 * far_y.abs(), 0.0)
    same = (got[:, cols] == far_y) | (got[:, cols].isnan() & far_y.isnan()) | ((got[:, cols] - far_y).abs() <= off)
    assert same.all(), got[:, cols][~same]

    dy = normal(gen(T), T, n)
    want = oc.linear_backward(x, pre, w, dy, act, F32)
    pre[:, cols] = far.to(BF)
    dw, db = op.backward(x, pre, w, b, dy, dx=False)[1:]
    near(dw[others], *(v[others] for v in want["dweight"]), "dweight")
    near(db[others], *(v[others] for v in want["dbias"]), "dbias")
    nan, down = torch.isnan(far).cpu(), (far < 0).cpu()
    assert torch.isnan(db[cols[nan]]).all()
    assert (db[cols[down]] == 0).all() and (dw[cols[down]] == 0).all()
    assert op.status() == moe.MOE_OK


@pytest.mark.parametrize("T,k,n", SOME + [(2500, 512, 4352)])
@pytest.mark.parametrize("y", [BF, F32])
def test_the_result_may_take_the_residuals_place(T, k, n, y):
    x, w, b, r = operands(gen(T + k), T, k, n, BF, y)
    op = moe.Linear(k, n, T, activation=moe.MOE_ACT_GELU)
    want = oc.linear(x, w, b, r, "gelu", y)["y"]
    apart = op.forward(x, w, b, r)
    near(apart, *want, "y")
    assert op.forward(x, w, b, r, y=r).data_ptr() == r.data_ptr()
    assert torch.equal(r, apart) and op.status() == moe.MOE_OK
