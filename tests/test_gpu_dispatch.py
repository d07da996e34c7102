"""Tokens sorted by expert and back, with their gradients (definitions and bounds: ops_case.py)."""
import pytest
import torch

import expert_routed_ffn_moe_gb300 as moe
import ops_case as oc
from test_gpu_ffn import BF, F32, gen, near, normal

pytestmark = pytest.mark.gpu
I32 = torch.int32


def random_picks(g, T, k, E, kind):
    if kind == "same":  # everything to one expert, several times by each token
        return torch.full((T, k), E - 1, dtype=I32, device="cuda")
    idx = torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=I32)  # (repeats within a token among them)
    if kind == "skewed":
        idx = (idx.float() * torch.rand(T, k, generator=g, device="cuda") ** 3).to(I32)
    if kind == "dropped":
        r = torch.rand(T, k, generator=g, device="cuda")
        idx[r < 0.3] = -1
        idx[r > 0.9] = E
        idx[(r > 0.6) & (r < 0.62)] = 0x7fffffff
        idx[(r > 0.5) & (r < 0.52)] = -0x80000000
    if kind == "none":
        idx.fill_(-1)
    return idx


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 256), (3, 32, 40), (31, 1, 7), (33, 2, 60), (128, 8, 256),
                                   (257, 4, 1024), (1000, 6, 60), (2049, 8, 256), (4096, 8, 33), (16411, 7, 300)])
@pytest.mark.parametrize("kind", ["random", "skewed", "same", "dropped", "none"])
def test_sort(T, k, E, kind):
    idx = random_picks(gen(T * 31 + k), T, k, E, kind)
    want = oc.sort(idx.cpu(), E)
    n = want[2].numel()
    perm = torch.full((T * k,), -7, dtype=I32, device="cuda")
    counts, offsets, got, slot = moe.TokenDispatch(E, k).sort(idx, perm=perm)
    assert got is perm
    for a, b, name in ((counts, want[0], "counts"), (offsets, want[1], "offsets"), (perm[:n], want[2], "perm"),
                       (slot, want[3], "slot")):
        assert torch.equal(a.cpu(), b), name
    assert (perm[n:] == -7).all()


def test_sort_agrees_with_the_layers_own_routing():
    T, d, E, k = 300, 256, 64, 6
    g = gen(3)
    layer = moe.MoeLayer(d, E, 128, k, T, has_shared=False)
    r = layer.route(normal(g, T, d), normal(g, E, d, dtype=F32), None)
    counts, offsets, perm, _ = moe.TokenDispatch(E, k).sort(r["idx"])
    for a, name in ((counts, "counts"), (offsets, "offsets"), (perm, "perm")):
        assert torch.equal(a, r[name]), name


def test_sort_outputs_are_optional_and_no_tokens():
    idx = random_picks(gen(4), 50, 3, 20, "random")
    want = moe.TokenDispatch(20, 3).sort(idx)
    L, p = moe.lib(), lambda t: None if t is None else t.data_ptr()
    for keep in range(4):
        out = [torch.empty_like(t) if i == keep else None for i, t in enumerate(want)]
        assert L.moe_sort_tokens(p(idx), 50, 3, 20, *map(p, out), None) == moe.MOE_OK
        assert torch.equal(out[keep], want[keep])
    counts, offsets, perm, slot = moe.TokenDispatch(20, 3).sort(torch.empty(0, 3, dtype=I32, device="cuda"))
    assert not counts.any() and not offsets.any() and perm.numel() == 0 and slot.shape == (0, 3)


def tables(g, T, k, E, drop, n_rows):
    """slot with dropped picks, slots past the rows and other negative ones."""
    idx = random_picks(g, T, k, E, "dropped" if drop else "random")
    slot = moe.TokenDispatch(E, k).sort(idx)[3]
    if drop and slot.numel() > 3:
        flat = slot.view(-1)
        flat[flat == 1] = -5
        flat[flat == 2] = 0x7fffffff
    assert drop or n_rows == T * k
    return slot


SIZES = [(1, 1, 1), (1, 8, 2048), (2, 3, 7), (5, 32, 8), (33, 8, 300), (40, 1, 513), (65, 9, 520), (130, 8, 1999),
         (17, 17, 4096), (2050, 2, 264), (2100, 12, 33), (3, 2, 20000)]


@pytest.mark.parametrize("T,k,d", SIZES)
@pytest.mark.parametrize("xt,rt,drop", [(BF, BF, False), (F32, BF, True), (BF, F32, True), (F32, F32, False)])
def test_dispatch_and_its_gradient(T, k, d, xt, rt, drop):
    g = gen(T * 7 + k * 3 + d)
    n_rows = max(1, T * k * 3 // 5) if drop else T * k
    slot = tables(g, T, k, 16, drop, n_rows)
    x, add = normal(g, T, d, dtype=xt), normal(g, T, d, dtype=xt)
    rows = torch.full((n_rows, d), 7.5, dtype=rt, device="cuda")
    op = moe.TokenDispatch(16, k)
    assert op.dispatch(x, slot, rows=rows) is rows
    t, _, r = oc.picks(slot, n_rows)
    want = torch.full_like(rows, 7.5)
    want[r] = x[t].to(rt)
    assert torch.equal(rows, want)
    if not drop:
        assert torch.equal(op.dispatch(x, slot, rows_dtype=rt), want)
    drows = normal(g, n_rows, d, dtype=rt)
    if drop:  # what no pick has is never read into a sum
        unused = torch.ones(n_rows, dtype=torch.bool, device="cuda")
        unused[r] = False
        drows[unused] = float("nan")
    near(op.dispatch_backward(drows, slot, add=add), *oc.combine(drows, slot, None, add, xt), "dx")
    near(op.dispatch_backward(drows, slot, x_dtype=xt), *oc.combine(drows, slot, None, None, xt), "dx alone")


@pytest.mark.parametrize("T,k,d", SIZES)
@pytest.mark.parametrize("yt,rt,drop", [(BF, BF, False), (F32, BF, True), (BF, F32, True), (F32, F32, False)])
def test_combine_and_its_gradients(T, k, d, yt, rt, drop):
    g = gen(T * 7 + k * 3 + d + 1)
    n_rows = max(1, T * k * 3 // 5) if drop else T * k
    slot = tables(g, T, k, 16, drop, n_rows)
    rows, add, dy = normal(g, n_rows, d, dtype=rt), normal(g, T, d, dtype=yt), normal(g, T, d, dtype=yt)
    w = torch.rand(T, k, generator=g, device="cuda")
    t, j, r = oc.picks(slot, n_rows)
    if drop:  # a dropped pick's weight and an unused row may be anything
        gone = torch.ones_like(slot, dtype=torch.bool)
        gone[t, j] = False
        w[gone] = float("nan")
        unused = torch.ones(n_rows, dtype=torch.bool, device="cuda")
        unused[r] = False
        rows[unused] = float("inf")
    op = moe.TokenDispatch(16, k)
    near(op.combine(rows, slot, w, add=add), *oc.combine(rows, slot, w, add, yt), "y")
    near(op.combine(rows, slot, w, y_dtype=yt), *oc.combine(rows, slot, w, None, yt), "y alone")
    over = add.clone()
    assert op.combine(rows, slot, w, add=over, y=over) is over
    assert torch.equal(over, op.combine(rows, slot, w, add=add))
    drows = torch.full((n_rows, d), 7.5, dtype=rt, device="cuda")
    got, dw = op.combine_backward(dy, rows, slot, w, drows=drows)
    want = torch.full_like(drows, 7.5)
    want[r] = (w[t, j, None] * dy[t].float()).to(rt)
    assert got is drows and torch.equal(drows, want)
    near(dw, *oc.combine_dw(dy, rows, slot), "dw")
    # one gradient alone, and drows over rows
    assert torch.equal(op.combine_backward(dy, rows, slot, w, drows=False)[1], dw)
    alone = torch.full_like(drows, 7.5)
    assert op.combine_backward(dy, rows, slot, w, drows=alone, dw=False)[1] is None and torch.equal(alone, want)
    used = rows.clone()
    assert torch.equal(op.combine_backward(dy, used, slot, w, drows=used)[1], dw) and torch.equal(used[r], want[r])


def test_combine_gradients_match_differences():
    T, k, d = 4, 3, 16
    g = gen(2)
    slot = tables(g, T, k, 16, False, T * k)
    rows, dy = normal(g, T * k, d, dtype=F32), normal(g, T, d, dtype=F32)
    w = torch.rand(T, k, generator=g, device="cuda")
    drows, dw = moe.TokenDispatch(16, k).combine_backward(dy, rows, slot, w)

    def loss(rows, w):  # linear in each: a difference of one step is exact
        return (oc.combine(rows, slot, w, None, F32)[0] * dy.to(oc.D)).sum()

    for at in ((0, 1), (3, 2)):
        up = w.to(oc.D).clone()
        up[at] += 1
        assert abs(float(loss(rows, up) - loss(rows, w)) - float(dw[at])) < 1e-4
    for at in ((0, 5), (11, 15)):
        up = rows.to(oc.D).clone()
        up[at] += 1
        assert abs(float(loss(up, w) - loss(rows, w)) - float(drows[at])) < 1e-4


def test_no_tokens_no_rows_streams_and_graphs():
    g = gen(11)
    T, k, d, E = 70, 4, 512, 32
    op = moe.TokenDispatch(E, k)
    z = torch.empty(0, d, dtype=BF, device="cuda")
    none = torch.empty(0, k, dtype=I32, device="cuda")
    assert op.dispatch(z, none).shape == (0, d) and op.combine(z, none).shape == (0, d)
    x = normal(g, T, d)
    gone = torch.full((T, k), -1, dtype=I32, device="cuda")
    w = torch.rand(T, k, generator=g, device="cuda")
    assert op.dispatch(x, gone, rows=z).shape == (0, d)  # every pick was dropped: no rows at all
    assert torch.equal(op.combine(z, gone, w, add=x), x) and not op.combine(z, gone, w).any()
    drows, dw = op.combine_backward(x, z, gone, w)
    assert drows.shape == (0, d) and not dw.any()

    def step(idx, stream=None):
        counts, offsets, perm, slot = op.sort(idx, stream=stream)
        rows = op.dispatch(x, slot, stream=stream)
        y = op.combine(rows, slot, w, add=x, stream=stream)
        drows, dw = op.combine_backward(y, rows, slot, w, stream=stream)
        return [counts, offsets, perm, slot, rows, y, drows, dw, op.dispatch_backward(drows, slot, add=y, stream=stream)]

    idx = random_picks(g, T, k, E, "random")
    want = step(idx)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(idx, side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(idx)
    idx.copy_(random_picks(g, T, k, E, "random"))
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(got, step(idx)))


def test_offsets_past_31_bits():
    T, k, d = 70000, 8, 4096  # 2.3e9 values of rows
    x = torch.zeros(T, d, dtype=BF, device="cuda")
    x[-1] = normal(gen(1), d)
    slot = torch.arange(T * k, dtype=I32, device="cuda").view(T, k)
    w = torch.rand(T, k, generator=gen(2), device="cuda")
    op = moe.TokenDispatch(16, k)
    rows = op.dispatch(x, slot)
    assert all(torch.equal(rows[-1 - i], x[-1]) for i in range(k)) and not rows[:1000].any()
    y = op.combine(rows, slot, w)
    near(y[-1:], *oc.combine(rows[-k:], slot[:1], w[-1:], None, BF), "last token")
    drows, dw = op.combine_backward(x, rows, slot, w, drows=rows)
    assert torch.equal(drows[-k:], (w[-1, :, None] * x[-1].float()).to(BF))
    near(dw[-1:], *oc.combine_dw(x[-1:], x[-1:].expand(k, d), slot[:1]), "dw of the last token")
