"""The gradients of the product with an activation over the whole range of its pre-activations, against the definition in
64 bits: the derivative at every bf16 value, and products where values of all sizes stand side by side."""
import pytest
import torch

import expert_routed_ffn_moe_gb300 as moe
import ops_case as oc
from test_gpu_ffn import BF, F32, gen, near, normal

pytestmark = pytest.mark.gpu
ACTS = {"silu": moe.MOE_ACT_SILU, "gelu": moe.MOE_ACT_GELU}
LARGE = [10.0, 16.0, 100.0, 256.0, 1000.0, 4096.0, 6.5e4, 1e6, 1e18, 1e30, 3e38]


def derivative_bound(da):
    # Two terms of at most about one each (|act'| <= 1.13), each from the fast exponential and division, counted at 2^-18 of
    # it as in ops_case; dy = 1 and one token, so that dbias in fp32 is act' itself.
    return 2.0 ** -18 * (1 + da.abs()) + oc.U * da.abs()


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dyt", [BF, F32])
@pytest.mark.parametrize("weights", [False, True])  # the kernel that leaves dweight too, and the one that does not
@pytest.mark.parametrize("seed", [1, 2, 3])
def test_the_derivative_at_every_finite_value(act, dyt, weights, seed):
    every = torch.arange(-2 ** 15, 2 ** 15, dtype=torch.int32).to(torch.int16).view(BF)
    every = every[every.isfinite()]
    n = every.numel()  # 65280, each beside two others that the seed chooses
    pre = every[torch.randperm(n, generator=torch.Generator().manual_seed(seed))].view(1, n).cuda()
    x, w = torch.ones(1, 8, dtype=BF, device="cuda"), torch.zeros(n, 8, dtype=BF, device="cuda")
    op = moe.Linear(8, n, 1, activation=ACTS[act], training=True)
    dy = torch.ones(1, n, dtype=dyt, device="cuda")
    _, dw, db = op.backward(x, pre, w, torch.zeros(n, dtype=F32, device="cuda"), dy, dx=False,
                            dweight=None if weights else False)
    da = oc.act_grad(pre[0].to(oc.D), act)
    near(db, da, derivative_bound(da), "act'")
    if weights:  # x is one: dweight is act' rounded to bf16, once as dpre (the product of one token is exact)
        bound = derivative_bound(da)
        near(dw, da[:, None].expand(n, 8), (oc.fc.HALF * (da.abs() + bound) + bound)[:, None], "dweight")
    assert op.status() == moe.MOE_OK


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("far", LARGE)
def test_a_far_value_beside_ordinary_ones(act, far):
    # in the even and in the odd columns, in both signs; the others from a normal distribution
    n = 4096
    g = gen(int(min(far, 1e9)))
    pre = normal(g, 1, n)
    pre[0, 0::4] = far
    pre[0, 3::4] = -far
    pre = pre[:, torch.arange(n).view(-1, 2).flip(1).flatten()] if far in LARGE[::2] else pre
    pre = pre.contiguous()
    x, w = normal(g, 1, 8), normal(g, n, 8)
    op = moe.Linear(8, n, 1, activation=ACTS[act], training=True)
    one = torch.ones(1, n, dtype=F32, device="cuda")
    db = op.backward(x, pre, w, torch.zeros(n, dtype=F32, device="cuda"), one, dx=False, dweight=False)[2]
    da = oc.act_grad(pre[0].to(oc.D), act)
    near(db, da, derivative_bound(da), "act'")


# the weight gradients' kernel of few tokens, a stream's, split tiles and tiles, clusters of 1 to 8 CTAs for dbias
@pytest.mark.parametrize("T,k,n", [(1, 64, 200), (7, 264, 1000), (16, 64, 520), (40, 512, 264), (64, 256, 8200),
                                   (300, 136, 520), (777, 1000, 2744), (2100, 72, 5000)])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dyt", [BF, F32])
def test_gradients_of_pre_activations_of_all_sizes(T, k, n, act, dyt):
    g = gen(T * 7 + n)
    x, w, dy = normal(g, T, k), normal(g, n, k, scale=k ** -0.5), normal(g, T, n, dtype=dyt)
    size = torch.tensor([1.0] * len(LARGE) * 3 + LARGE, device="cuda")
    pre = normal(g, T, n, dtype=F32)
    pre = (pre * size[torch.randint(size.numel(), (T, n), generator=g, device="cuda")]).clamp(-3e38, 3e38).to(BF)
    op = moe.Linear(k, n, T, activation=ACTS[act], training=True)
    bias = torch.zeros(n, dtype=F32, device="cuda")
    got = op.backward(x, pre, w, bias, dy)
    want = oc.linear_backward(x, pre, w, dy, act, F32)
    near(got[0], *want["dx"], "dx")
    near(got[1], *want["dweight"], "dweight")
    # dbias: a thread has every 32nd row at the most, then 32 threads and up to 8 blocks add up
    da = oc.act_grad(pre.to(oc.D), act)
    mags = (dy.to(oc.D) * da).abs().sum(0)
    e = (2.0 ** -18 * dy.to(oc.D).abs() * (1 + da.abs())).sum(0) + (T / 32 + 48) * oc.U * mags
    near(got[2], want["dbias"][0], e + oc.U * mags + 1e-30, "dbias")
    assert op.status() == moe.MOE_OK
