"""The narrow bound on the mx8 block's output (ffn_mx_case.py) holds for a block
computed in fp32 and for none of several wrong ones (no GPU)."""
import pytest
import torch

import ffn_case as fc
import ffn_mx_case as mc

SMALL = [s for s in mc.SHAPES if s[0] * s[1] * s[2] < 1 << 28 and s[1] * s[2] <= 1 << 25]


def fp32_block(x, gate_up, down, gelu, hold=True):
    """The block in fp32 steps; hold=False leaves h as it is.  Returns (y before rounding, h)."""
    pre = x @ gate_up.t()
    I = pre.shape[1] // 2
    g = pre[:, :I]
    z = 1.5957691216057308 * (g + 0.044715 * g * g * g) if gelu else g
    h = g / (1 + torch.exp(-z)) * pre[:, I:]
    if hold:
        h = mc.codes_of(h.to(mc.D), fc.exponents(h)).float()
    return h @ down.t(), h


def outside(y, want, bound):
    return ((y.to(torch.bfloat16).to(mc.D) - want).abs() > bound).any()


@pytest.mark.parametrize("T,d,I", SMALL)
@pytest.mark.parametrize("gelu", [False, True])
def test_operands_are_exact(T, d, I, gelu):
    x, gu, dn = mc.operands(T, d, I, T + d + I)
    for t in (x, gu, dn):
        assert torch.equal(fc.dequantize(*fc.quantize(t)), t.to(mc.D))
    assert torch.equal((x @ gu.t()).to(mc.D), x.to(mc.D) @ gu.to(mc.D).t())


@pytest.mark.parametrize("T,d,I", SMALL)
@pytest.mark.parametrize("gelu", [False, True])
def test_bound_tells_right_from_wrong(T, d, I, gelu):
    x, gu, dn = mc.operands(T, d, I, T + d + I)
    want, bound = mc.forward(x, gu, dn, gelu)
    y, h = fp32_block(x, gu, dn, gelu)
    assert not outside(y, want, bound)
    # h not held in mx8; held in bf16
    raw = fp32_block(x, gu, dn, gelu, hold=False)[1]
    assert outside(raw @ dn.t(), want, bound)
    assert outside(raw.to(torch.bfloat16).float() @ dn.t(), want, bound)

    def with_h(change):
        m = h.clone()
        change(m)
        return m @ dn.t()

    def halve_one_group(m):  # the first row's, with its largest value
        k = int(m[0].abs().argmax()) // 32 * 32
        m[0, k:k + 32] /= 2

    assert outside(with_h(lambda m: m[:, -8:].zero_()), want, bound)
    assert outside(with_h(lambda m: m[:, -32:].zero_()), want, bound)
    assert outside(with_h(lambda m: m[:, :32].div_(2)), want, bound)
    assert outside(with_h(halve_one_group), want, bound)
    # one scale of down doubled, where the first row feels it most
    parts = (h[0].view(1, -1, 32) * dn.view(d, -1, 32)).sum(-1).abs()
    n, k = divmod(int(parts.argmax()), parts.shape[1])
    wrong = dn.clone()
    wrong[n, 32 * k:32 * k + 32] *= 2
    assert outside(h @ wrong.t(), want, bound)
    # the scales of gate_up's first two groups exchanged, in every row
    wrong = gu.clone()
    if d >= 64:
        s = [2.0 ** fc.exponents(gu)[:, i:i + 1].float() for i in (0, 1)]
        wrong[:, :32], wrong[:, 32:64] = gu[:, :32] / s[0] * s[1], gu[:, 32:64] / s[1] * s[0]
        assert outside(fp32_block(x, wrong, dn, gelu)[0], want, bound)
