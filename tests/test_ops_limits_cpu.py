"""The sizes that the token sort's and the product's entry points refuse are those that the header gives (no GPU)."""
import ctypes
import re

import pytest

import expert_routed_ffn_moe_gb300 as moe

B, A, OK, UNSUP = moe.MOE_BF16, ctypes.c_void_p(16), moe.MOE_OK, moe.MOE_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    moe.build()
    return moe.lib()


@pytest.fixture(scope="module")
def header():
    return re.sub(r"\s+", " ", open(moe.HEADER).read().replace("\n * ", "\n "))


def test_widths_and_picks_of_rows(lib, header):
    m = re.search(r"d is any width up to 2\^(\d+), top_k at most (\d+), T \* top_k and T \* ceil\(d / 256\) at most 2\^(\d+) "
                  r"\(MOE_ERR_UNSUPPORTED beyond\)", header)
    d, k, n = 1 << int(m[1]), int(m[2]), 1 << int(m[3])
    for call in (lambda T, k, d: lib.moe_dispatch(A, B, None, T, k, d, A, B, 8, None),
                 lambda T, k, d: lib.moe_combine(A, B, 8, None, A, T, k, d, A, A, B, None),
                 lambda T, k, d: lib.moe_combine_backward(A, B, A, B, 8, None, A, T, k, d, A, A, None)):
        refused = moe.MOE_ERR_ARG  # (the missing slot: the sizes are taken)
        assert call(0, k, d) == OK and call(0, k, d + 1) == UNSUP and call(0, k + 1, d) == UNSUP
        assert call(n // k, k, 256) == refused and call(n // k + 1, k, 256) == UNSUP
        assert call(n, 1, 256) == refused and call(n // 2, 1, 512) == refused and call(n // 2 + 1, 1, 257) == UNSUP


def test_sizes_of_the_product(lib, header):
    body = re.search(r"typedef struct moe_linear_config \{(.*?)\} moe_linear_config;", header)[1]
    most = {n: 1 << int(p) for n, p in re.findall(r"int (\w+); /\*[^/]*?at most 2\^(\d+) \*/", body)}
    assert sorted(most) == ["in_features", "max_tokens", "out_features"]
    for name, limit in most.items():
        for size, past in ((limit, False), (limit + 8, True)):
            sizes = dict(dict(in_features=64, out_features=64, max_tokens=8, activation=2, training=0), **{name: size})
            h = ctypes.c_void_p()
            code = lib.moe_linear_init(ctypes.byref(moe.moe_linear_config(**sizes)), ctypes.byref(h))
            lib.moe_linear_destroy(h)
            # (without a GPU the sizes that it takes end with the missing device)
            assert code == UNSUP if past else code in (OK, moe.MOE_ERR_CUDA), sizes
