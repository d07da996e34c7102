"""The layer norm's, the token sort's and the product's calls refuse tensors, contexts and shapes that they
cannot take.  Host only, on the stand-ins of test_ffn_devices_cpu."""
import ctypes

import pytest
import torch

import expert_routed_ffn_moe_gb300 as moe
from test_ffn_devices_cpu import BF, F32, Library, Tensor, host  # noqa: F401

T, K, N, E, P = 4, 64, 32, 8, 2
I32 = torch.int32


@pytest.fixture(autouse=True)
def sizes(monkeypatch):
    monkeypatch.setattr(Library, "moe_layer_norm_workspace", lambda self, d: 64, raising=False)


def calls(at):
    """{name: (call(operands, stream), operands)}, every operand on device `at`; all outputs are given where they can be."""
    x, dy, w, b, n = Tensor((T, K), at), Tensor((T, N), at), Tensor((N, K), at), Tensor((N,), at), Tensor((K,), at)
    rows, f = Tensor((T * P, K), at), Tensor((T, P), at, F32)

    def ints(*s):
        return Tensor(s, at, I32)

    sort, lin = moe.TokenDispatch(E, P), lambda: moe.Linear(K, N, T, training=True)
    return {
        "sort": (lambda o, st: sort.sort(*o, stream=st), [ints(T, P), ints(E), ints(E + 1), ints(T * P), ints(T, P)]),
        "dispatch": (lambda o, st: sort.dispatch(*o, stream=st), [x, ints(T, P), rows]),
        "combine": (lambda o, st: sort.combine(*o, stream=st), [rows, ints(T, P), f, x, x]),
        "combine_backward": (lambda o, st: sort.combine_backward(*o, stream=st), [x, rows, ints(T, P), f, rows, f]),
        "linear": (lambda o, st: lin().forward(*o[:5], pre=o[5], stream=st), [x, w, b, dy, dy, dy]),
        "linear_backward": (lambda o, st: lin().backward(*o, stream=st), [x, dy, w, b, dy, x, w, b]),
    }


NAMES = sorted(calls(0))


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("current", [0, 1])
def test_all_on_the_current_device_is_launched(host, name, current):  # noqa: F811
    host.current, host.lib.calls = current, []
    call, ops = calls(current)[name]
    call(ops, None)
    assert [c for c in host.lib.calls if c not in ("moe_linear_init", "moe_linear_destroy")] == \
        ["moe_sort_tokens" if name == "sort" else "moe_linear_forward" if name == "linear" else "moe_" + name]


@pytest.mark.parametrize("name", NAMES)
def test_an_operand_on_another_device_is_refused(host, name):  # noqa: F811
    there = calls(1)[name][1]
    for i in range(len(there) + 1):
        call, ops = calls(0)[name]
        if i < len(there):
            ops[i] = there[i]
        else:
            ops = there
        host.lib.calls = []
        with pytest.raises(ValueError, match="device"):
            call(ops, None)
        assert not [c for c in host.lib.calls if c not in ("moe_linear_init", "moe_linear_destroy")]


@pytest.mark.parametrize("name", NAMES)
def test_a_wrong_shape_or_dtype_is_refused(host, name):  # noqa: F811
    good = calls(0)[name][1]
    for i, t in enumerate(good):
        for bad in (Tensor(t.shape + (1,), 0, t.dtype), Tensor((3,) + tuple(t.shape[1:]), 0, t.dtype),
                    Tensor(t.shape, 0, torch.float16)):
            if name == "dispatch" and i == 2 and bad.dtype == BF and len(bad.shape) == 2:
                continue  # (fewer rows are allowed: picks past them are dropped)
            if name == "combine" and i == 0 and bad.dtype == BF and len(bad.shape) == 2:
                continue
            call, ops = calls(0)[name]
            ops[i] = bad
            with pytest.raises(ValueError):
                call(ops, None)


def test_layer_norm_and_a_context_of_another_device(host):  # noqa: F811
    x, w = Tensor((T, K), 1), Tensor((K,), 1)
    for call in (lambda: moe.LayerNorm(K).forward(x, None, w), lambda: moe.LayerNorm(K).backward(x, w, x)):
        with pytest.raises(ValueError, match="device"):
            call()
    lin = moe.Linear(K, N, T)
    host.current = 1
    with pytest.raises(ValueError, match="context was made on device 0"):
        lin.forward(x, Tensor((N, K), 1))
    with pytest.raises(ValueError, match="weight must have shape"):
        moe.LayerNorm(K).forward(x, x, Tensor((K + 1,), 1))
    with pytest.raises(ValueError, match="y_dtype"):
        moe.LayerNorm(K).forward(x, x, w, y_dtype=moe.MOE_MX8)
    x = torch.zeros(T, K, dtype=BF)
    for call in (lambda: moe.LayerNorm(K).forward(x, None, None), lambda: moe.TokenDispatch(E, P).dispatch(x, x),
                 lambda: moe.TokenDispatch(E, P).sort(torch.zeros(T, P, dtype=I32))):
        with pytest.raises(ValueError, match="must be a contiguous CUDA tensor"):
            call()


def test_status_and_close_wait_for_the_contexts_device(host, monkeypatch):  # noqa: F811
    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, host.current = host.current, self.index

        def __exit__(self, *args):
            host.current = self.before

    seen = []
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(moe, "moe_linear_status", lambda ctx: seen.append(("status", host.current)) or moe.MOE_OK)
    monkeypatch.setattr(moe, "moe_linear_destroy", lambda ctx: seen.append(("close", host.current)))
    lin = moe.Linear(K, N, T)
    lin.ctx = ctypes.c_void_p(16)  # (a handle that only the functions above get)
    host.current = 1
    assert lin.status() == moe.MOE_OK
    lin.close()
    assert seen == [("status", 0), ("close", 0)] and host.current == 1 and lin.ctx is None
