"""The feed-forward block's and the norm's calls refuse tensors, contexts and
streams of a device other than the one on which they would launch.  Host only:
stand-ins for tensors and for the library, nothing is launched."""
import ctypes

import pytest
import torch

import expert_routed_ffn_moe_gb300 as moe

BF, F32 = torch.bfloat16, torch.float32
T, D, I = 4, 64, 32


class Tensor:
    """What the checks look at, on cuda:`index`."""

    def __init__(self, shape, index, dtype=BF):
        self.shape, self.dtype, self.index = torch.Size(shape), dtype, index
        self.is_cuda, self.device = True, torch.device("cuda", index)

    def get_device(self):
        return self.index

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 4096

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return torch.empty(0, dtype=self.dtype).element_size()


class Stream:
    def __init__(self, index):
        self.device_index, self.device, self.cuda_stream = index, torch.device("cuda", index), 77


class Library:
    """Counts the calls that would reach the device."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            if name == "moe_add_norm_workspace":
                return 64
            if name not in ("moe_ffn_init", "moe_ffn_destroy"):
                self.calls.append(name)
            return moe.MOE_OK

        return call


@pytest.fixture
def host(monkeypatch):
    """host.current: the current device."""
    class Host:
        current, lib = 0, Library()

    monkeypatch.setattr(moe, "_lib", Host.lib)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: Host.current)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: Host.current, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 5, raising=False)
    return Host


def mx(rows, cols, index):
    return [Tensor((rows, cols), index, torch.float8_e4m3fn),
            Tensor((moe._mx_bytes(rows, cols),), index, torch.uint8)]


def calls(at):
    """{name: (call(operands, stream), operands)}, every operand on device `at`; all outputs are given."""
    x, w = Tensor((T, D), at), Tensor((D,), at)
    gu, dn, pre = Tensor((2 * I, D), at), Tensor((D, I), at), Tensor((T, 2 * I), at)
    ws = Tensor((64,), at, torch.uint8)
    return {
        "norm": (lambda o, st: moe.moe_add_norm(o[0], o[1], o[2], 1e-6, o[3], o[4], stream=st), [x, x, w, x, x]),
        "norm_mx8": (lambda o, st: moe.moe_add_norm(o[0], o[1], o[2], 1e-6, o[3], o[4], o[5], stream=st),
                     [x, x, w, x] + mx(T, D, at)),
        "norm_backward": (lambda o, st: moe.moe_add_norm_backward(o[0], o[1], o[2], o[3], 1e-6, o[4], o[5], o[6],
                                                                  stream=st), [x, w, x, x, x, w, ws]),
        "quantize": (lambda o, st: moe.moe_quantize_mx(o[0], o[1], o[2]), [x] + mx(T, D, at)),
        "ffn": (lambda o, st: moe.GatedFfn(D, I, T).forward(o[0], o[1], o[2], o[3], o[4]), [x, gu, dn, x, pre]),
        "ffn_mx8": (lambda o, st: moe.GatedFfn(D, I, T, weight_format=moe.MOE_W_MX8).forward(
            o[0:2], o[2:4], o[4:6], o[6]), mx(T, D, at) + mx(2 * I, D, at) + mx(D, I, at) + [x]),
        "ffn_backward": (lambda o, st: moe.GatedFfn(D, I, T, training=True).backward(*o),
                         [x, pre, gu, dn, x, x, gu, dn]),
    }


NAMES = sorted(calls(0))


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("current", [0, 1])
def test_all_on_the_current_device_is_launched(host, name, current):
    host.current, host.lib.calls = current, []
    call, ops = calls(current)[name]
    call(ops, None)
    assert len(host.lib.calls) == 1


@pytest.mark.parametrize("name", NAMES)
def test_all_on_another_device_is_refused(host, name):
    host.lib.calls = []
    call, ops = calls(1)[name]
    with pytest.raises(ValueError, match="device"):
        call(ops, None)
    assert not host.lib.calls


@pytest.mark.parametrize("name", NAMES)
def test_one_operand_on_another_device_is_refused(host, name):
    host.lib.calls = []
    there = calls(1)[name][1]
    for i in range(len(there)):
        call, ops = calls(0)[name]
        ops[i] = there[i]
        with pytest.raises(ValueError, match="device"):
            call(ops, None)
    assert not host.lib.calls


@pytest.mark.parametrize("name", ["norm", "norm_mx8", "norm_backward"])
def test_a_stream_of_another_device_is_refused(host, name):
    host.lib.calls = []
    call, ops = calls(0)[name]
    call(ops, Stream(0))
    assert len(host.lib.calls) == 1
    with pytest.raises(ValueError, match="device"):
        call(ops, Stream(1))
    assert len(host.lib.calls) == 1


def test_a_context_of_another_device_is_refused(host):
    host.lib.calls = []
    ffn, ffn8 = moe.GatedFfn(D, I, T, training=True), moe.GatedFfn(D, I, T, weight_format=moe.MOE_W_MX8)
    host.current = 1  # the tensors' device, not the contexts'
    c = calls(1)
    x, gu, dn, y, pre = c["ffn"][1]
    o = c["ffn_mx8"][1]
    for call in (lambda: ffn.forward(x, gu, dn, y, pre), lambda: ffn.backward(*c["ffn_backward"][1]),
                 lambda: ffn8.forward(o[0:2], o[2:4], o[4:6], o[6])):
        with pytest.raises(ValueError, match="device"):
            call()
    assert not host.lib.calls


def test_the_classes_that_make_their_outputs_refuse_too(host):
    host.lib.calls = []
    op = moe.AddNorm(D)
    here, there = calls(0)["norm"][1], calls(1)["norm"][1]
    for a in (there, [there[0], here[1], here[2]], [here[0], there[1], here[2]], [here[0], here[1], there[2]]):
        with pytest.raises(ValueError, match="device"):
            op.forward(a[0], a[1], a[2], s_out=a[1])
        with pytest.raises(ValueError, match="device"):
            op.backward(a[0], a[2], a[1])
    assert not host.lib.calls


def test_a_tensor_of_the_host_is_still_named_as_such(host):
    x, w = torch.zeros(T, D, dtype=BF), torch.zeros(D, dtype=BF)
    for call in (lambda: moe.AddNorm(D).forward(x, None, w), lambda: moe.moe_quantize_mx(x),
                 lambda: moe.GatedFfn(D, I, T).forward(x, x, x)):
        with pytest.raises(ValueError, match="must be a contiguous CUDA tensor"):
            call()


def test_status_and_close_wait_for_the_contexts_device(host, monkeypatch):
    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, host.current = host.current, self.index

        def __exit__(self, *args):
            host.current = self.before

    seen = []
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(moe, "moe_ffn_status", lambda ctx: seen.append(("status", host.current)) or moe.MOE_OK)
    monkeypatch.setattr(moe, "moe_ffn_destroy", lambda ctx: seen.append(("close", host.current)))
    ffn = moe.GatedFfn(D, I, T)
    ffn.ctx = ctypes.c_void_p(16)  # (a handle that only the functions above get)
    host.current = 1
    assert ffn.status() == moe.MOE_OK
    ffn.close()
    assert seen == [("status", 0), ("close", 0)] and host.current == 1 and ffn.ctx is None
