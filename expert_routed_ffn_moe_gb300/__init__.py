"""Python binding of the GB300 routed-expert SwiGLU MoE layer.

Thin ctypes marshalling over the C ABI in ``include/moe.h`` (same function
names): tensors are passed as device pointers, the stream is torch's current
stream.  Every step of the layer runs in the CUDA kernels of
``libmoe_gb300.so``; there is no fallback, and the functions raise if the
library has not been built.
"""
from __future__ import annotations

import ctypes
import os
import re

from ._build import LIB, build  # noqa: F401

MOE_OK, MOE_ERR_ARG, MOE_ERR_ALIGN, MOE_ERR_UNSUPPORTED, MOE_ERR_CUDA, MOE_ERR_TIMEOUT, MOE_ERR_BOUNDS, \
    MOE_ERR_NOMEM = range(8)
MOE_F32, MOE_BF16, MOE_MX8 = 0, 1, 2
MOE_W_BF16, MOE_W_Q4G64, MOE_W_MX8 = 0, 1, 2
MOE_ACT_SILU, MOE_ACT_GELU = 0, 1
MOE_PATH_AUTO, MOE_PATH_GEMV, MOE_PATH_GEMM = 0, 1, 2
MOE_ROUTER_AUTO, MOE_ROUTER_SIMT, MOE_ROUTER_TENSOR = 0, 1, 2
(MOE_K_ROUTER, MOE_K_SELECT, MOE_K_GROUP, MOE_K_GEMV_GATE_UP, MOE_K_GEMV_DOWN, MOE_K_GEMM_GATE_UP, MOE_K_GEMM_DOWN,
 MOE_K_COMBINE, MOE_K_DECODE_FUSED) = range(9)

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "moe.h")


class MoeError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {moe_strerror(code)} (code {code})")
        self.code = code


class moe_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("d", "n_experts", "inter", "shared_inter", "top_k", "max_tokens",
                                            "x_dtype", "has_router_bias", "has_shared", "bias_select_only",
                                            "shared_gate", "weight_format")]


class moe_ffn_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("d", "inter", "max_tokens", "activation", "weight_format", "training")]


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded C library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB):
            raise RuntimeError(f"{os.path.basename(LIB)} is not built: run __graft_entry__.build() first")
        L = ctypes.CDLL(LIB)
        P, I, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
        L.moe_init.argtypes = [ctypes.POINTER(moe_config), ctypes.POINTER(P)]
        L.moe_route.argtypes = [P, P, I, P, P, I, P, P, P, P, P, P]
        L.moe_forward.argtypes = [P, P, I, P, P, P, P, P, I, P, P]
        L.moe_set_path.argtypes = [P, I]
        L.moe_set_router.argtypes = [P, I]
        L.moe_set_spin_limit.argtypes = [P, ctypes.c_longlong]
        L.moe_record_event.argtypes = [P, P]
        L.moe_record_event.restype = I
        L.moe_set_chunk_tokens.argtypes = [P, I]
        L.moe_set_chunk_tokens.restype = I
        L.moe_set_overlap.argtypes = [P, I]
        L.moe_set_overlap.restype = I
        L.moe_set_prefetch.argtypes = [P, P, P]
        L.moe_set_prefetch.restype = I
        L.moe_inject_stall.argtypes = [P, I]
        L.moe_inject_stall.restype = I
        L.moe_time_kernel.argtypes = [P, I, P, P]
        L.moe_time_kernel.restype = I
        L.moe_launch_count.argtypes = [P]
        L.moe_launch_count.restype = ctypes.c_longlong
        L.moe_decode_noalloc.argtypes = [P, I, I, I, I, I, I, P, P, P, P, P, P, P, P]
        L.moe_decode_noalloc.restype = I
        L.moe_last_routing.argtypes = [P, P, P, P, P, P, P, ctypes.POINTER(I), ctypes.POINTER(I), P]
        L.moe_last_routing.restype = I
        L.moe_add_norm.argtypes = [P, I, P, I, P, I, I, I, F, P, P, I, P, P]
        L.moe_add_norm_backward.argtypes = [P, P, P, P, I, I, I, I, F, P, P, P, P]
        L.moe_quantize_mx.argtypes = [P, I, I, I, P, P, P]
        L.moe_ffn_init.argtypes = [ctypes.POINTER(moe_ffn_config), ctypes.POINTER(P)]
        L.moe_ffn_forward.argtypes = [P, P, P, I, P, P, P, P, P, P, P]
        L.moe_ffn_backward.argtypes = [P, P, P, I, P, P, P, P, P, P, P]
        L.moe_ffn_set_spin_limit.argtypes = [P, ctypes.c_longlong]
        L.moe_ffn_inject_stall.argtypes = [P, I]
        L.moe_ffn_status.argtypes = [P]
        for f in ("moe_ffn_set_spin_limit", "moe_ffn_inject_stall", "moe_add_norm", "moe_add_norm_backward",
                  "moe_quantize_mx", "moe_ffn_init", "moe_ffn_forward", "moe_ffn_backward", "moe_ffn_status"):
            getattr(L, f).restype = I
        L.moe_add_norm_workspace.argtypes = [I]
        L.moe_mx_scale_bytes.argtypes = [I, I]
        L.moe_ffn_launch_count.argtypes = [P]
        for f in ("moe_add_norm_workspace", "moe_mx_scale_bytes", "moe_ffn_launch_count"):
            getattr(L, f).restype = ctypes.c_longlong
        L.moe_ffn_destroy.argtypes = [P]
        L.moe_ffn_destroy.restype = None
        L.moe_status.argtypes = [P]
        L.moe_strerror.argtypes = [I]
        L.moe_strerror.restype = ctypes.c_char_p
        L.moe_destroy.argtypes = [P]
        L.moe_destroy.restype = None
        for f in ("moe_init", "moe_route", "moe_forward", "moe_set_path", "moe_set_router", "moe_set_spin_limit",
                  "moe_status"):
            getattr(L, f).restype = I
        _lib = L
    return _lib


def header_functions() -> list[str]:
    """Names of the functions declared in include/moe.h."""
    text = open(HEADER).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(moe_[a-z_]+)\s*\(", text)))


def _check(code: int, what: str) -> None:
    if code != MOE_OK:
        raise MoeError(code, what)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    import torch

    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _need_cuda(t, name, dtype=None):
    if t is None:
        return
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")


def moe_strerror(code: int) -> str:
    return lib().moe_strerror(code).decode()


def moe_init(d, n_experts, inter, shared_inter, top_k, max_tokens, x_dtype=MOE_BF16, has_router_bias=False,
             has_shared=True, bias_select_only=False, shared_gate=False,
             weight_format=MOE_W_BF16) -> ctypes.c_void_p:
    cfg = moe_config(d, n_experts, inter, shared_inter, top_k, max_tokens, x_dtype, int(has_router_bias),
                     int(has_shared), int(bias_select_only), int(shared_gate), int(weight_format))
    h = ctypes.c_void_p()
    _check(lib().moe_init(ctypes.byref(cfg), ctypes.byref(h)), "moe_init")
    return h


def moe_destroy(ctx) -> None:
    lib().moe_destroy(ctx)


def moe_set_path(ctx, path: int) -> None:
    _check(lib().moe_set_path(ctx, path), "moe_set_path")


def moe_set_router(ctx, router: int) -> None:
    _check(lib().moe_set_router(ctx, router), "moe_set_router")


def moe_set_spin_limit(ctx, limit_ns: int) -> None:
    _check(lib().moe_set_spin_limit(ctx, limit_ns), "moe_set_spin_limit")


def moe_record_event(event, stream=None) -> None:
    """Record a torch.cuda.Event on a stream; timeable also under graph capture."""
    _check(lib().moe_record_event(ctypes.c_void_p(event.cuda_event), _stream(stream)), "moe_record_event")


def moe_set_chunk_tokens(ctx, chunk: int) -> None:
    """Chunked prefill (see moe.h): with chunk > 0 moe_forward accepts any T and runs
    slices of at most `chunk` tokens through the context's bounded workspace."""
    _check(lib().moe_set_chunk_tokens(ctx, int(chunk)), "moe_set_chunk_tokens")


def moe_set_overlap(ctx, on: bool) -> None:
    """Launch the fused small-T kernel with programmatic stream serialization
    (see moe.h); the caller promises the preceding work does not write the weights."""
    _check(lib().moe_set_overlap(ctx, 1 if on else 0), "moe_set_overlap")


def moe_set_prefetch(ctx, next_router_w=None, next_shared_w=None) -> None:
    """Hint: the next small-T forward pulls these next-layer weights into L2."""
    _check(lib().moe_set_prefetch(ctx, _ptr(next_router_w), _ptr(next_shared_w)), "moe_set_prefetch")


def moe_inject_stall(ctx, on: bool) -> None:
    _check(lib().moe_inject_stall(ctx, int(on)), "moe_inject_stall")


def moe_time_kernel(ctx, kernel_id: int, ev_start, ev_stop) -> None:
    """Arm the next call to record torch.cuda.Event pair around kernel `kernel_id`."""
    _check(lib().moe_time_kernel(ctx, kernel_id, ctypes.c_void_p(ev_start.cuda_event),
                                 ctypes.c_void_p(ev_stop.cuda_event)), "moe_time_kernel")


def moe_launch_count(ctx) -> int:
    return lib().moe_launch_count(ctx)


def moe_status(ctx) -> int:
    return lib().moe_status(ctx)


def moe_route(ctx, x, router_w, router_b, top_k, idx=None, w=None, counts=None, offsets=None, perm=None,
              stream=None) -> None:
    import torch

    for name, t, dt in (("x", x, None), ("router_w", router_w, torch.float32), ("router_b", router_b, torch.float32),
                        ("idx", idx, torch.int32), ("w", w, torch.float32), ("counts", counts, torch.int32),
                        ("offsets", offsets, torch.int32), ("perm", perm, torch.int32)):
        _need_cuda(t, name, dt)
    _check(lib().moe_route(ctx, _ptr(x), x.shape[0], _ptr(router_w), _ptr(router_b), top_k, _ptr(idx), _ptr(w),
                           _ptr(counts), _ptr(offsets), _ptr(perm), _stream(stream)), "moe_route")


def moe_forward(ctx, x, router_w, router_b, experts_gate_up, experts_down, shared_w, top_k, y,
                stream=None, packed_weights=False) -> None:
    """``packed_weights``: the expert tensors are 4-bit planes (MOE_W_Q4G64, see
    moe.h), passed as raw byte buffers of any dtype."""
    import torch

    wdt = None if packed_weights else torch.bfloat16
    for name, t, dt in (("x", x, None), ("router_w", router_w, torch.float32), ("router_b", router_b, torch.float32),
                        ("experts_gate_up", experts_gate_up, wdt),
                        ("experts_down", experts_down, wdt), ("shared_w", shared_w, wdt),
                        ("y", y, x.dtype)):
        _need_cuda(t, name, dt)
    _check(lib().moe_forward(ctx, _ptr(x), x.shape[0], _ptr(router_w), _ptr(router_b), _ptr(experts_gate_up),
                             _ptr(experts_down), _ptr(shared_w), top_k, _ptr(y), _stream(stream)), "moe_forward")


def moe_last_routing(ctx, n_experts, stream=None) -> dict:
    """The routing tables the last ``moe_forward`` on ``ctx`` computed and used
    (idx, w, counts, offsets, perm, slot), as device tensors; see moe.h."""
    import torch

    T, k = ctypes.c_int(), ctypes.c_int()
    _check(lib().moe_last_routing(ctx, None, None, None, None, None, None, ctypes.byref(T), ctypes.byref(k), None),
           "moe_last_routing")
    T, k = T.value, k.value
    dev = torch.device("cuda", torch.cuda.current_device())
    out = dict(idx=torch.empty(T, k, dtype=torch.int32, device=dev), w=torch.empty(T, k, dtype=torch.float32, device=dev),
               counts=torch.empty(n_experts, dtype=torch.int32, device=dev),
               offsets=torch.empty(n_experts + 1, dtype=torch.int32, device=dev),
               perm=torch.empty(T * k, dtype=torch.int32, device=dev),
               slot=torch.empty(T, k, dtype=torch.int32, device=dev))
    _check(lib().moe_last_routing(ctx, _ptr(out["idx"]), _ptr(out["w"]), _ptr(out["counts"]), _ptr(out["offsets"]),
                                  _ptr(out["perm"]), _ptr(out["slot"]), None, None, _stream(stream)),
           "moe_last_routing")
    return out


def moe_decode_noalloc(x, router_w, router_b, experts_gate_up, experts_down, shared_w, top_k, y, status=None,
                       stream=None) -> None:
    """The small-T layer without a context, for callers that cannot allocate
    device memory (a plugin whose host owns every device buffer, a serving loop
    that must not risk an allocation's device synchronisation).  Scratch memory
    is a fixed device array inside the library; see moe.h."""
    import torch

    for name, t, dt in (("x", x, None), ("router_w", router_w, torch.float32), ("router_b", router_b, torch.float32),
                        ("experts_gate_up", experts_gate_up, torch.bfloat16),
                        ("experts_down", experts_down, torch.bfloat16), ("shared_w", shared_w, torch.bfloat16),
                        ("y", y, x.dtype), ("status", status, torch.int32)):
        _need_cuda(t, name, dt)
    T, d = x.shape
    E, inter = experts_down.shape[0], experts_down.shape[2]
    x_dtype = MOE_BF16 if x.dtype == torch.bfloat16 else MOE_F32
    _check(lib().moe_decode_noalloc(_ptr(x), T, x_dtype, d, E, inter, top_k, _ptr(router_w), _ptr(router_b),
                                    _ptr(experts_gate_up), _ptr(experts_down), _ptr(shared_w), _ptr(y), _ptr(status),
                                    _stream(stream)), "moe_decode_noalloc")


class MoeLayer:
    """Owns one context; ``forward`` / ``route`` call the C ABI on torch tensors."""

    def __init__(self, d, n_experts, inter, top_k, max_tokens, *, shared_inter=None, x_dtype=MOE_BF16,
                 has_router_bias=False, has_shared=True, bias_select_only=False, shared_gate=False,
                 weight_format=MOE_W_BF16):
        """``shared_gate``: sigmoid-gated shared expert; router_w then holds n_experts + 1
        rows, the last being the gate vector.  ``weight_format``: MOE_W_BF16, or
        MOE_W_Q4G64 for 4-bit experts (planes as in moe.h; see ``pack_q4``)."""
        self.top_k = top_k
        self.d = d
        self.n_experts = n_experts
        self.x_dtype = x_dtype
        self.weight_format = weight_format
        self.ctx = moe_init(d, n_experts, inter, inter if shared_inter is None else shared_inter, top_k,
                            max_tokens, x_dtype, has_router_bias, has_shared, bias_select_only, shared_gate,
                            weight_format)

    def forward(self, x, router_w, router_b, gate_up, down, shared_w, y=None, top_k=None, stream=None):
        import torch

        if y is None:
            y = torch.empty_like(x)
        moe_forward(self.ctx, x, router_w, router_b, gate_up, down, shared_w, top_k or self.top_k, y, stream,
                    packed_weights=self.weight_format == MOE_W_Q4G64)
        return y

    def route(self, x, router_w, router_b, top_k=None, stream=None):
        import torch

        k = top_k or self.top_k
        T = x.shape[0]
        E = self.n_experts
        dev = x.device
        out = dict(idx=torch.empty(T, k, dtype=torch.int32, device=dev),
                   w=torch.empty(T, k, dtype=torch.float32, device=dev),
                   counts=torch.empty(E, dtype=torch.int32, device=dev),
                   offsets=torch.empty(E + 1, dtype=torch.int32, device=dev),
                   perm=torch.empty(T * k, dtype=torch.int32, device=dev))
        moe_route(self.ctx, x, router_w, router_b, k, stream=stream, **out)
        return out

    def last_routing(self, stream=None) -> dict:
        """Routing tables of the last ``forward`` (device tensors)."""
        return moe_last_routing(self.ctx, self.n_experts, stream)

    def status(self) -> int:
        return moe_status(self.ctx)

    def close(self):
        if self.ctx:
            moe_destroy(self.ctx)
            self.ctx = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ---------------------------------------------------------------- feed-forward block and its norm
# These calls take a few microseconds on the device, so the checks are kept
# cheap: tensors' properties are compared directly, and the stream's handle is
# read without making a stream object.  Calls that make tensors make them as the
# given stream's: with memory of the present stream a call on another one could
# write what kernels on the present one still read.
#
# A call is launched on the current device.  Its tensors, its stream and its
# context must be of that device: anything else would hand a kernel addresses of
# another device's memory.
_torch = None
_DTYPES = {}  # torch dtype -> MOE_F32 / MOE_BF16


def _t():
    global _torch
    if _torch is None:
        import torch

        _DTYPES.update({torch.float32: MOE_F32, torch.bfloat16: MOE_BF16})
        _torch = torch
    return _torch


def _device(t, name, home=None):
    """The index of the current device, after the check that t and the context (made on ``home``) are of it."""
    device = t.get_device()
    if device < 0:  # (the host's)
        raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if device != _torch._C._cuda_getDevice():
        raise ValueError(f"{name} is on device {device}, but the current device is {_torch._C._cuda_getDevice()}")
    if home is not None and home != device:
        raise ValueError(f"the context was made on device {home}, but the current device is {device}")
    return device


def _handle(stream, device):
    if stream is None:
        return _torch._C._cuda_getCurrentRawStream(device)
    if stream.device_index != device:
        raise ValueError(f"the stream is of device {stream.device_index}, but the current device is {device}")
    return stream.cuda_stream


def _checked(t, name, shape, device, dtype=None):
    """t's address, after the checks; None for None.  Without ``dtype`` t is float32 or bfloat16."""
    if t is None:
        return None
    if t.get_device() == device and t.shape == shape and (t.dtype in _DTYPES if dtype is None else t.dtype is dtype) \
            and t.is_contiguous():  # (a tensor of the host has device -1)
        return t.data_ptr()
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if t.get_device() != device:
        raise ValueError(f"{name} is on device {t.get_device()}, but the current device is {device}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be {'float32 or bfloat16' if dtype is None else dtype}, got {t.dtype}")


def _rows(t, name, cols=None):
    shape = t.shape
    if len(shape) != 2 or (cols is not None and shape[1] != cols):
        raise ValueError(f"{name} must have shape [rows, {'cols' if cols is None else cols}], got {tuple(shape)}")
    if shape[0] > 0x7fffffff or shape[1] > 0x7fffffff:
        raise ValueError(f"{name} of shape {tuple(shape)}: more rows or columns than an int holds")
    return shape


def _mx_bytes(rows, cols):
    return (rows + 127) // 128 * ((cols + 127) // 128) * 512


def moe_mx_scale_bytes(rows: int, cols: int) -> int:
    """Bytes of the scales of an mx8 matrix (MOE_MX8, see moe.h)."""
    return lib().moe_mx_scale_bytes(rows, cols)


def _mx_checked(pair, name, rows, cols, device):
    """Addresses of the codes and scales of an mx8 matrix, after the checks."""
    if not isinstance(pair, (tuple, list)) or len(pair) != 2:
        raise ValueError(f"{name} must be a pair (codes, scales)")
    codes, scales = pair
    if not (codes.is_cuda and scales.is_cuda and codes.is_contiguous() and scales.is_contiguous()):
        raise ValueError(f"{name} codes and scales must be contiguous CUDA tensors")
    if codes.get_device() != device or scales.get_device() != device:
        raise ValueError(f"{name} codes and scales are on devices {codes.get_device()} and {scales.get_device()}, but "
                         f"the current device is {device}")
    if codes.dtype != _t().float8_e4m3fn and codes.dtype != _torch.uint8:
        raise ValueError(f"{name} codes must be float8_e4m3fn or uint8, got {codes.dtype}")
    if codes.shape != (rows, cols):
        raise ValueError(f"{name} codes must have shape {(rows, cols)}, got {tuple(codes.shape)}")
    if scales.element_size() != 1 or scales.numel() != _mx_bytes(rows, cols):
        raise ValueError(f"{name} scales must be {_mx_bytes(rows, cols)} bytes, got {scales.numel()} of {scales.dtype}")
    return codes.data_ptr(), scales.data_ptr()


def _mx_empty(rows, cols, device):
    torch = _t()
    return (torch.empty(rows, cols, dtype=torch.float8_e4m3fn, device=device),
            torch.empty(_mx_bytes(rows, cols), dtype=torch.uint8, device=device))


def moe_quantize_mx(v, codes=None, scales=None, stream=None):
    """Round a float32 or bfloat16 matrix to mx8: (codes, scales), into the given ones; see moe.h."""
    torch = _t()
    if stream is not None:
        with torch.cuda.stream(stream):
            return moe_quantize_mx(v, codes, scales)
    rows, cols = _rows(v, "v")
    device = _device(v, "v")
    pv = _checked(v, "v", v.shape, device)
    if codes is None:
        codes = torch.empty(rows, cols, dtype=torch.float8_e4m3fn, device=v.device)
    if scales is None:
        scales = torch.empty(_mx_bytes(rows, cols), dtype=torch.uint8, device=v.device)
    pc, ps = _mx_checked((codes, scales), "output", rows, cols, device)
    _check(lib().moe_quantize_mx(pv, _DTYPES[v.dtype], rows, cols, pc, ps, _handle(None, device)), "moe_quantize_mx")
    return codes, scales


def moe_add_norm(x, residual, weight, eps, s_out, y, y_scales=None, stream=None) -> None:
    """See moe.h.  ``y`` is float32, bfloat16, or float8_e4m3fn codes with ``y_scales``."""
    torch = _t()
    shape = _rows(x, "x")
    T, d = shape
    device = _device(x, "x")
    px, pr = _checked(x, "x", shape, device), _checked(residual, "residual", shape, device)
    ps = _checked(s_out, "s_out", shape, device, None if residual is None else residual.dtype)
    pw = _checked(weight, "weight", (d,), device)
    if y.dtype == torch.float8_e4m3fn:
        if y_scales is None:
            raise ValueError("y_scales are needed for float8_e4m3fn codes")
        py, pys = _mx_checked((y, y_scales), "y", T, d, device)
        y_dtype = MOE_MX8
    else:
        py, pys = _checked(y, "y", shape, device), None if y_scales is None else y_scales.data_ptr()
        y_dtype = _DTYPES[y.dtype]
    s_like = residual if residual is not None else s_out
    _check(lib().moe_add_norm(px, _DTYPES[x.dtype], pr, MOE_F32 if s_like is None else _DTYPES[s_like.dtype], pw,
                              _DTYPES[weight.dtype], T, d, eps, ps, py, y_dtype, pys, _handle(stream, device)),
           "moe_add_norm")


def moe_add_norm_backward(s, weight, dy, ds, eps, dx, dweight, workspace, stream=None) -> None:
    """See moe.h.  ``ds``, ``dx`` and ``dweight`` may be None."""
    _t()
    shape = _rows(s, "s")
    T, d = shape
    device = _device(s, "s")
    ps, pw = _checked(s, "s", shape, device), _checked(weight, "weight", (d,), device)
    pdy, pds, pdx = (_checked(t, n, shape, device, s.dtype) for n, t in (("dy", dy), ("ds", ds), ("dx", dx)))
    pdw = _checked(dweight, "dweight", (d,), device, weight.dtype)
    pws = None
    if workspace is not None:
        if not workspace.is_cuda or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous CUDA tensor")
        if workspace.get_device() != device:
            raise ValueError(f"workspace is on device {workspace.get_device()}, but the current device is {device}")
        if workspace.numel() * workspace.element_size() < lib().moe_add_norm_workspace(d):
            raise ValueError("workspace is smaller than moe_add_norm_workspace(d) bytes")
        pws = workspace.data_ptr()
    _check(lib().moe_add_norm_backward(ps, pw, pdy, pds, _DTYPES[s.dtype], _DTYPES[weight.dtype], T, d, eps, pdx, pdw,
                                       pws, _handle(stream, device)), "moe_add_norm_backward")


class AddNorm:
    """The norm of rows of width ``d`` with the residual's addition.  Holds no
    device memory: a backward call takes its workspace from its stream's."""

    def __init__(self, d, eps=1e-6):
        self.d = d
        self.eps = float(eps)
        self._workspace_bytes = lib().moe_add_norm_workspace(d)

    def forward(self, x, residual, weight, y_dtype=MOE_BF16, s_out=None, stream=None):
        """(y, s): y in ``y_dtype`` (MOE_MX8: the pair (codes, scales)), s = x + residual
        in the residual's dtype (x's without a residual)."""
        torch = _t()
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.forward(x, residual, weight, y_dtype, s_out)
        shape = _rows(x, "x", self.d)
        T, d = shape
        device = _device(x, "x")
        px, pr, pw = _checked(x, "x", shape, device), _checked(residual, "residual", shape, device), \
            _checked(weight, "weight", (d,), device)
        like = x if residual is None else residual
        if s_out is None:
            s_out = torch.empty_like(like)
        else:
            _checked(s_out, "s_out", shape, device, like.dtype)
        pys = None
        if y_dtype == MOE_BF16:
            y = torch.empty_like(x, dtype=torch.bfloat16)
            py = y.data_ptr()
        elif y_dtype == MOE_F32:
            y = torch.empty_like(x, dtype=torch.float32)
            py = y.data_ptr()
        elif y_dtype == MOE_MX8:
            y = _mx_empty(T, d, x.device)
            py, pys = y[0].data_ptr(), y[1].data_ptr()
        else:
            raise ValueError("y_dtype must be MOE_F32, MOE_BF16 or MOE_MX8")
        code = (_lib or lib()).moe_add_norm(px, _DTYPES[x.dtype], pr, _DTYPES[like.dtype], pw, _DTYPES[weight.dtype], T,
                                            d, self.eps, s_out.data_ptr(), py, y_dtype, pys, _handle(None, device))
        if code:
            _check(code, "moe_add_norm")
        return y, s_out

    def backward(self, s, weight, dy, ds=None, stream=None):
        """(dx, dweight); dx is the gradient of x and of the residual alike.  dy and ds have s's dtype."""
        torch = _t()
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.backward(s, weight, dy, ds)
        shape = _rows(s, "s", self.d)
        T, d = shape
        dtype = s.dtype
        device = _device(s, "s")
        ps, pw, pdy = _checked(s, "s", shape, device), _checked(weight, "weight", (d,), device), \
            _checked(dy, "dy", shape, device, dtype)
        pds = _checked(ds, "ds", shape, device, dtype)
        dx, dweight = torch.empty_like(s), torch.empty_like(weight)
        workspace = torch.empty(self._workspace_bytes, dtype=torch.uint8, device=s.device)
        code = (_lib or lib()).moe_add_norm_backward(ps, pw, pdy, pds, _DTYPES[dtype], _DTYPES[weight.dtype], T, d,
                                                     self.eps, dx.data_ptr(), dweight.data_ptr(), workspace.data_ptr(),
                                                     _handle(None, device))
        if code:
            _check(code, "moe_add_norm_backward")
        return dx, dweight


def moe_ffn_init(d, inter, max_tokens, activation=MOE_ACT_SILU, weight_format=MOE_W_BF16,
                 training=False) -> ctypes.c_void_p:
    cfg = moe_ffn_config(d, inter, max_tokens, activation, weight_format, int(training))
    h = ctypes.c_void_p()
    _check(lib().moe_ffn_init(ctypes.byref(cfg), ctypes.byref(h)), "moe_ffn_init")
    return h


def moe_ffn_destroy(ctx) -> None:
    lib().moe_ffn_destroy(ctx)


def moe_ffn_status(ctx) -> int:
    return lib().moe_ffn_status(ctx)


def moe_ffn_set_spin_limit(ctx, limit_ns: int) -> None:
    _check(lib().moe_ffn_set_spin_limit(ctx, limit_ns), "moe_ffn_set_spin_limit")


def moe_ffn_inject_stall(ctx, on: bool) -> None:
    _check(lib().moe_ffn_inject_stall(ctx, int(on)), "moe_ffn_inject_stall")


def moe_ffn_launch_count(ctx) -> int:
    return lib().moe_ffn_launch_count(ctx)


class GatedFfn:
    """Owns one context of the dense gated feed-forward block (moe_ffn_*, see moe.h);
    with MOE_W_MX8 x and the weights are pairs (codes, scales)."""

    def __init__(self, d, inter, max_tokens, *, activation=MOE_ACT_SILU, weight_format=MOE_W_BF16, training=False):
        self.ctx = None
        self.d, self.inter, self.mx = d, inter, weight_format == MOE_W_MX8
        self.ctx = moe_ffn_init(d, inter, max_tokens, activation, weight_format, training)
        self.device = _t().cuda.current_device()

    def forward(self, x, gate_up, down, y=None, pre=None, save=False, stream=None):
        """y, or (y, pre) with ``save`` (pre: the pre-activations that ``backward`` needs)."""
        torch = _t()
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.forward(x, gate_up, down, y, pre, save)
        d, I, bf16 = self.d, self.inter, torch.bfloat16
        if self.mx:
            rows = x[0] if isinstance(x, (tuple, list)) else x
            T = _rows(rows, "x", d)[0]
            device = _device(rows, "x", self.device)
            px, pxs = _mx_checked(x, "x", T, d, device)
            pg, pgs = _mx_checked(gate_up, "gate_up", 2 * I, d, device)
            pd, pds = _mx_checked(down, "down", d, I, device)
        else:
            rows = x
            T = _rows(x, "x", d)[0]
            device = _device(x, "x", self.device)
            px, pg, pd = _checked(x, "x", (T, d), device, bf16), \
                _checked(gate_up, "gate_up", (2 * I, d), device, bf16), _checked(down, "down", (d, I), device, bf16)
            pxs = pgs = pds = None
        if y is None:
            y = torch.empty_like(rows, dtype=bf16) if self.mx else torch.empty_like(x)
            py = y.data_ptr()
        else:
            py = _checked(y, "y", (T, d), device, bf16)
        if pre is None and save:
            pre = torch.empty(T, 2 * I, dtype=bf16, device=rows.device)
        pp = _checked(pre, "pre", (T, 2 * I), device, bf16)
        code = (_lib or lib()).moe_ffn_forward(self.ctx, px, pxs, T, pg, pgs, pd, pds, py, pp, _handle(None, device))
        if code:
            _check(code, "moe_ffn_forward")
        return (y, pre) if pre is not None else y

    def backward(self, x, pre, gate_up, down, dy, dx=None, dgate_up=None, ddown=None, stream=None):
        """(dx, dgate_up, ddown); pass ``False`` for one of them to leave it out (None comes back)."""
        torch = _t()
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.backward(x, pre, gate_up, down, dy, dx, dgate_up, ddown)
        d, I, bf16 = self.d, self.inter, torch.bfloat16
        T = _rows(x, "x", d)[0]
        device = _device(x, "x", self.device)
        px, ppre, pdy = _checked(x, "x", (T, d), device, bf16), _checked(pre, "pre", (T, 2 * I), device, bf16), \
            _checked(dy, "dy", (T, d), device, bf16)
        pg, pd = _checked(gate_up, "gate_up", (2 * I, d), device, bf16), _checked(down, "down", (d, I), device, bf16)

        def output(t, name, like):
            if t is None:
                t = torch.empty_like(like)
                return t, t.data_ptr()
            return (None, None) if t is False else (t, _checked(t, name, like.shape, device, bf16))

        dx, pdx = output(dx, "dx", x)
        dgate_up, pdg = output(dgate_up, "dgate_up", gate_up)
        ddown, pdd = output(ddown, "ddown", down)
        code = (_lib or lib()).moe_ffn_backward(self.ctx, px, ppre, T, pg, pd, pdy, pdx, pdg, pdd,
                                                _handle(None, device))
        if code:
            _check(code, "moe_ffn_backward")
        return dx, dgate_up, ddown

    def status(self) -> int:
        with _t().cuda.device(self.device):  # (it waits for the current device)
            return moe_ffn_status(self.ctx)

    def close(self):
        if self.ctx:
            with _t().cuda.device(self.device):
                moe_ffn_destroy(self.ctx)
            self.ctx = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
