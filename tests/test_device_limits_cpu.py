"""Grids and clusters that follow from what a device runs at a time: asked for each device, and asked again after an
answer that failed.  Host only, with a stand-in for the CUDA runtime's functions (no GPU, nothing runs)."""
import json
import os
import subprocess
import sys

import pytest

import expert_routed_ffn_moe_gb300 as moe
from expert_routed_ffn_moe_gb300 import _build

RUNTIME = r"""
#include <cuda_runtime_api.h>
#include <stdio.h>
#include <string.h>
int stand_device, stand_fail, stand_pending;  /* the current device; fail queries; the error that a failure leaves */
static const int sms[2] = {152, 64}, clusters[2] = {19, 8};
static cudaError_t answer(int* to, int v) {
  if (stand_fail) return (cudaError_t)(stand_pending = cudaErrorUnknown);
  *to = v;
  return cudaSuccess;
}
static int encode(void) { return 0; }
cudaError_t cudaGetDevice(int* d) { *d = stand_device; return cudaSuccess; }
cudaError_t cudaGetLastError(void) { cudaError_t e = (cudaError_t)stand_pending; stand_pending = 0; return e; }
cudaError_t cudaDeviceGetAttribute(int* v, enum cudaDeviceAttr a, int d) { (void)a; *v = sms[d]; return cudaSuccess; }
cudaError_t cudaOccupancyMaxActiveBlocksPerMultiprocessor(int* n, const void* f, int b, size_t s) {
  (void)f; (void)b; (void)s; return answer(n, 2);
}
cudaError_t cudaOccupancyMaxActiveBlocksPerMultiprocessorWithFlags(int* n, const void* f, int b, size_t s, unsigned g) {
  (void)f; (void)b; (void)s; (void)g; return answer(n, 2);
}
cudaError_t cudaOccupancyMaxActiveClusters(int* n, const void* f, const cudaLaunchConfig_t* c) {
  (void)f; (void)c; return answer(n, 2 * clusters[stand_device]);
}
cudaError_t cudaFuncSetAttribute(const void* f, enum cudaFuncAttribute a, int v) { (void)f; (void)a; (void)v; return cudaSuccess; }
cudaError_t cudaGetDeviceProperties(struct cudaDeviceProp* p, int d) {
  (void)d; memset(p, 0, sizeof *p); p->major = 10; p->minor = 3; p->multiProcessorCount = 152; return cudaSuccess;
}
cudaError_t cudaGetDriverEntryPointByVersion(const char* s, void** f, unsigned v, unsigned long long g,
                                             enum cudaDriverEntryPointQueryResult* q) {
  (void)s; (void)v; (void)g; *f = (void*)encode; *q = cudaDriverEntryPointSuccess; return cudaSuccess;
}
cudaError_t cudaMalloc(void** p, size_t n) { (void)n; *p = (void*)(1 << 20); return cudaSuccess; }
cudaError_t cudaFree(void* p) { (void)p; return cudaSuccess; }
cudaError_t cudaMemset(void* p, int v, size_t n) { (void)p; (void)v; (void)n; return cudaSuccess; }
cudaError_t cudaDeviceSynchronize(void) { return cudaSuccess; }
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void** args) {
  unsigned i, cluster = 1;
  (void)f; (void)args;
  for (i = 0; i < c->numAttrs; ++i)
    if (c->attrs[i].id == cudaLaunchAttributeClusterDimension) cluster = c->attrs[i].val.clusterDim.x;
  printf("launch %u %u\n", c->gridDim.x, cluster);
  fflush(stdout);
  return cudaSuccess;
}
"""

CALLS = r"""
import ctypes, json, sys
import expert_routed_ffn_moe_gb300 as moe
L, a, B, T = moe.lib(), ctypes.c_void_p(4096), moe.MOE_BF16, 20000
stand = ctypes.CDLL(None)
var = {n: ctypes.c_int.in_dll(stand, "stand_" + n) for n in ("device", "fail", "pending")}
linear = {}

def product(k, n):  # of the current device
    key = var["device"].value, k, n
    if key not in linear:
        linear[key] = moe.moe_linear_init(k, n, 16, training=True)
    return linear[key]

calls = {
    "layer_norm": lambda: L.moe_layer_norm(a, B, a, B, a, a, B, T, 4096, 1e-5, a, a, B, None),
    "layer_norm_odd": lambda: L.moe_layer_norm(a, B, a, B, a, a, B, T, 2501, 1e-5, a, a, B, None),
    "layer_norm_backward": lambda: L.moe_layer_norm_backward(a, a, a, a, B, B, T, 4096, 1e-5, a, a, a, a, None),
    "layer_norm_backward_odd": lambda: L.moe_layer_norm_backward(a, a, a, a, B, B, T, 2501, 1e-5, a, a, a, a, None),
    "combine": lambda: L.moe_combine(a, B, T, a, a, T, 1, 4096, a, a, B, None),
    "add_norm": lambda: L.moe_add_norm(a, B, a, B, a, B, T, 4096, 1e-6, a, a, B, None, None),
    "add_norm_odd": lambda: L.moe_add_norm(a, B, a, B, a, B, T, 2501, 1e-6, a, a, B, None, None),
    "add_norm_backward": lambda: L.moe_add_norm_backward(a, a, a, a, B, B, T, 4096, 1e-6, a, a, a, None),
    "add_norm_backward_odd": lambda: L.moe_add_norm_backward(a, a, a, a, B, B, T, 2501, 1e-6, a, a, a, None),
    "sort": lambda: L.moe_sort_tokens(a, T, 8, 256, a, a, a, a, None),
    "linear": lambda: L.moe_linear_forward(product(4096, 2048), a, 16, a, None, B, None, a, B, None, None),
    "linear_dx": lambda: L.moe_linear_backward(product(2048, 4096), a, None, 16, a, a, B, a, None, None, B, None),
}
for var["device"].value in (0, 1):
    product(4096, 2048), product(2048, 4096)
for device, fail in json.loads(sys.argv[2]):
    var["device"].value, var["fail"].value = device, fail
    print("call", flush=True)
    print("code", calls[sys.argv[1]](), var["pending"].value, flush=True)
"""

# {call: what its first kernel is launched with, (grid, cluster), on either device}
WANT = {"layer_norm": ((304, 1), (128, 1)), "layer_norm_odd": ((304, 1), (128, 1)),
        "layer_norm_backward": ((304, 1), (128, 1)), "layer_norm_backward_odd": ((304, 1), (128, 1)),
        "combine": ((304, 1), (128, 1)), "add_norm": ((304, 1), (128, 1)), "add_norm_odd": ((304, 1), (128, 1)),
        "add_norm_backward": ((304, 1), (128, 1)), "add_norm_backward_odd": ((304, 1), (128, 1)),
        "sort": ((16, 16), (16, 16)), "linear": ((128, 8), (64, 4)), "linear_dx": ((128, 8), (64, 4))}


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    """run(call, [(device, queries fail)]): of each [return code, error left behind, (grid, cluster) or None]."""
    moe.build()
    at = tmp_path_factory.mktemp("runtime")
    (at / "runtime.c").write_text(RUNTIME)
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_build.nvcc()))), "include")
    subprocess.run(["gcc", "-shared", "-fPIC", "-I", include, "-o", str(at / "runtime.so"), str(at / "runtime.c")],
                   check=True)
    root = os.path.dirname(os.path.dirname(os.path.abspath(moe.__file__)))

    def go(call, steps):
        env = dict(os.environ, LD_PRELOAD=str(at / "runtime.so"), PYTHONPATH=root)
        out = subprocess.run([sys.executable, "-c", CALLS, call, json.dumps(steps)], env=env, check=True,
                             capture_output=True, text=True).stdout
        steps = []
        for word in map(str.split, out.splitlines()):
            if word[0] == "call":
                steps.append([None, None, None])
            elif word[0] == "code":
                steps[-1][:2] = int(word[1]), int(word[2])
            elif steps[-1][2] is None:
                steps[-1][2] = (int(word[1]), int(word[2]))
        return steps

    return go


@pytest.mark.parametrize("call", sorted(WANT))
def test_each_device_is_asked_for_its_own_limit(run, call):
    for order in ((0, 1, 0, 1), (1, 0, 1, 0)):  # (each in a process of its own)
        assert run(call, [(d, 0) for d in order]) == [[moe.MOE_OK, 0, WANT[call][d]] for d in order]


@pytest.mark.parametrize("call", sorted(WANT))
def test_an_answer_that_failed_is_not_kept(run, call):
    first, *later = run(call, [(0, 1), (0, 0), (1, 0)])
    # that call is launched with a number that is right on any device, and leaves no error for the next one
    assert first == [moe.MOE_OK, 0, {"sort": (8, 8), "linear": (64, 4), "linear_dx": (64, 4)}.get(call, (152, 1))]
    assert later == [[moe.MOE_OK, 0, WANT[call][d]] for d in (0, 1)]
