"""What the norm's calls ask of the CUDA runtime on the host, with a stand-in for
the runtime's functions that they use (no GPU, nothing runs)."""
import collections
import os
import subprocess
import sys

import pytest

import expert_routed_ffn_moe_gb300 as moe

RUNTIME = r"""
#include <stddef.h>
#include <stdio.h>
struct config { unsigned grid[3], block[3]; size_t shared; };
int cudaFuncSetAttribute(const void* f, int what, int v) { printf("set %p %d %d\n", f, what, v); fflush(stdout); return 0; }
int cudaLaunchKernelExC(const struct config* c, const void* f, void** args) {
  (void)args; printf("launch %p %u %zu\n", f, c->block[0], c->shared); fflush(stdout); return 0;
}
int cudaGetDevice(int* d) { *d = 0; return 0; }
int cudaDeviceGetAttribute(int* v, int a, int d) { (void)a; (void)d; *v = 152; return 0; }
int cudaOccupancyMaxActiveBlocksPerMultiprocessor(int* n, const void* f, int b, size_t s) {
  (void)f; (void)b; (void)s; *n = 1; return 0;
}
"""

CALLS = r"""
import ctypes, sys
import expert_routed_ffn_moe_gb300 as moe
L, a, B, F = moe.lib(), ctypes.c_void_p(4096), moe.MOE_BF16, moe.MOE_F32
for T in (1, 300):
    for d in [int(v) for v in sys.argv[1:]]:
        for dt in (B, F):
            print("call forward", d, flush=True)
            assert L.moe_add_norm(a, dt, a, dt, a, B, T, d, 1e-6, a, a, B, None, None) == 0
            print("call backward", d, flush=True)
            assert L.moe_add_norm_backward(a, a, a, a, dt, B, T, d, 1e-6, a, a, a, None) == 0
"""


@pytest.fixture(scope="module")
def record(tmp_path_factory):
    """record(widths): [(call, width, [lines of the runtime])]."""
    moe.build()
    at = tmp_path_factory.mktemp("runtime")
    (at / "runtime.c").write_text(RUNTIME)
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", str(at / "runtime.so"), str(at / "runtime.c")], check=True)
    root = os.path.dirname(os.path.dirname(os.path.abspath(moe.__file__)))

    def run(widths):
        env = dict(os.environ, LD_PRELOAD=str(at / "runtime.so"), PYTHONPATH=root)
        out = subprocess.run([sys.executable, "-c", CALLS] + [str(d) for d in widths], env=env, check=True,
                             capture_output=True, text=True).stdout
        calls = []
        for line in out.splitlines():
            word = line.split()
            if word[0] == "call":
                calls.append((word[1], int(word[2]), []))
            else:
                calls[-1][2].append(word)
        return calls

    return run


def test_a_kernels_shared_memory_does_not_follow_the_last_width(record):
    # One kernel serves many widths, and its limit is the kernel's, not the call's: set to a call's own need, it could be
    # lowered by another thread's call between a wider call's setting and its launch.
    widths = (75, 301, 1999, 4097, 6201, 7001, 8001, 9001, 12301, 16301, 16377, 16383)
    limits, needs, served = collections.defaultdict(set), collections.defaultdict(int), collections.defaultdict(set)
    here = {}
    for what, d, lines in record(widths):
        for word in lines:
            if word[0] == "set":
                limits[word[1]].add(int(word[3]))
                here[word[1]] = int(word[3])
            else:
                smem = int(word[3])
                needs[word[1]] = max(needs[word[1]], smem)
                served[word[1]].add(d)
                assert smem <= here.get(word[1], 48 * 1024), (what, d)
    assert any(len(served[k]) > 1 for k in limits)  # the case in question is among them
    for k, v in limits.items():
        assert len(v) == 1 and needs[k] <= min(v) <= 227 * 1024, (sorted(served[k]), sorted(v), needs[k])
