// What the kernels over rows share: 8 neighbouring columns as a chunk, a row's
// sums over its threads, launches that overlap the kernel before.
#pragma once

#include "ffn_internal.h"

namespace moe {

struct F8 {
  float v[8];
};

// These kernels are launched while the kernel before may still run
// (programmatic stream serialization): their blocks come up during its end, and
// read and write nothing before it has finished.
MOE_DEV void follow() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), int grid, dim3 block, size_t smem, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

// A chunk as it lies in memory.
template <typename T>
struct Raw;
template <>
struct Raw<float> {
  float4 a, b;
  MOE_DEV void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  MOE_DEV void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  MOE_DEV F8 get() const { return F8{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}}; }
};
template <>
struct Raw<__nv_bfloat16> {
  uint4 a;
  MOE_DEV void load(const __nv_bfloat16* p) { a = *reinterpret_cast<const uint4*>(p); }
  MOE_DEV void zero() { a = make_uint4(0u, 0u, 0u, 0u); }
  MOE_DEV F8 get() const {
    return F8{{bf16_lo(a.x), bf16_hi(a.x), bf16_lo(a.y), bf16_hi(a.y), bf16_lo(a.z), bf16_hi(a.z), bf16_lo(a.w),
               bf16_hi(a.w)}};
  }
};
template <typename T>
MOE_DEV F8 load8(const T* p) {
  Raw<T> r;
  r.load(p);
  return r.get();
}
MOE_DEV void store8(float* p, const F8& f) {
  reinterpret_cast<float4*>(p)[0] = make_float4(f.v[0], f.v[1], f.v[2], f.v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(f.v[4], f.v[5], f.v[6], f.v[7]);
}
MOE_DEV void store8(__nv_bfloat16* p, const F8& f) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(f.v[0], f.v[1]), pack_bf16x2(f.v[2], f.v[3]),
                                            pack_bf16x2(f.v[4], f.v[5]), pack_bf16x2(f.v[6], f.v[7]));
}
MOE_DEV float to_f(float v) { return v; }
MOE_DEV float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
MOE_DEV void put(float* p, float v) { *p = v; }
MOE_DEV void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// Two values at once.  (Written out, these are not contracted: a product is rounded before it is added to.)
MOE_DEV uint64_t bits2(float2 a) { return *reinterpret_cast<const uint64_t*>(&a); }
MOE_DEV float2 float2_of(uint64_t a) { return *reinterpret_cast<const float2*>(&a); }
MOE_DEV float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)), "l"(bits2(c)));
  return float2_of(r);
}
MOE_DEV float2 mul2(float2 a, float2 b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
  return float2_of(r);
}
MOE_DEV float2 add2(float2 a, float2 b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
  return float2_of(r);
}
MOE_DEV float2 both(float v) { return make_float2(v, v); }
MOE_DEV float2 bf16_two(uint32_t v) { return make_float2(bf16_lo(v), bf16_hi(v)); }

MOE_DEV float exp2_fast(float v) {  // 2^v
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
MOE_DEV float reciprocal_fast(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
// The activations' common part for two values: e = -z log2(e), where logistic(z) = 1 / (1 + 2^e) is what act(g) multiplies
// g by, z = g or the argument of gelu's tanh form doubled.  g2 = g^2.
template <int ACT>
MOE_DEV float2 act_exponent2(float2 g, float2 g2) {
  constexpr float kLog2e = 1.4426950408889634f, kGelu = 1.5957691216057308f;
  if (ACT == MOE_ACT_SILU) return mul2(g, both(-kLog2e));
  return mul2(g, fma2(g2, both(-kLog2e * kGelu * 0.044715f), both(-kLog2e * kGelu)));
}
// 1 / (1 + 2^e), 0 from 2^-60 down (a huge negative g then gives 0; NaN stays NaN through the product with g): one
// reciprocal for both values, 1 / (a b) times b and a, as the special functions are what a tile's epilogue takes longest for.
// A value's last places thus follow its neighbour, and where 2^e vanishes the result is 1 to 2^-22, not exactly: one minus
// it is `rest`, 2^e / (1 + 2^e), which is 0 there, and never a difference (a gradient multiplies it by g).
// (The form for one value, logistic(), which few tokens' kernels use, ends at e^-80: act(g) for silu below -42 or gelu
// below -7.5, at most 4e-17 in size, is 0 or not by the number of tokens.)
MOE_DEV float2 logistic2(float2 e, float2& rest) {
  constexpr float kFar = 60.f;
  const float2 t = make_float2(exp2_fast(fminf(e.x, kFar)), exp2_fast(fminf(e.y, kFar))), d = add2(t, both(1.f));
  const float r = reciprocal_fast(d.x * d.y);
  float2 p = mul2(make_float2(d.y, d.x), both(r));
  rest = mul2(t, p);
  p.x = e.x > kFar ? 0.f : p.x;
  p.y = e.y > kFar ? 0.f : p.y;
  return p;
}
MOE_DEV float2 logistic2(float2 e) {
  float2 rest;
  return logistic2(e, rest);
}
template <int ACT>
MOE_DEV float2 act_value2(float2 g) {
  if (ACT == MOE_ACT_NONE) return g;
  return mul2(g, logistic2(act_exponent2<ACT>(g, mul2(g, g))));
}

// The sums over the R threads of a row, in every one of them.  `red` is another
// half of its memory from one row to the next, so one barrier per row suffices.
template <int R, int N>
MOE_DEV void row_sums(float (&v)[N], float (*red)[N][32]) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
  if (R == 32) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) (*red)[i][warp] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum(lane < R / 32 ? (*red)[i][lane] : 0.f);
}

// Asynchronous copies of 16 bytes, or of their first `bytes`: the rest becomes 0.  Those of fp32 go through L1: a layer
// norm's window of 8 is two copies of half its sectors each, of which the second finds the first's there (d = 4096, backward:
// 179 us for 260 through L2 alone); others pass L1 by (a window of bf16: 94 us for 98).
template <typename T>
MOE_DEV void copy16(uint32_t to, const T* from, int bytes) {
  if (sizeof(T) == 4)
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
  else
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
}
MOE_DEV void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
MOE_DEV void copies_wait() {  // all but the last N groups of this thread
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Blocks that walk the rows: as many as are resident on the device's SMs (one on each where the device does not say).
template <typename K>
cudaError_t ask_resident(K kernel, int block, size_t smem, int* n) {
  int dev = 0, sms = 8, per = 0;  // (a multiple of 8: every walk takes it)
  cudaError_t err = cudaGetDevice(&dev);
  if (err == cudaSuccess) err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (err == cudaSuccess) err = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, block, smem);
  *n = sms * (err == cudaSuccess && per > 0 ? per : 1);
  return err;
}
template <typename K>
int resident_blocks(K kernel, int block, size_t smem) {
  int n = 0;
  if (ask_resident(kernel, block, smem, &n) != cudaSuccess) cudaGetLastError();
  return n;
}
// The same, asked once for each device; `known` is one for each kernel, block and smem.
template <typename K>
int resident_blocks(K kernel, int block, size_t smem, ByDevice& known) {
  return once_per_device(known, [&](int* n) { return ask_resident(kernel, block, smem, n); });
}

// Sets a kernel's limit on shared memory once for each device (`done`: the devices that have it).
template <typename K>
cudaError_t allow_once(K kernel, size_t bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  const uint64_t bit = 1ull << (dev & 63);
  if (dev < 64 && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
  err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (err == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return err;
}
// A kernel's limit on shared memory belongs to all its launches, which threads of the host may issue side by side: it
// is set for the widest rows, never lower for narrower ones.
template <typename K>
cudaError_t allow(K kernel, size_t smem, size_t most) {
  return smem <= 48 * 1024
             ? cudaSuccess
             : cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
}

}  // namespace moe
