// Internal declarations of the dense gated feed-forward block and the norm in
// front of it: shapes, the context's workspace and the kernel launchers.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "moe.h"
#include "moe_common.cuh"

namespace moe {

// ---------------------------------------------------------------- mx8
// Scale bytes of a [rows, cols] mx8 matrix: tiles of 128 rows x 4 groups of 32
// columns, 512 bytes each, in the order in which tcgen05.cp moves them into
// tensor memory (row r of the tile at byte (r % 32) * 16 + (r / 32) * 4).
__host__ __device__ inline size_t mx_tile_cols(size_t cols) { return (cols + 127) / 128; }
__host__ __device__ inline size_t mx_scale_bytes(size_t rows, size_t cols) {
  return (rows + 127) / 128 * mx_tile_cols(cols) * 512;
}
// Byte of the first of the four groups 4 w .. 4 w + 3 of row r.
__host__ __device__ inline size_t mx_scale_word(size_t r, size_t w, size_t tile_cols) {
  return (r / 128 * tile_cols + w) * 512 + r % 32 * 16 + r / 32 % 4 * 4;
}

// The scale byte of a group whose largest magnitude is amax: e + 127 with e the
// least integer >= -127 such that amax <= 448 * 2^e.  amax = 1.m * 2^p: e is
// p - 8 where 1.m <= 1.75 (448 = 1.75 * 2^8), else p - 7.  Infinity and NaN give
// 255, the scale that is not a number.
MOE_DEV uint32_t mx_scale_byte(float amax) {
  const uint32_t b = __float_as_uint(amax) & 0x7fffffffu;
  if (b >= 0x7f800000u) return 255u;
  const int e = (int)(b >> 23) - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  return (uint32_t)max(e, 0);
}
// 2^-e, what the values are multiplied by before they are rounded to e4m3.
// Exact for every byte 0..247 that a finite amax can have (2^127 .. 2^-120); byte 255 gives NaN.
MOE_DEV float mx_inverse_scale(uint32_t byte) {
  return byte == 255u ? __uint_as_float(0x7fffffffu) : __uint_as_float((254u - byte) << 23);
}
MOE_DEV float mx_scale(uint32_t byte) {  // 2^e; 2^-127 is subnormal
  return byte == 255u ? __uint_as_float(0x7fffffffu) : (byte ? __uint_as_float(byte << 23) : __uint_as_float(0x400000u));
}
// |v| for a running maximum that keeps NaN (fmaxf drops it): as an integer the
// magnitude bits of a NaN lie above those of infinity.
MOE_DEV uint32_t mag_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// Two values to e4m3, to the nearest even (the scales keep them within 448).
MOE_DEV uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
MOE_DEV uint32_t e4m3x4(float a, float b, float c, float d) { return e4m3x2(a, b) | (e4m3x2(c, d) << 16); }

// Instruction descriptor of the block-scaled form: e4m3 A and B (K-major), e8m0
// scales, byte `id` of each row's four.
__host__ __device__ constexpr uint32_t umma_idesc_mx(int M, int N, int id) {
  return (static_cast<uint32_t>(id) << 4)          // scale byte of B
         | (static_cast<uint32_t>(N >> 3) << 17)   // N / 8
         | (1u << 23)                              // e8m0 scales
         | (static_cast<uint32_t>(M >> 4) << 24)   // M / 16
         | (static_cast<uint32_t>(id) << 29);      // scale byte of A
}
// Descriptor of 512 bytes of scales in shared memory, the source of tcgen05.cp:
// no swizzle, 8-row groups of 128 bytes.
MOE_DEV uint64_t mx_scale_desc(uint32_t saddr) {
  return static_cast<uint64_t>((saddr & 0x3ffffu) >> 4) | (static_cast<uint64_t>(128 >> 4) << 32) |
         (static_cast<uint64_t>(1) << 46);
}
// Shared-memory matrix descriptor of an MN-major bf16 operand, 128-byte swizzle:
// each of 64 k is a 128-byte row of 64 elements along m (or n), 8 k rows make a
// 1024-byte atom; the next 64 elements along m lie 64 k rows further.
MOE_DEV uint64_t desc_mn(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3ffffu) >> 4);
  d |= static_cast<uint64_t>((64 * 128) >> 4) << 16;  // leading: from 64 elements of m to the next 64
  d |= static_cast<uint64_t>(1024 >> 4) << 32;        // stride: from 8 k rows to the next 8
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}
// 16 consecutive fp32 columns of this thread's TMEM lane, valid after tmem_ld_wait().
MOE_DEV void tmem_ld16_async(uint32_t taddr, float* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
        "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
      : "r"(taddr)
      : "memory");
}

// ---------------------------------------------------------------- clusters
MOE_DEV uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
MOE_DEV void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Address of `p` (this CTA's shared memory) in the cluster's CTA `rank`.
MOE_DEV uint32_t map_cta(const void* p, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
MOE_DEV void arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// For waits that end by themselves, on what the CTA itself has in flight before
// it leaves: 1 s, however short the caller's limit.
MOE_DEV DevCtl drain_ctl(const DevCtl& c) {
  DevCtl d = c;
  d.spin_limit = 1000000000LL;
  return d;
}

// ---------------------------------------------------------------- activations
// silu(g) = g sigmoid(g); gelu in its tanh form, 0.5 g (1 + tanh z) =
// g sigmoid(2 z): both from the fast exponential and division of sigmoid
// (~2^-21 relative).
// The logistic function, 0 below e^-80 (so that a huge negative g gives 0 and
// not g e^-80; NaN stays NaN through the product with g).  Computed first and
// selected after: as a branch every value would wait out the exponential's and
// the division's latency alone.
MOE_DEV float logistic(float z) {
  const float p = sigmoid(z);
  return z < -80.0f ? 0.0f : p;
}
// act(g), and the second form with its derivative.  ACT is a constant so that
// the loops over values have no branch; with_act() picks it once per loop.
template <int ACT>
MOE_DEV float act_value(float g) {
  if (ACT == MOE_ACT_SILU) return g * logistic(g);
  return g * logistic(1.5957691216057308f * (g + 0.044715f * g * g * g));
}
template <int ACT>
MOE_DEV void act_and_grad(float g, float& a, float& da) {
  if (ACT == MOE_ACT_SILU) {
    const float p = logistic(g);
    a = g * p;
    da = p + a * (1.0f - p);
  } else {
    const float g2 = g * g;
    const float p = logistic(1.5957691216057308f * (g + 0.044715f * g * g2));
    a = g * p;
    // beyond |g| = 10 p is 0 or 1 to fp32 and the second term vanishes; the bound keeps an overflowing g^2 out
    da = p + a * (1.0f - p) * (1.5957691216057308f * (1.0f + 0.134145f * fminf(g2, 100.0f)));
  }
}
template <int ACT>
struct ActTag {
  static constexpr int value = ACT;
};
template <typename F>
MOE_DEV void with_act(int act, F&& f) {
  if (act == MOE_ACT_SILU)
    f(ActTag<MOE_ACT_SILU>());
  else
    f(ActTag<MOE_ACT_GELU>());
}

struct FfnShape {
  int T, d, I, act;
};

// ffn_norm.cu
constexpr int kMaxNormWidth = 16384;
constexpr int kNormPartials = 1216;  // rows of partial weight gradients (8 for each of 152 SMs)
struct NormArgs {
  const void *x, *res, *w;
  void *s, *y;
  uint8_t* scales;
  int T, d;
  int x_dtype, s_dtype, w_dtype, y_dtype;
  float eps;
};
cudaError_t launch_norm(const NormArgs& a, cudaStream_t st);
struct NormGradArgs {
  const void *s, *w, *dy, *ds;
  void *dx, *dw;
  float* partial;  // [kNormPartials, d]
  int T, d;
  int dtype, w_dtype;
  float eps;
};
cudaError_t launch_norm_backward(const NormGradArgs& a, cudaStream_t st);
cudaError_t launch_mx_quantize(const void* v, int dtype, int rows, int cols, uint8_t* codes, uint8_t* scales,
                               cudaStream_t st);

// Operands and outputs of one call on device memory (NULL where absent).
struct FfnForwardArgs {
  const void *x, *gate_up, *down;
  const uint8_t *xs, *gate_up_s, *down_s;  // mx8 scales
  void* y;
  void* pre;
};
struct FfnBackwardArgs {
  const uint16_t *x, *pre, *gate_up, *down, *dy;
  uint16_t *dx, *dgate_up, *ddown;
};
struct FfnScratch {
  uint16_t* h;       // [max_tokens, I] bf16 act(gate) * up
  uint8_t* hq;       // the same as mx8 codes
  uint8_t* hs;       // and scales
  uint8_t* up_s;     // [I, d] scales of the up weights, where launch_mx_up_scales is needed
  uint16_t* dpre;    // [max_tokens, 2 I] bf16 gradients of the pre-activations (training)
  unsigned* status;  // device status word
};

// Signature of the driver's cuTensorMapEncodeTiled (fetched at run time, so the
// library needs no link-time dependency on libcuda).
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
// A 2-D bf16 map: `inner` contiguous elements per row, rows `pitch` elements apart.
inline bool make_bf16_map(EncodeTiledFn encode, CUtensorMap* m, const void* ptr, uint64_t inner, uint64_t outer,
                          uint64_t pitch, uint32_t box_inner, uint32_t box_outer) {
  const cuuint64_t dims[2] = {inner, outer};
  const cuuint64_t strides[1] = {pitch * 2};
  const cuuint32_t box[2] = {box_inner, box_outer};
  const cuuint32_t estr[2] = {1, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(ptr), dims, strides, box, estr,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// mx8 codes [rows, K]; and scale tiles as [row tile][column tile][64 x 8 bytes].
inline bool make_code_map(EncodeTiledFn encode, CUtensorMap* m, const void* ptr, uint64_t K, uint64_t rows,
                          uint32_t box_rows) {
  const cuuint64_t dims[2] = {K, rows};
  const cuuint64_t strides[1] = {K};
  const cuuint32_t box[2] = {128, box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(ptr), dims, strides, box, estr,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
inline bool make_scale_map(EncodeTiledFn encode, CUtensorMap* m, const void* ptr, uint64_t cols, uint64_t row_tiles) {
  const uint64_t tile_cols = mx_tile_cols(cols);
  const cuuint64_t dims[3] = {64, tile_cols, row_tiles};
  const cuuint64_t strides[2] = {512, 512 * tile_cols};
  const cuuint32_t box[3] = {64, 1, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT64, 3, const_cast<void*>(ptr), dims, strides, box, estr,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct FfnEngine {
  EncodeTiledFn encode;
  int sms;
  int pairs, pairs2, pairs4;  // clusters of 1, 2 and 4 CTA pairs that run at a time
  DevCtl ctl;
};

// ffn_gemm.cu
cudaError_t prepare_ffn_gemm(FfnEngine* e);  // kernel attributes; fills in e->pairs*
cudaError_t launch_ffn_gate_up(const FfnEngine& e, const FfnShape& s, const void* x, const void* gate_up, uint16_t* h,
                               uint16_t* pre, cudaStream_t st);
cudaError_t launch_ffn_down(const FfnEngine& e, const FfnShape& s, const uint16_t* h, const void* down, void* y,
                            cudaStream_t st);
cudaError_t launch_ffn_grad_h(const FfnEngine& e, const FfnShape& s, const FfnBackwardArgs& a, const FfnScratch& sc,
                              cudaStream_t st);
// dx, dgate_up and ddown, as far as wanted, from what launch_ffn_grad_h left; *launches: kernels launched
cudaError_t launch_ffn_grads(const FfnEngine& e, const FfnShape& s, const FfnBackwardArgs& a, const FfnScratch& sc,
                             int* launches, cudaStream_t st);

// mx8.  up_s: the scales of gate_up's rows I .. 2I - 1 as a matrix of their own:
// where I is a multiple of 128 they are one inside gate_up_s, else
// launch_mx_up_scales lays them out.
cudaError_t launch_mx_up_scales(const FfnShape& s, const uint8_t* gate_up_s, uint8_t* up_s, cudaStream_t st);
cudaError_t launch_ffn_gate_up_mx(const FfnEngine& e, const FfnShape& s, const FfnForwardArgs& a, const uint8_t* up_s,
                                  uint8_t* hq, uint8_t* hs, cudaStream_t st);
cudaError_t launch_ffn_down_mx(const FfnEngine& e, const FfnShape& s, const uint8_t* hq, const uint8_t* hs,
                               const FfnForwardArgs& a, cudaStream_t st);

// ffn_skinny.cu: for few tokens the whole forward call, and of the backward call
// what reads the weights: grad_h and, where it is wanted, dx
//
// Up to 32 tokens always; up to 64 where reading the weights is most of the time:
// with 64 tokens the parts' exchange grows and waits for the ring's memory.
// Forward call at T = 33 and 64, as a stream against as tiles (us): d = 4096, I =
// 16384: 84, 87 against 95, 95 (mx8: 52, 56 against 67, 67); d = 4096, I = 4096:
// 30, 32 against 34, 34; d = 2048, I = 2048: 24, 27 against 21, 21.  One rule serves
// both directions: the smallest weights would gain 1 to 3 us forward (d = 2048, I =
// 512: 14, 16 against 17, 17) but not backward (20, 22 against 20, 20).
constexpr int kSkinnyTokens = 64;
inline bool few_tokens(const FfnShape& s) {
  return s.T <= 32 || (s.T <= kSkinnyTokens && 3LL * s.d * s.I >= 1LL << 25);
}
cudaError_t prepare_ffn_skinny();
cudaError_t launch_skinny_forward(const FfnEngine& e, const FfnShape& s, bool mx, const FfnForwardArgs& a,
                                  const uint8_t* up_s, const FfnScratch& sc, cudaStream_t st);
cudaError_t launch_skinny_backward(const FfnEngine& e, const FfnShape& s, const FfnBackwardArgs& a,
                                   const FfnScratch& sc, cudaStream_t st);

}  // namespace moe
