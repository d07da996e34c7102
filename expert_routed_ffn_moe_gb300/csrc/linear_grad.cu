// What the gradients of the matrix product with its epilogue start from:
//
//   dpre = dy act'(pre), rounded to bf16 for the products;  dbias = the sum of
//   its rows, before that rounding
//
// Bound by memory where there is no activation; its derivative takes as long (two
// special functions and a dozen operations a value, done for two values at once where
// there is an instruction for that).  dy and pre are read once, dpre written once.  A
// cluster of up to 8 CTAs has 64 columns (a row of 128 bytes of bf16), its CTAs' threads every
// 256th row; the sums meet in shared memory and then in the cluster's first CTA,
// in a fixed order.
#include "ops_internal.h"
#include "rows_common.cuh"

namespace moe {
namespace {

constexpr int kCols = 64, kThreads = 256, kLanes = kThreads / (kCols / 8);  // 32 rows at a time
constexpr int kMaxRanks = 8;

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
// act'(g) of two values, as act_and_grad(): with p = logistic(z), z = g or the argument of gelu's tanh form doubled,
//   act' = p + g p (1 - p) z'(g).
template <int ACT>
MOE_DEV float2 act_grad2(float2 g) {
  constexpr float kLog2e = 1.4426950408889634f, kGelu = 1.5957691216057308f, kFar = 80.f * kLog2e;
  const float2 g2 = mul2(g, g);
  // e = -z log2(e)
  const float2 e = ACT == MOE_ACT_SILU
                       ? mul2(g, both(-kLog2e))
                       : mul2(g, fma2(g2, both(-kLog2e * kGelu * 0.044715f), both(-kLog2e * kGelu)));
  const float2 d = add2(make_float2(exp2_fast(fminf(e.x, kFar)), exp2_fast(fminf(e.y, kFar))), both(1.f));
  float2 p = make_float2(reciprocal_fast(d.x), reciprocal_fast(d.y));
  p.x = e.x > kFar ? 0.f : p.x;  // (a huge negative g gives 0 and not g e^-80)
  p.y = e.y > kFar ? 0.f : p.y;
  const float2 a = mul2(g, p), q = fma2(p, both(-1.f), both(1.f));
  if (ACT == MOE_ACT_SILU) return fma2(a, q, p);
  // (beyond |g| = 10 the second term vanishes; the bound keeps an overflowing g^2 out)
  const float2 dz = fma2(make_float2(fminf(g2.x, 100.f), fminf(g2.y, 100.f)), both(kGelu * 0.134145f), both(kGelu));
  return fma2(mul2(a, q), dz, p);
}

template <typename DY, int ACT>
__global__ void __launch_bounds__(kThreads) linear_grad_kernel(LinearGradArgs a, int ranks) {
  __shared__ float part[kLanes][kCols + 1];
  __shared__ float mine[kCols];
  follow();
  const int rank = (int)cluster_rank(), tile = blockIdx.x / ranks;
  const int at = threadIdx.x % (kCols / 8), lane = threadIdx.x / (kCols / 8);
  const int c = tile * kCols + at * 8;
  const DY* dy = static_cast<const DY*>(a.dy);
  const __nv_bfloat16* pre = reinterpret_cast<const __nv_bfloat16*>(a.pre);
  __nv_bfloat16* dpre = reinterpret_cast<__nv_bfloat16*>(a.dpre);
  float2 sum[4] = {};
  if (c < a.n) {
    constexpr int kRows = ACT == MOE_ACT_NONE ? 4 : 2;  // at a time; the next ones are asked for before they are used
    const long long step = (long long)ranks * kLanes;
    Raw<DY> g[kRows], g_next[kRows];
    Raw<__nv_bfloat16> p[kRows], p_next[kRows];
    auto load = [&](long long r0) {
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        const long long r = r0 + u * step;
        if (r < a.T) {
          g_next[u].load(dy + r * a.n + c);
          if (ACT != MOE_ACT_NONE) p_next[u].load(pre + r * a.n + c);
        }
      }
    };
    load(rank * kLanes + lane);
    for (long long r0 = rank * kLanes + lane; r0 < a.T; r0 += step * kRows) {
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        g[u] = g_next[u];
        p[u] = p_next[u];
      }
      load(r0 + step * kRows);
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        const long long r = r0 + u * step;
        if (r < a.T) {
          F8 v = g[u].get();
          if constexpr (ACT != MOE_ACT_NONE) {
            const uint4 z = p[u].a;
            const uint32_t zw[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 t = mul2(make_float2(v.v[2 * i], v.v[2 * i + 1]), act_grad2<ACT>(bf16_two(zw[i])));
              v.v[2 * i] = t.x, v.v[2 * i + 1] = t.y;
            }
          }
          if (dpre) store8(dpre + r * a.n + c, v);
#pragma unroll
          for (int i = 0; i < 4; ++i) sum[i] = add2(sum[i], make_float2(v.v[2 * i], v.v[2 * i + 1]));
        }
      }
    }
  }
  if (!a.dbias) return;  // (in all CTAs alike)
#pragma unroll
  for (int i = 0; i < 4; ++i) part[lane][at * 8 + 2 * i] = sum[i].x, part[lane][at * 8 + 2 * i + 1] = sum[i].y;
  __syncthreads();
  if (threadIdx.x < kCols) {
    float v = 0.f;
#pragma unroll 8
    for (int l = 0; l < kLanes; ++l) v += part[l][threadIdx.x];
    mine[threadIdx.x] = v;
  }
  cluster_sync();
  const int k = tile * kCols + threadIdx.x;
  if (rank == 0 && threadIdx.x < kCols && k < a.n) {
    float v = 0.f;
    for (int r = 0; r < ranks; ++r) {
      float x;
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(map_cta(mine + threadIdx.x, r)));
      v += x;
    }
    if (a.bias_dtype == MOE_BF16)
      put(static_cast<__nv_bfloat16*>(a.dbias) + k, v);
    else
      put(static_cast<float*>(a.dbias) + k, v);
  }
  cluster_sync();  // no CTA leaves while the first reads its sums
}

template <typename DY, int ACT>
cudaError_t launch(const LinearGradArgs& a, cudaStream_t st) {
  // as many as give 4 blocks for each of 152 SMs, and each thread a row
  const int tiles = (a.n + kCols - 1) / kCols;
  int ranks = 1;
  while (ranks < kMaxRanks && ranks * kLanes < a.T && ranks * tiles < 4 * 152) ranks *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(tiles * ranks);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = ranks;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, linear_grad_kernel<DY, ACT>, a, ranks);
}
template <typename DY>
cudaError_t by_act(const LinearGradArgs& a, cudaStream_t st) {
  return a.act == MOE_ACT_SILU   ? launch<DY, MOE_ACT_SILU>(a, st)
         : a.act == MOE_ACT_GELU ? launch<DY, MOE_ACT_GELU>(a, st)
                                 : launch<DY, MOE_ACT_NONE>(a, st);
}

}  // namespace

cudaError_t launch_linear_grad(const LinearGradArgs& a, cudaStream_t st) {
  return a.dy_dtype == MOE_BF16 ? by_act<__nv_bfloat16>(a, st) : by_act<float>(a, st);
}

}  // namespace moe
