// What the gradients of the matrix product with its epilogue start from:
//
//   dpre = dy act'(pre), rounded to bf16 for the products;  dbias = the sum of
//   its rows, before that rounding
//
// Bound by memory: dy and pre are read once, dpre written once.  A cluster of up
// to 8 CTAs has 64 columns (a row of 128 bytes of bf16), its CTAs' threads every
// 256th row; the sums meet in shared memory and then in the cluster's first CTA,
// in a fixed order.
#include "ops_internal.h"
#include "rows_common.cuh"

namespace moe {
namespace {

constexpr int kCols = 64, kThreads = 256, kLanes = kThreads / (kCols / 8);  // 32 rows at a time
constexpr int kMaxRanks = 8;

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
  float sum[8] = {};
  if (c < a.n) {
    constexpr int kAhead = 4;
    const long long step = (long long)ranks * kLanes;
    for (long long r0 = rank * kLanes + lane; r0 < a.T; r0 += step * kAhead) {
      Raw<DY> g[kAhead];
      Raw<__nv_bfloat16> p[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const long long r = r0 + u * step;
        if (r < a.T) {
          g[u].load(dy + r * a.n + c);
          if (ACT != MOE_ACT_NONE) p[u].load(pre + r * a.n + c);
        }
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const long long r = r0 + u * step;
        if (r < a.T) {
          F8 v = g[u].get();
          if constexpr (ACT != MOE_ACT_NONE) {
            const F8 z = p[u].get();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              float f, df;
              act_and_grad<ACT>(z.v[i], f, df);
              v.v[i] = __fmul_rn(v.v[i], df);  // (not contracted into the sum in a branch without dpre: one value in both)
            }
          }
          if (dpre) store8(dpre + r * a.n + c, v);
#pragma unroll
          for (int i = 0; i < 8; ++i) sum[i] += v.v[i];
        }
      }
    }
  }
  if (!a.dbias) return;  // (in all CTAs alike)
#pragma unroll
  for (int i = 0; i < 8; ++i) part[lane][at * 8 + i] = sum[i];
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
  int ranks = 1;
  while (ranks < kMaxRanks && ranks * kLanes < a.T) ranks *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((a.n + kCols - 1) / kCols * ranks);
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
