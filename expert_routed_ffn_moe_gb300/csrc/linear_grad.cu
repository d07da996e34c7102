// What the gradients of the matrix product with its epilogue start from:
//
//   dpre = dy act'(pre), rounded to bf16 for the products;  dbias = the sum of
//   its rows, before that rounding
//
// The rounding is the products' price: the tensor cores take both operands in bf16, and
// dpre in two parts would double them.  It is off by 2^-8 of a term at most, each term's
// by itself: dx and dweight come to 0.0023 of their size (root mean square) from the
// definition, where their own rounding alone leaves 0.0017.
//
// Bound by memory where there is no activation; its derivative takes as long (two
// special functions and a dozen operations a value, done for two values at once where
// there is an instruction for that).  dy and pre are read once, dpre written once.  A
// cluster of up to 8 CTAs has 64 columns (a row of 128 bytes of bf16), a thread of it one
// of each 32 rows per CTA (with 8 CTAs every 256th row, with one every 32nd); the sums meet
// in shared memory and then in the cluster's first CTA, in a fixed order.
#include "ops_internal.h"
#include "rows_common.cuh"

namespace moe {
namespace {

constexpr int kCols = 64, kThreads = 256, kLanes = kThreads / (kCols / 8);  // 32 rows at a time
constexpr int kMaxRanks = 8;

// act'(g) of two values: with p = logistic(z), z = g or the argument of gelu's tanh form doubled, and q = 1 - p,
//   act' = p + g p q z'(g).
// Beyond g = 10 (gelu) or 88 (silu) q is 0 and act' is p, 1 to 2^-22; below -7.5 or -42 p and act' are 0.
template <int ACT>
MOE_DEV float2 act_grad2(float2 g) {
  constexpr float kGelu = 1.5957691216057308f;
  float2 q;
  const float2 g2 = mul2(g, g), p = logistic2(act_exponent2<ACT>(g, g2), q), a = mul2(g, p);
  if (ACT == MOE_ACT_SILU) return fma2(a, q, p);
  // (beyond |g| = 10 the second term is 0; the bound keeps an overflowing g^2 out)
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

// ------------------------------------------------------------------ few tokens
// For up to 16 tokens the same with the weight's gradient, dweight = dpre^T x, in one
// pass: bound by writing it and, from some eight tokens on, by a multiply-add per token
// and value on the CUDA cores.  A block has 64 rows of it and 256 columns, a warp 8 rows,
// a lane 8 columns of each; dpre is made in shared memory, rounded to bf16 as the other
// product reads it, each value twice, so that a multiply-add of two values finds its pair.
// The blocks of the first columns leave dpre and dbias.  (Tiles of the tensor cores have
// one k block each here and then an epilogue of ~2.4 us: few_grad_tokens() has the times.)
constexpr int kFewRows = 64, kFewCols = 256;

template <typename DY, int ACT>
__global__ void __launch_bounds__(kThreads) linear_few_grad_kernel(LinearGradArgs a, const __nv_bfloat16* x,
                                                                   __nv_bfloat16* dw, int k, int col_tiles) {
  __shared__ __align__(16) float2 d[kFewTokens][kFewRows];  // (each value twice)
  __shared__ float2 exact[kFewTokens][kFewRows / 2];        // before the rounding
  __shared__ uint4 xs[kFewTokens][kFewCols / 8];
  follow();
  const int ct = blockIdx.x % col_tiles, n0 = blockIdx.x / col_tiles * kFewRows;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const __nv_bfloat16* pre = reinterpret_cast<const __nv_bfloat16*>(a.pre);
  const int c = ct * kFewCols + lane * 8, row = n0 + warp * 8;
#pragma unroll
  for (int t = warp; t < kFewTokens; t += kThreads / 32)
    if (t < a.T && c < k) xs[t][lane] = *reinterpret_cast<const uint4*>(x + (size_t)t * k + c);
  for (int i = threadIdx.x; i < a.T * (kFewRows / 2); i += kThreads) {
    const int t = i / (kFewRows / 2), j = i % (kFewRows / 2), n = n0 + 2 * j;
    float2 v = both(0.f);
    if (n < a.n) {
      const size_t at = (size_t)t * a.n + n;
      v = sizeof(DY) == 2 ? bf16_two(*reinterpret_cast<const uint32_t*>(static_cast<const DY*>(a.dy) + at))
                          : *reinterpret_cast<const float2*>(static_cast<const DY*>(a.dy) + at);
      if constexpr (ACT != MOE_ACT_NONE)
        v = mul2(v, act_grad2<ACT>(bf16_two(*reinterpret_cast<const uint32_t*>(pre + at))));
      if (ct == 0 && a.dpre) *reinterpret_cast<uint32_t*>(a.dpre + at) = pack_bf16x2(v.x, v.y);
    }
    exact[t][j] = v;
    const float2 r = bf16_two(pack_bf16x2(v.x, v.y));
    d[t][2 * j] = both(r.x);
    d[t][2 * j + 1] = both(r.y);
  }
  __syncthreads();
  if (ct == 0 && a.dbias && threadIdx.x < kFewRows && n0 + (int)threadIdx.x < a.n) {
    float v = 0.f;  // in the tokens' order, as linear_grad_kernel
    for (int t = 0; t < a.T; ++t) v += reinterpret_cast<const float*>(&exact[t][0])[threadIdx.x];
    if (a.bias_dtype == MOE_BF16)
      put(static_cast<__nv_bfloat16*>(a.dbias) + n0 + threadIdx.x, v);
    else
      put(static_cast<float*>(a.dbias) + n0 + threadIdx.x, v);
  }
  if (c >= k || row >= a.n) return;
  float2 acc[8][4];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[i][e] = both(0.f);
#pragma unroll 2
  for (int t = 0; t < a.T; ++t) {
    const uint4 w = xs[t][lane];
    const float2 xf[4] = {bf16_two(w.x), bf16_two(w.y), bf16_two(w.z), bf16_two(w.w)};
    const float4* dt = reinterpret_cast<const float4*>(&d[t][warp * 8]);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const float4 q = dt[i / 2];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        acc[i][e] = fma2(make_float2(q.x, q.y), xf[e], acc[i][e]);
        acc[i + 1][e] = fma2(make_float2(q.z, q.w), xf[e], acc[i + 1][e]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    *reinterpret_cast<uint4*>(dw + (size_t)(row + i) * k + c) =
        make_uint4(pack_bf16x2(acc[i][0].x, acc[i][0].y), pack_bf16x2(acc[i][1].x, acc[i][1].y),
                   pack_bf16x2(acc[i][2].x, acc[i][2].y), pack_bf16x2(acc[i][3].x, acc[i][3].y));
}
template <typename DY>
cudaError_t few_by_act(const LinearGradArgs& a, const void* x, void* dw, int k, cudaStream_t st) {
  const int col_tiles = (k + kFewCols - 1) / kFewCols, row_tiles = (a.n + kFewRows - 1) / kFewRows;
  if ((long long)col_tiles * row_tiles > 0x7fffffff) return cudaErrorInvalidValue;
  const auto kernel = a.act == MOE_ACT_SILU   ? linear_few_grad_kernel<DY, MOE_ACT_SILU>
                      : a.act == MOE_ACT_GELU ? linear_few_grad_kernel<DY, MOE_ACT_GELU>
                                              : linear_few_grad_kernel<DY, MOE_ACT_NONE>;
  return launch_after(kernel, col_tiles * row_tiles, dim3(kThreads), 0, st, a, static_cast<const __nv_bfloat16*>(x),
                      static_cast<__nv_bfloat16*>(dw), k, col_tiles);
}

}  // namespace

cudaError_t launch_linear_grad(const LinearGradArgs& a, cudaStream_t st) {
  return a.dy_dtype == MOE_BF16 ? by_act<__nv_bfloat16>(a, st) : by_act<float>(a, st);
}

cudaError_t launch_linear_few_grad(const LinearGradArgs& a, const void* x, void* dw, int k, cudaStream_t st) {
  return a.dy_dtype == MOE_BF16 ? few_by_act<__nv_bfloat16>(a, x, dw, k, st) : few_by_act<float>(a, x, dw, k, st);
}

}  // namespace moe
