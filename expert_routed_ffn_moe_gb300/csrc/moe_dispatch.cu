// Tokens sorted by expert and back.
//
//   sort       counts, offsets, perm and slot from idx [T, k]: the picks in the
//              order (expert, token, pick); a pick whose expert id is not one of
//              0 .. E - 1 is dropped (slot -1)
//   dispatch   rows[slot[t, j]] = x[t]
//   combine    y[t] = sum_j w[t, j] rows[slot[t, j]] + add[t]; without weights the
//              gradient of dispatch
//   backward   of combine: rows'[slot[t, j]] = w[t, j] dy[t], dw[t, j] = dy[t] .
//              rows[slot[t, j]]
//
// All but the sort are bound by memory.  Each works from the tokens' side: a token's
// row is read or written once, its k sorted rows once each, and a sum over the picks
// runs in their order, with no atomics.  A slot outside 0 .. n_rows - 1 is taken as
// dropped, so no access leaves the rows.
#include "ops_internal.h"
#include "rows_common.cuh"

namespace moe {
namespace {

// ------------------------------------------------------------------ sort
// One cluster of up to 8 CTAs of 32 warps.  A warp owns a contiguous range of the
// picks.  It counts its picks per expert (one warp-wide match per 32 picks; equal
// experts' first lane adds their number), the counts become start positions by a
// prefix over the warps, the CTAs (distributed shared memory) and the experts, and a
// second walk over the picks hands them out in order.
constexpr int kSortThreads = 1024, kSortWarps = 32, kSortCluster = 8;
constexpr int kSortAhead = 4;  // loads of 32 picks in flight per warp

__global__ void __launch_bounds__(kSortThreads, 1) sort_tokens_kernel(SortArgs a) {
  extern __shared__ int sort_sm[];
  int* hist = sort_sm;                     // [32][E]: counts, then next positions
  int* total = sort_sm + kSortWarps * a.E; // [E] of this CTA, read by the others
  __shared__ int warp_part[kSortWarps];
  follow();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)cluster_rank(), ranks = gridDim.x;
  // picks per warp, a multiple of 32
  const long long per = (((long long)a.picks + (long long)ranks * kSortThreads - 1) / ((long long)ranks * kSortThreads)) * 32;
  const long long first = ((long long)rank * kSortWarps + warp) * per;
  const int lo = (int)min(first, (long long)a.picks), hi = (int)min(first + per, (long long)a.picks);
  int* mine = hist + warp * a.E;
  for (int e = lane; e < a.E; e += 32) mine[e] = 0;
  __syncwarp();

  auto walk = [&](auto&& each) {
    for (int p0 = lo; p0 < hi; p0 += 32 * kSortAhead) {
      int e[kSortAhead];
#pragma unroll
      for (int u = 0; u < kSortAhead; ++u) {
        const int p = p0 + u * 32 + lane;
        e[u] = p < hi ? a.idx[p] : -1;
      }
#pragma unroll
      for (int u = 0; u < kSortAhead; ++u) {
        if (p0 + u * 32 >= hi) break;
        const bool in = e[u] >= 0 && e[u] < a.E;
        const unsigned same = __match_any_sync(0xffffffffu, in ? e[u] : -1);
        each(p0 + u * 32 + lane, e[u], in, same);
        __syncwarp();
      }
    }
  };
  walk([&](int, int e, bool in, unsigned same) {
    if (in && lane == __ffs(same) - 1) mine[e] += __popc(same);
  });
  __syncthreads();
  // prefix over the warps
  for (int e = tid; e < a.E; e += kSortThreads) {
    int sum = 0;
#pragma unroll 8
    for (int w = 0; w < kSortWarps; ++w) {
      const int c = hist[w * a.E + e];
      hist[w * a.E + e] = sum;
      sum += c;
    }
    total[e] = sum;
  }
  cluster_sync();
  // prefix over the CTAs, then over the experts: E <= 1024, one per thread
  int before = 0, all = 0;
  if (tid < a.E) {
    for (int r = 0; r < ranks; ++r) {
      int c;
      asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(c) : "r"(map_cta(total + tid, r)));
      if (r < rank) before += c;
      all += c;
    }
  }
  int scan = all;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, scan, o);
    if (lane >= o) scan += v;
  }
  if (lane == 31) warp_part[warp] = scan;
  __syncthreads();
  int below = lane < warp ? warp_part[lane] : 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) below += __shfl_xor_sync(0xffffffffu, below, o);
  const int offset = below + scan - all;  // of expert tid
  if (rank == 0 && tid < a.E) {
    if (a.counts) a.counts[tid] = all;
    if (a.offsets) {
      a.offsets[tid] = offset;
      if (tid == a.E - 1) a.offsets[a.E] = offset + all;
    }
  }
  if (tid < a.E)
    for (int w = 0; w < kSortWarps; ++w) hist[w * a.E + tid] += offset + before;
  __syncthreads();
  walk([&](int p, int e, bool in, unsigned same) {
    int at = -1;
    if (in) at = mine[e] + __popc(same & ((1u << lane) - 1u));
    __syncwarp();
    if (in && lane == __ffs(same) - 1) mine[e] += __popc(same);
    if (p < hi) {
      if (a.slot) a.slot[p] = at;
      if (a.perm && in) a.perm[at] = p / a.k;
    }
  });
  cluster_sync();  // no CTA leaves while another reads its totals
}

// ------------------------------------------------------------------ rows
// A warp has 32 chunks of neighbouring columns at a time: of 8 columns where rows
// are aligned, else of one.
template <typename T, int VEC>
struct Piece;
template <typename T>
struct Piece<T, 1> {
  T v;
  MOE_DEV void load(const T* p) { v = *p; }
  MOE_DEV void get(float (&f)[1]) const { f[0] = to_f(v); }
  static MOE_DEV void store(T* p, const float (&f)[1]) { put(p, f[0]); }
};
template <typename T>
struct Piece<T, 8> {
  Raw<T> r;
  MOE_DEV void load(const T* p) { r.load(p); }
  MOE_DEV void get(float (&f)[8]) const {
    const F8 t = r.get();
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = t.v[i];
  }
  static MOE_DEV void store(T* p, const float (&f)[8]) {
    store8(p, F8{{f[0], f[1], f[2], f[3], f[4], f[5], f[6], f[7]}});
  }
};

constexpr int kRowThreads = 256;
constexpr int kPieces = 2;  // chunks per lane and slice
template <int VEC>
constexpr int kSlice = 32 * VEC * (VEC == 8 ? kPieces : 4 * kPieces);  // columns per slice

// The slot of lane j's pick, -1 where there is none.
MOE_DEV int slot_of(const RowsArgs& a, int t, int j) {
  const int s = j < a.k ? a.slot[(size_t)t * a.k + j] : -1;
  return s < 0 || s >= a.n_rows ? -1 : s;
}

template <typename XT, typename RT, int VEC>
__global__ void __launch_bounds__(kRowThreads) dispatch_kernel(RowsArgs a) {
  constexpr int P = kSlice<VEC> / (32 * VEC);
  follow();
  const int lane = threadIdx.x & 31;
  const int slices = (a.d + kSlice<VEC> - 1) / kSlice<VEC>;
  const long long unit = (long long)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);
  if (unit >= (long long)a.T * slices) return;
  const int t = (int)(unit / slices), c0 = (int)(unit - (long long)t * slices) * kSlice<VEC> + lane * VEC;
  const XT* x = static_cast<const XT*>(a.tokens) + (size_t)t * a.d;
  const int slot = slot_of(a, t, lane);
  Piece<XT, VEC> in[P];
#pragma unroll
  for (int i = 0; i < P; ++i)
    if (c0 + i * 32 * VEC < a.d) in[i].load(x + c0 + i * 32 * VEC);
  for (int j = 0; j < a.k; ++j) {
    const int s = __shfl_sync(0xffffffffu, slot, j);
    if (s < 0) continue;
    RT* to = static_cast<RT*>(a.out) + (size_t)s * a.d;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int c = c0 + i * 32 * VEC;
      if (c < a.d) {
        float f[VEC];
        in[i].get(f);
        Piece<RT, VEC>::store(to + c, f);
      }
    }
  }
}

template <typename RT, typename YT, int VEC>
__global__ void __launch_bounds__(kRowThreads) combine_rows_kernel(RowsArgs a) {
  constexpr int P = kSlice<VEC> / (32 * VEC), kAhead = VEC == 8 ? 8 / kPieces : 2;  // rows in flight
  follow();
  const int lane = threadIdx.x & 31;
  const int slices = (a.d + kSlice<VEC> - 1) / kSlice<VEC>;
  const long long unit = (long long)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);
  if (unit >= (long long)a.T * slices) return;
  const int t = (int)(unit / slices), c0 = (int)(unit - (long long)t * slices) * kSlice<VEC> + lane * VEC;
  const RT* rows = static_cast<const RT*>(a.rows_in);
  const YT* add = static_cast<const YT*>(a.tokens);
  const int slot = slot_of(a, t, lane);
  const float w = a.w && lane < a.k ? a.w[(size_t)t * a.k + lane] : 1.f;
  Piece<YT, VEC> last[P];
  if (add) {
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (c0 + i * 32 * VEC < a.d) last[i].load(add + (size_t)t * a.d + c0 + i * 32 * VEC);
  }
  float acc[P][VEC];
#pragma unroll
  for (int i = 0; i < P; ++i)
#pragma unroll
    for (int v = 0; v < VEC; ++v) acc[i][v] = 0.f;
  for (int j0 = 0; j0 < a.k; j0 += kAhead) {
    Piece<RT, VEC> in[kAhead][P];
    int s[kAhead];
    float wj[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      s[u] = __shfl_sync(0xffffffffu, slot, min(j0 + u, 31));
      wj[u] = __shfl_sync(0xffffffffu, w, min(j0 + u, 31));
      if (j0 + u >= a.k) s[u] = -1;
#pragma unroll
      for (int i = 0; i < P; ++i)
        if (s[u] >= 0 && c0 + i * 32 * VEC < a.d) in[u][i].load(rows + (size_t)s[u] * a.d + c0 + i * 32 * VEC);
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (s[u] >= 0) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
          float f[VEC];
          in[u][i].get(f);
#pragma unroll
          for (int v = 0; v < VEC; ++v) acc[i][v] = fmaf(wj[u], f[v], acc[i][v]);
        }
      }
  }
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int c = c0 + i * 32 * VEC;
    if (c < a.d) {
      if (add) {
        float f[VEC];
        last[i].get(f);
#pragma unroll
        for (int v = 0; v < VEC; ++v) acc[i][v] += f[v];
      }
      Piece<YT, VEC>::store(static_cast<YT*>(a.out) + (size_t)t * a.d + c, acc[i]);
    }
  }
}

// A token belongs to W warps of a block, which take its slices in turn; their parts
// of dw meet in shared memory, in order.  Eight picks at a time.
template <typename YT, typename RT, int VEC, int W>
__global__ void __launch_bounds__(kRowThreads) combine_grad_kernel(RowsArgs a) {
  constexpr int P = kSlice<VEC> / (32 * VEC), kTokens = kRowThreads / 32 / W, kPicks = 8;
  __shared__ float part[kTokens][W][kPicks];
  follow();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = warp % W;
  const int slices = (a.d + kSlice<VEC> - 1) / kSlice<VEC>;
  const long long token = (long long)blockIdx.x * kTokens + warp / W;
  const bool live = token < a.T;
  const int t = live ? (int)token : 0;
  const YT* dy = static_cast<const YT*>(a.tokens) + (size_t)t * a.d;
  const RT* rows = static_cast<const RT*>(a.rows_in);
  RT* out = static_cast<RT*>(a.out);
  const int slot = live ? slot_of(a, t, lane) : -1;
  const float w = live && lane < a.k ? a.w[(size_t)t * a.k + lane] : 0.f;
  for (int j0 = 0; j0 < a.k; j0 += kPicks) {
    float dot[kPicks];
#pragma unroll
    for (int u = 0; u < kPicks; ++u) dot[u] = 0.f;
    for (int sl = sub; sl < slices; sl += W) {
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const int c = sl * kSlice<VEC> + lane * VEC + i * 32 * VEC;
        const bool in = live && c < a.d;
        Piece<YT, VEC> g;
        Piece<RT, VEC> r[kPicks];
        if (in) g.load(dy + c);
#pragma unroll
        for (int u = 0; u < kPicks; ++u) {
          const int s = j0 + u < a.k ? __shfl_sync(0xffffffffu, slot, (j0 + u) & 31) : -1;
          if (in && s >= 0 && a.dw) r[u].load(rows + (size_t)s * a.d + c);
        }
        float gf[VEC];
        if (in) g.get(gf);
#pragma unroll
        for (int u = 0; u < kPicks; ++u) {
          const int s = j0 + u < a.k ? __shfl_sync(0xffffffffu, slot, (j0 + u) & 31) : -1;
          const float wj = __shfl_sync(0xffffffffu, w, (j0 + u) & 31);
          if (in && s >= 0) {
            float f[VEC];
            if (a.dw) {
              r[u].get(f);
#pragma unroll
              for (int v = 0; v < VEC; ++v) dot[u] = fmaf(gf[v], f[v], dot[u]);
            }
            if (out) {
#pragma unroll
              for (int v = 0; v < VEC; ++v) f[v] = wj * gf[v];
              Piece<RT, VEC>::store(out + (size_t)s * a.d + c, f);
            }
          }
        }
      }
    }
    if (!a.dw) continue;
#pragma unroll
    for (int u = 0; u < kPicks; ++u) dot[u] = warp_sum(dot[u]);
    if (W == 1) {
      float v = 0.f;
#pragma unroll
      for (int u = 0; u < kPicks; ++u)
        if (lane == u) v = dot[u];
      if (live && lane < kPicks && j0 + lane < a.k) a.dw[(size_t)t * a.k + j0 + lane] = v;
    } else {
      if (lane == 0) {
#pragma unroll
        for (int u = 0; u < kPicks; ++u) part[warp / W][sub][u] = dot[u];
      }
      __syncthreads();
      if (live && sub == 0 && lane < kPicks && j0 + lane < a.k) {
        float v = 0.f;
#pragma unroll
        for (int q = 0; q < W; ++q) v += part[warp / W][q][lane];
        a.dw[(size_t)t * a.k + j0 + lane] = v;
      }
      __syncthreads();
    }
  }
}

template <int VEC>
cudaError_t blocks_of(const RowsArgs& a, int* grid) {
  const long long units = (long long)a.T * ((a.d + kSlice<VEC> - 1) / kSlice<VEC>), per = kRowThreads / 32;
  const long long n = (units + per - 1) / per;
  *grid = (int)n;
  return n > 0x7fffffff ? cudaErrorInvalidValue : cudaSuccess;
}

template <template <typename, typename, int> class Launch>
cudaError_t pick(const RowsArgs& a, int first, int second, cudaStream_t st) {
  typedef __nv_bfloat16 B;
  if (a.d % 8 == 0) {
    if (first == MOE_BF16) return second == MOE_BF16 ? Launch<B, B, 8>::run(a, st) : Launch<B, float, 8>::run(a, st);
    return second == MOE_BF16 ? Launch<float, B, 8>::run(a, st) : Launch<float, float, 8>::run(a, st);
  }
  if (first == MOE_BF16) return second == MOE_BF16 ? Launch<B, B, 1>::run(a, st) : Launch<B, float, 1>::run(a, st);
  return second == MOE_BF16 ? Launch<float, B, 1>::run(a, st) : Launch<float, float, 1>::run(a, st);
}
template <typename XT, typename RT, int VEC>
struct Dispatch {
  static cudaError_t run(const RowsArgs& a, cudaStream_t st) {
    int grid;
    const cudaError_t err = blocks_of<VEC>(a, &grid);
    return err != cudaSuccess ? err : launch_after(dispatch_kernel<XT, RT, VEC>, grid, dim3(kRowThreads), 0, st, a);
  }
};
template <typename RT, typename YT, int VEC>
struct Combine {
  static cudaError_t run(const RowsArgs& a, cudaStream_t st) {
    int grid;
    const cudaError_t err = blocks_of<VEC>(a, &grid);
    return err != cudaSuccess ? err : launch_after(combine_rows_kernel<RT, YT, VEC>, grid, dim3(kRowThreads), 0, st, a);
  }
};
template <typename YT, typename RT, int VEC>
struct CombineGrad {
  static cudaError_t run(const RowsArgs& a, cudaStream_t st) {
    constexpr int kWarps = kRowThreads / 32;
    if (a.T < 2048) return launch_after(combine_grad_kernel<YT, RT, VEC, kWarps>, a.T, dim3(kRowThreads), 0, st, a);
    return launch_after(combine_grad_kernel<YT, RT, VEC, 1>, (a.T + kWarps - 1) / kWarps, dim3(kRowThreads), 0, st, a);
  }
};

}  // namespace

cudaError_t launch_sort_tokens(const SortArgs& a, cudaStream_t st) {
  const size_t smem = (size_t)(kSortWarps + 1) * a.E * 4;
  const cudaError_t err = allow(sort_tokens_kernel, smem, (size_t)(kSortWarps + 1) * kMaxSortExperts * 4);
  if (err != cudaSuccess) return err;
  int ranks = 1;
  while (ranks < kSortCluster && ranks * 2 * kSortThreads <= a.picks) ranks *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ranks);
  cfg.blockDim = dim3(kSortThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = ranks;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, sort_tokens_kernel, a);
}

cudaError_t launch_dispatch(const RowsArgs& a, cudaStream_t st) { return pick<Dispatch>(a, a.t_dtype, a.r_dtype, st); }
cudaError_t launch_combine_rows(const RowsArgs& a, cudaStream_t st) {
  return pick<Combine>(a, a.r_dtype, a.t_dtype, st);
}
cudaError_t launch_combine_backward(const RowsArgs& a, cudaStream_t st) {
  return pick<CombineGrad>(a, a.t_dtype, a.r_dtype, st);
}

}  // namespace moe
