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
// row is read or written once (dy of backward once for every 2, 4 or 8 picks, from L2 but
// for the first time), its k sorted rows once each, and a sum over the picks runs in
// their order, with no atomics.  A slot outside 0 .. n_rows - 1 is taken as
// dropped, so no access leaves the rows.
#include "ops_internal.h"
#include "rows_common.cuh"

namespace moe {
namespace {

// ------------------------------------------------------------------ sort
// One cluster of up to 16 CTAs of 32 warps.  A warp owns a contiguous range of the
// picks.  It counts its picks per expert, the counts become start positions by a
// prefix over the warps, the CTAs (distributed shared memory) and the experts, and a
// second walk over the picks hands them out in order: of 32 picks those of the same
// expert find one another by a ballot for each bit of the id (the instruction that
// matches values over a warp takes some 275 cycles here: 131072 picks 37 us).
//
// Bound by its chain of steps: a launch, a read of idx, two walks, and the exchange
// between the CTAs.
constexpr int kSortThreads = 1024, kSortWarps = 32, kSortCluster = 16;
constexpr int kSortAhead = 4;  // loads of 32 picks in flight per warp

__global__ void __launch_bounds__(kSortThreads, 1) sort_tokens_kernel(SortArgs a) {
  extern __shared__ int sort_sm[];
  const int E = a.E;
  int* hist = sort_sm;                  // [32][E]: of each warp, its counts, then its next positions within its part
  int* part = hist + kSortWarps * E;    // [parts][E]: sums over a part of the warps, then where the part begins
  __shared__ int warp_part[kSortWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)cluster_rank(), ranks = gridDim.x;
  // picks per warp, a multiple of 32, and the warps that have some
  const long long per =
      (((long long)a.picks + (long long)ranks * kSortThreads - 1) / ((long long)ranks * kSortThreads)) * 32;
  const long long first = ((long long)rank * kSortWarps + warp) * per;
  const int lo = (int)min(first, (long long)a.picks), hi = (int)min(first + per, (long long)a.picks);
  const int warps = per ? (int)min((long long)kSortWarps, (a.picks + per - 1) / per) : 1;
  // The warps' counts of an expert are added up by several threads, each a part of the warps.
  const int parts = E <= 32 ? 32 : E <= 64 ? 16 : E <= 128 ? 8 : E <= 256 ? 4 : E <= 512 ? 2 : 1;
  const int part_warps = kSortWarps / parts;
  int* total = part + parts * E;        // [E] of this CTA, read by the others
  int* mine = hist + warp * E;
  for (int e = lane; e < E; e += 32) mine[e] = 0;
  follow();
  __syncwarp();

  auto walk = [&](auto&& each) {
    for (int p0 = lo; p0 < hi; p0 += 32 * kSortAhead) {
      int e[kSortAhead];
#pragma unroll
      for (int u = 0; u < kSortAhead; ++u) {
        const int p = p0 + u * 32 + lane;
        e[u] = p < hi ? a.idx[p] : -1;
        if (e[u] < 0 || e[u] >= E) e[u] = E;  // dropped
      }
#pragma unroll
      for (int u = 0; u < kSortAhead; ++u)
        if (p0 + u * 32 < hi) each(p0 + u * 32 + lane, e[u]);
    }
  };
  walk([&](int, int e) {
    if (e < E) atomicAdd(&mine[e], 1);  // (a count: the order does not matter)
  });
  __syncthreads();
  // prefix over the warps of a part, then over the parts
  const int pe = tid % E, pq = tid / E;
  if (pq < parts) {
    int sum = 0;
    const int w1 = min((pq + 1) * part_warps, warps);
#pragma unroll 8
    for (int w = pq * part_warps; w < w1; ++w) {
      const int c = hist[w * E + pe];
      hist[w * E + pe] = sum;
      sum += c;
    }
    part[pq * E + pe] = sum;
  }
  __syncthreads();
  if (tid < E) {
    int sum = 0;
    for (int q = 0; q < parts; ++q) sum += part[q * E + tid];
    total[tid] = sum;
  }
  cluster_sync();
  // prefix over the CTAs, then over the experts: E <= 1024, one per thread
  int before = 0, all = 0;
  if (tid < E) {
    int c[kSortCluster];
#pragma unroll
    for (int r = 0; r < kSortCluster; ++r) {
      c[r] = 0;
      if (r < ranks) asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(c[r]) : "r"(map_cta(total + tid, r)));
    }
#pragma unroll
    for (int r = 0; r < kSortCluster; ++r) {
      if (r < rank) before += c[r];
      all += c[r];
    }
  }
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");  // the others' totals have been read
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
  if (tid < E) {
    if (rank == 0) {
      if (a.counts) a.counts[tid] = all;
      if (a.offsets) {
        a.offsets[tid] = offset;
        if (tid == E - 1) a.offsets[E] = offset + all;
      }
    }
    int at = offset + before;
    for (int q = 0; q < parts; ++q) {
      const int c = part[q * E + tid];
      part[q * E + tid] = at;
      at += c;
    }
  }
  __syncthreads();
  const int bits = 32 - __clz(E);  // of 0 .. E
  const int* begin = part + warp / part_warps * E;
  walk([&](int p, int e) {
    unsigned same = 0xffffffffu;
    for (int b = 0; b < bits; ++b) {
      const bool bit = (e >> b & 1) != 0;
      const unsigned votes = __ballot_sync(0xffffffffu, bit);
      same &= bit ? votes : ~votes;
    }
    const int rank_here = __popc(same & ((1u << lane) - 1u));
    const bool in = e < E;
    const int at = in ? begin[e] + mine[e] + rank_here : -1;
    __syncwarp();
    if (in && rank_here == 0) mine[e] += __popc(same);
    __syncwarp();
    if (p < hi) {
      if (a.slot) a.slot[p] = at;
      if (a.perm && in) a.perm[at] = p / a.k;
    }
  });
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // no CTA leaves while another reads its totals
}

// ------------------------------------------------------------------ rows
// A lane's columns come in chunks of VEC neighbouring ones: 8 where rows are aligned,
// 2 where the width is even, else one.
template <typename T, int VEC>
struct Piece;
template <typename T>
struct Piece<T, 1> {
  T v;
  MOE_DEV void load(const T* p) { v = *p; }
  MOE_DEV void get(float (&f)[1]) const { f[0] = to_f(v); }
  static MOE_DEV void store(T* p, const float (&f)[1]) { put(p, f[0]); }
};
template <>
struct Piece<float, 2> {
  float2 v;
  MOE_DEV void load(const float* p) { v = *reinterpret_cast<const float2*>(p); }
  MOE_DEV void get(float (&f)[2]) const { f[0] = v.x, f[1] = v.y; }
  static MOE_DEV void store(float* p, const float (&f)[2]) { *reinterpret_cast<float2*>(p) = make_float2(f[0], f[1]); }
};
template <>
struct Piece<__nv_bfloat16, 2> {
  uint32_t v;
  MOE_DEV void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint32_t*>(p); }
  MOE_DEV void get(float (&f)[2]) const { f[0] = bf16_lo(v), f[1] = bf16_hi(v); }
  static MOE_DEV void store(__nv_bfloat16* p, const float (&f)[2]) {
    *reinterpret_cast<uint32_t*>(p) = pack_bf16x2(f[0], f[1]);
  }
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
// A warp's unit of work is a slice of a token's columns: P chunks per lane.
constexpr int slice_columns(int VEC, int P) { return 32 * VEC * P; }

// The slot of lane j's pick, -1 where there is none.
MOE_DEV int slot_of(const RowsArgs& a, int t, int j) {
  const int s = j < a.k ? a.slot[(size_t)t * a.k + j] : -1;
  return s < 0 || s >= a.n_rows ? -1 : s;
}

template <int VEC>
constexpr int kDispatchPieces = VEC == 8 ? 2 : VEC == 2 ? 4 : 8;

template <typename XT, typename RT, int VEC>
__global__ void __launch_bounds__(kRowThreads) dispatch_kernel(RowsArgs a) {
  constexpr int P = kDispatchPieces<VEC>, kCols = slice_columns(VEC, P);
  follow();
  const int lane = threadIdx.x & 31;
  const int slices = (a.d + kCols - 1) / kCols;
  const long long unit = (long long)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);
  if (unit >= (long long)a.T * slices) return;
  const int t = (int)(unit / slices), c0 = (int)(unit - (long long)t * slices) * kCols + lane * VEC;
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

// P chunks of A rows in flight at a time: fewer rows, more of each.  With one row or
// two a unit is short beside the wait for its slots, so the blocks walk over units and
// ask for the next one's slots ahead (WALK; T = 16384, d = 4096: k = 1 83 to 70 us, k = 2
// 95 to 83; with more rows that costs registers and warps: k = 8, d = 2048 101 to 111).
template <typename RT, typename YT, int VEC, int P, int A>
__global__ void __launch_bounds__(kRowThreads) combine_rows_kernel(RowsArgs a) {
  constexpr int kCols = slice_columns(VEC, P);
  constexpr bool WALK = A <= 2;
  follow();
  const int lane = threadIdx.x & 31;
  const int slices = (a.d + kCols - 1) / kCols;
  const long long units = (long long)a.T * slices, stride = (long long)gridDim.x * (kRowThreads / 32);
  long long unit = (long long)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);
  if (unit >= units) return;
  const RT* rows = static_cast<const RT*>(a.rows_in);
  const YT* add = static_cast<const YT*>(a.tokens);
  int t = (int)(unit / slices), slot = slot_of(a, t, lane);
  float w = a.w && lane < a.k ? a.w[(size_t)t * a.k + lane] : 1.f;
  while (true) {
    const int c0 = (int)(unit - (long long)t * slices) * kCols + lane * VEC;
    int next_t = 0, next_slot = -1;
    float next_w = 1.f;
    if (WALK && unit + stride < units) {
      next_t = (int)((unit + stride) / slices);
      next_slot = slot_of(a, next_t, lane);
      if (a.w && lane < a.k) next_w = a.w[(size_t)next_t * a.k + lane];
    }
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
    for (int j0 = 0; j0 < a.k; j0 += A) {
      Piece<RT, VEC> in[A][P];
      int s[A];
      float wj[A];
#pragma unroll
      for (int u = 0; u < A; ++u) {
        s[u] = __shfl_sync(0xffffffffu, slot, (j0 + u) & 31);
        wj[u] = __shfl_sync(0xffffffffu, w, (j0 + u) & 31);
        if (j0 + u >= a.k) s[u] = -1;
        if (s[u] >= 0) {
          const RT* from = rows + (size_t)s[u] * a.d + c0;
#pragma unroll
          for (int i = 0; i < P; ++i)
            if (c0 + i * 32 * VEC < a.d) in[u][i].load(from + i * 32 * VEC);
        }
      }
#pragma unroll
      for (int u = 0; u < A; ++u)
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
    unit += stride;
    if (!WALK || unit >= units) return;
    t = next_t, slot = next_slot, w = next_w;
  }
}

// A token belongs to W warps of a block, which take its slices in turn; their parts
// of dw meet in shared memory, in order.  K picks at a time.
template <int VEC, int K>
constexpr int kGradPieces = (VEC == 8 ? 1 : VEC == 2 ? 2 : 4) * (K == 2 ? VEC == 8 ? 4 : 2 : K == 4 && VEC == 8 ? 2 : 1);
template <typename YT, typename RT, int VEC, int W, int K>
__global__ void __launch_bounds__(kRowThreads) combine_grad_kernel(RowsArgs a) {
  constexpr int P = kGradPieces<VEC, K>, kTokens = kRowThreads / 32 / W, kPicks = K;
  constexpr int kStep = 32 * VEC * P;  // columns of a warp at a time
  __shared__ float part[kTokens][W][kPicks];
  follow();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = warp % W;
  const long long token = (long long)blockIdx.x * kTokens + warp / W;
  const bool live = token < a.T;  // (others stay for the barriers)
  const int t = live ? (int)token : 0;
  const YT* dy = static_cast<const YT*>(a.tokens) + (size_t)t * a.d;
  const RT* rows = static_cast<const RT*>(a.rows_in);
  RT* out = static_cast<RT*>(a.out);
  const int slot = live ? slot_of(a, t, lane) : -1;
  const float w = live && lane < a.k ? a.w[(size_t)t * a.k + lane] : 0.f;
  for (int j0 = 0; j0 < a.k; j0 += kPicks) {
    float dot[kPicks], wj[kPicks];
    size_t row[kPicks];  // first value of the pick's row
    unsigned kept = 0;
#pragma unroll
    for (int u = 0; u < kPicks; ++u) {
      dot[u] = 0.f;
      const int s = __shfl_sync(0xffffffffu, slot, (j0 + u) & 31);
      wj[u] = __shfl_sync(0xffffffffu, w, (j0 + u) & 31);
      if (j0 + u < a.k && s >= 0) kept |= 1u << u;
      row[u] = (size_t)max(s, 0) * a.d;
    }
    for (int c0 = sub * kStep + lane * VEC; c0 < a.d; c0 += W * kStep) {
      Piece<YT, VEC> g[P];
      Piece<RT, VEC> r[P][kPicks];
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const int c = c0 + i * 32 * VEC;
        if (c < a.d) g[i].load(dy + c);
      }
      if (a.dw) {
#pragma unroll
        for (int u = 0; u < kPicks; ++u)
          if (kept >> u & 1) {
            const RT* from = rows + row[u] + c0;
#pragma unroll
            for (int i = 0; i < P; ++i)
              if (c0 + i * 32 * VEC < a.d) r[i][u].load(from + i * 32 * VEC);
          }
      }
      float gf[P][VEC];
#pragma unroll
      for (int i = 0; i < P; ++i) g[i].get(gf[i]);
#pragma unroll
      for (int u = 0; u < kPicks; ++u)
        if (kept >> u & 1) {
          RT* to = out + row[u] + c0;
#pragma unroll
          for (int i = 0; i < P; ++i)
            if (c0 + i * 32 * VEC < a.d) {
              float f[VEC];
              if (a.dw) {
                r[i][u].get(f);
#pragma unroll
                for (int v = 0; v < VEC; ++v) dot[u] = fmaf(gf[i][v], f[v], dot[u]);
              }
              if (out) {
#pragma unroll
                for (int v = 0; v < VEC; ++v) f[v] = wj[u] * gf[i][v];
                Piece<RT, VEC>::store(to + i * 32 * VEC, f);
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

int blocks_of(const RowsArgs& a, int columns) {  // of a warp per unit of work; fewer than 2^30 (check_rows)
  const long long units = (long long)a.T * ((a.d + columns - 1) / columns);
  return (int)((units + kRowThreads / 32 - 1) / (kRowThreads / 32));
}

template <template <typename, typename, int> class Launch>
cudaError_t pick(const RowsArgs& a, int first, int second, cudaStream_t st) {
  typedef __nv_bfloat16 B;
  auto types = [&](auto vec) {
    constexpr int V = decltype(vec)::value;
    if (first == MOE_BF16) return second == MOE_BF16 ? Launch<B, B, V>::run(a, st) : Launch<B, float, V>::run(a, st);
    return second == MOE_BF16 ? Launch<float, B, V>::run(a, st) : Launch<float, float, V>::run(a, st);
  };
  return a.d % 8 == 0 ? types(ActTag<8>()) : a.d % 2 == 0 ? types(ActTag<2>()) : types(ActTag<1>());
}
template <typename XT, typename RT, int VEC>
struct Dispatch {
  static cudaError_t run(const RowsArgs& a, cudaStream_t st) {
    const int grid = blocks_of(a, slice_columns(VEC, kDispatchPieces<VEC>));
    return launch_after(dispatch_kernel<XT, RT, VEC>, grid, dim3(kRowThreads), 0, st, a);
  }
};
template <typename RT, typename YT, int VEC>
struct Combine {
  template <int P, int A>
  static cudaError_t launch(const RowsArgs& a, cudaStream_t st) {
    const auto kernel = combine_rows_kernel<RT, YT, VEC, P, A>;
    int grid = blocks_of(a, slice_columns(VEC, P));
    if (A <= 2 && grid > 128) {
      static ByDevice known;
      const int resident = resident_blocks(kernel, kRowThreads, 0, known);
      if (grid > resident) grid = resident;
    }
    return launch_after(kernel, grid, dim3(kRowThreads), 0, st, a);
  }
  static cudaError_t run(const RowsArgs& a, cudaStream_t st) {
    constexpr int M = VEC == 8 ? 1 : VEC == 2 ? 2 : 4;
    return a.k == 1 ? launch<4 * M, 1>(a, st) : a.k == 2 ? launch<4 * M, 2>(a, st) : launch<VEC == 1 ? 4 : 2 * M, 4>(a, st);
  }
};
template <typename YT, typename RT, int VEC>
struct CombineGrad {
  template <int W, int K>
  static cudaError_t launch(const RowsArgs& a, cudaStream_t st) {
    constexpr int kTokens = kRowThreads / 32 / W;
    return launch_after(combine_grad_kernel<YT, RT, VEC, W, K>, (a.T + kTokens - 1) / kTokens, dim3(kRowThreads), 0, st, a);
  }
  template <int K>
  static cudaError_t split(const RowsArgs& a, cudaStream_t st) {
    // Warps per token.  Aligned: as many as keep the warps of all tokens below 16 per SM (k = 8, d = 2048: T = 500 12.2,
    // 8.4, 7.3, 8.1 us with 1, 2, 4, 8; T = 2000 23.2, 25.0, 26.7, 29.9).  Others move smaller pieces, which several warps
    // side by side do better at any T (k = 8, T = 4000, d = 2501: 89, 90, 82, 81; d = 2502: 85, 73, 67, 72), as far as each has
    // two rounds of them.
    const int rounds = a.d / (2 * 32 * VEC * kGradPieces<VEC, K>);
    const int most = VEC == 8 ? 16 * 152 / a.T : rounds < 1 ? 1 : VEC == 1 ? rounds : rounds < 4 ? rounds : 4;
    return most >= 8 ? launch<8, K>(a, st) : most >= 4 ? launch<4, K>(a, st) : most >= 2 ? launch<2, K>(a, st) : launch<1, K>(a, st);
  }
  // Picks at a time: 2, 4 or 8, with as many loads in flight (T = 2458, d = 3688, k = 4 28.8 us for 43.1 with 8 places for
  // them; k = 8 the other way round, T = 4000, d = 2048 in fp32 48.6 for 56.7 with 4).  Odd widths, whose loads are of one
  // value, have no registers for 8: k = 8, T = 16384, d = 513 137 us for 77.8 with 4; T = 4000, d = 2501 89.3 for 80.4.
  static cudaError_t run(const RowsArgs& a, cudaStream_t st) {
    return a.k <= 2 ? split<2>(a, st) : a.k <= 4 || VEC == 1 ? split<4>(a, st) : split<VEC == 1 ? 4 : 8>(a, st);
  }
};

}  // namespace

// Prepares the sort on the current device: the most CTAs of a cluster there, 16 (more than every device promises a cluster)
// or 8.
static cudaError_t prepare_sort(int* ranks) {
  constexpr size_t most = (size_t)(kSortWarps + 2) * kMaxSortExperts * 4;  // (parts: 1024 sums at most)
  *ranks = 8;
  cudaError_t err = cudaFuncSetAttribute(sort_tokens_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
  if (err == cudaSuccess) err = cudaFuncSetAttribute(sort_tokens_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3(kSortCluster);
  c.blockDim = dim3(kSortThreads);
  c.dynamicSmemBytes = most;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = kSortCluster;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  c.attrs = &at;
  c.numAttrs = 1;
  int n = 0;
  err = cudaOccupancyMaxActiveClusters(&n, sort_tokens_kernel, &c);
  if (err == cudaSuccess && n > 0) *ranks = kSortCluster;
  return err;
}

cudaError_t launch_sort_tokens(const SortArgs& a, cudaStream_t st) {
  static ByDevice prepared;
  const int most_ranks = once_per_device(prepared, prepare_sort);
  const size_t smem = (size_t)(kSortWarps + 1) * a.E * 4 + 1024 * 4;
  int ranks = 1;
  while (ranks < most_ranks && ranks * 2 * kSortThreads <= a.picks) ranks *= 2;
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
