// The gated feed-forward block's matrix products on the 5th-generation tensor
// cores, for the forward and the backward pass.
//
//   gate_up   [g | u] = x gate_up^T; h = act(g) * u        (x, weights K-major)
//   down      y = h down^T
//   grad_h    dh = dy down; dpre = [dh u act'(g) | dh act(g)]; h = act(g) * u
//   dx        dx = dpre gate_up
//   dgate_up  dpre^T x
//   ddown     dy^T h
//   linear    y = act(x weight^T + bias) + residual        (not gated; a block of its own)
//
// One persistent kernel.  A pair of CTAs on neighbouring SMs (a cluster of two)
// computes a 256 x 256 tile with tcgen05.mma.cta_group::2: each CTA loads its
// own 128 rows of A and half of B's 256 rows, so a 64-deep k block costs each
// SM 32 KB of shared-memory fill for 512 cycles of MMA (a lone CTA's 128 x 256
// tile takes 48 KB for the same work).  Per CTA 11 warps (12 for mx8, 19 for linear):
//   warp 0 and the last  TMA producers (one thread each) of a ring of k blocks,
//              128-byte swizzle: A, B, and mx8's scales.  A thread takes some 100
//              cycles to issue a copy and up to 300 to see that a stage is free,
//              against a k block's 512 cycles of MMAs;
//   warp 1     allocates all 512 TMEM columns: two fp32 accumulators of 256
//              columns; in the pair's first CTA one thread issues the MMAs;
//   warps 2 on  epilogue: two warps (linear: four) for each quarter of the TMEM
//              lanes, each taking its part of the columns; a thread has a row of
//              the sums.  Products leave through shared memory by whole lines; for
//              linear the sums change hands there (see the two blocks below); the
//              other forms write 16 columns (32 bytes) of a row at a time.
// The epilogue of tile i overlaps the main loop of tile i + 1.  In the gate/up
// product B's first half holds gate rows and the second half the up rows of the
// same 128 neurons, so the activation finishes in the accumulator's columns.
//
// A product with fewer tiles than pairs splits the reduction over 2 or 4 pairs
// of one cluster (SPLIT; linear and its gradients also over 3: 16 tiles find 15
// clusters of 4 pairs on the device, T = 128, 4096 to 4096 17.5 us with 2, 16.0
// with 3; backward T = 300, 2048 to 8192 50.0 and 43.3).  Each pair ends with fp32
// sums of the whole tile; the columns are divided among the pairs, every CTA sends its sums of the others'
// columns to them through distributed shared memory (the ring's memory, free by
// then), and each adds its columns' sums in the order of k and finishes them.
//
// Operands may lie K-major (the reduction contiguous in memory) or MN-major:
// dx, dgate_up and ddown read the forward pass's matrices where they lie, with
// no transposed copies.  A ragged M, N or K reads zeros from TMA's bounds fill.
//
// The mx8 form of gate_up and down runs on the block-scaled 8-bit instruction
// (kind::mxf8f6f4, one e8m0 scale per 32 values of k): a k block is 128 values,
// the same 128 bytes.  The scale bytes are stored in the order in which
// tcgen05.cp moves them into tensor memory, so a k block brings 512 bytes of
// scales per 128 rows and three copies; each CTA needs its own rows' and all of
// B's.  They take TMEM columns, so the two accumulators there share 48 columns:
// the epilogue reads those first and the next tile's MMAs may then start.  h is
// rounded to mx8 in the epilogue, where a thread holds a whole group of 32.
//
// Every wait is bounded; on expiry the kernel drains what it has in flight,
// frees TMEM and returns (see the end of the kernel).
//
// What bounds it: large bf16 products the MMAs (the tensor pipe is active 82-85%
// of the time, in grad_h 65%) and, run back to back, the card's power: T = 8192, d
// = 4096, I = 16384 with pre saved, 1.96-2.11 ms, 1.57-1.68 PFLOP/s; the backward
// call at T = 4096 2.06-2.17 ms.  mx8 at T = 8191 1.16-1.27 ms, 2.6-2.8 PFLOP/s,
// the tensor pipe active 61% (T = 4096, I = 8192): a block's data,
// its scales' copies and the sight of both have to come in time for 512 cycles of
// MMAs (TMEM has room for four blocks' scales).  Few tiles: the ~1 us that each
// of a launch's start, first loads, epilogue and end take.
#include "rows_common.cuh"

namespace moe {
namespace {

constexpr int kBM = 128;                    // rows of A per CTA
constexpr int kBN = 256;                    // accumulator columns
constexpr int kRowBytes = 128;              // a k block: 64 bf16 or 128 e4m3 values
constexpr int kBK = 64;                     // k block of bf16
constexpr int kOpBytes = 128 * kRowBytes;   // one operand's half tile: 16 KB
constexpr int kStageBytes = 2 * kOpBytes;   // per CTA
constexpr int kEpiWarps = 8;                // epilogue warps; twice as many where results are staged, see there
constexpr int roles_of(bool mx) { return mx ? 3 : 2; }  // producers: A on warp 0, B on the first after the epilogue's, mx8's scales
constexpr int kScaleBytes = 3 * 512;        // mx8 scales of a k block: A's 128 rows, B's 2 x 128
constexpr int kScaleSets = 4;               // mx8: k blocks whose scales TMEM holds, 12 columns each
constexpr int kSharedCols = 12 * kScaleSets;  // mx8: accumulator columns that both tiles use
static_assert(kSharedCols % 16 == 0 && kSharedCols <= 64, "the epilogue reads them in whole chunks, at most two groups");
constexpr uint32_t kScaleCol = 2 * kBN - kSharedCols;
// What a tile costs besides its k blocks, in k blocks (~0.27 us), see split_of(): its start and end; its epilogue by kind
// (a split divides that too); the exchange of a split.
constexpr int kTileCost = 6, kSplitCost = 7, kLaunchCost = 8;  // (and of another launch)
constexpr int kNextTileCost = 6;  // a weight gradient's tile after the pair's first
constexpr int epilogue_cost(int epi) { return epi == 0 ? 4 : epi == 2 ? 16 : 9; }
constexpr int kGroupM = 8;                  // m-tiles that share a sweep over n (L2 reuse)

enum { kEpiStore, kEpiGateUp, kEpiGrad, kEpiLinear };

// One product: result [M, N] = a b^T over K.
struct Product {
  CUtensorMap a, b;
  uint16_t* y;                     // bf16 result: y / dx / dW, or h
  int M, N, K;                     // N: columns of the result (gate/up: neurons)
  int a_mn;                        // MULTI: a is MN-major
  int wide;                        // rows of the results are 32-byte aligned (a tensor's first row need only be 16)
  int mt, nt, tiles, blocks;       // m-tiles, n-tiles, their product, k blocks
};
struct GemmParams {
  Product q[3];                    // MULTI: up to three, those with the longer reduction first; else one
  int count;                       // MULTI: products
  int heavy_count, heavy_tiles;    // MULTI: the first products, of the longer reduction, and their tiles
  int early;                       // MULTI: light tiles that take as long as a heavy one
  CUtensorMap as, bs0, bs1;        // mx8 scales: of A, and of the two 128-row halves of B
  uint8_t *hq, *hs;                // mx8 gate/up: codes and scales of h
  uint16_t* pre_out;               // gate/up: pre [M, 2N], or NULL; linear: pre [M, N], or NULL
  const uint16_t* pre;             // grad: pre [M, 2N]
  uint16_t* dpre;                  // grad: [M, 2N]
  const void *bias, *res;          // linear: [N] and [M, N], or NULL
  int bias_bf16, y32;              // linear: the bias is bf16; result and residual are fp32
  int wide32;                      // linear: rows of an fp32 result are 32-byte aligned
  int act;
  DevCtl ctl;
};

constexpr int kStages = 6;
constexpr int stage_bytes(bool mx) { return kStageBytes + (mx ? kScaleBytes : 0); }

struct __align__(8) Bars {
  uint64_t full[6];    // used in the first CTA: both CTAs' copies of a k block have landed
  uint64_t empty[6];   // the MMAs of a k block are done (committed to both CTAs)
  uint64_t tfull[2];   // an accumulator is complete (both CTAs)
  uint64_t tempty[2];  // used in the first CTA: both CTAs' epilogues have read an accumulator
  uint64_t mma_done;
  uint64_t free[4];          // SPLIT: the cluster's i-th pair takes in sums now
  uint64_t recv[kEpiWarps];  // SPLIT: the other pairs' sums of an epilogue warp's columns have come
  uint32_t tmem_base;
  int abort_flag;
  uint32_t issued[2][3];  // k blocks loaded by each CTA's producers (first CTA: both's)
  uint32_t any_abort;     // some CTA of the cluster has given up
};

// Results that go to memory by way of shared memory: an epilogue warp's place there has its 32 rows of 128 bytes.
constexpr int kPlaceBytes = 32 * 128;
constexpr bool staged(int epi, bool mx, int split) { return (epi == kEpiStore || epi == kEpiLinear) && !mx && split == 1; }
constexpr int stages_of(int epi, bool mx, int split) { return staged(epi, mx, split) && epi == kEpiLinear ? kStages - 1 : kStages; }
constexpr int epi_warps(int epi, bool mx, int split) { return staged(epi, mx, split) && epi == kEpiLinear ? 2 * kEpiWarps : kEpiWarps; }
constexpr int threads_of(int epi, bool mx, int split) { return (2 + epi_warps(epi, mx, split) + roles_of(mx) - 1) * 32; }
constexpr size_t smem_of(int epi, bool mx, int split) {
  return 1024 + (size_t)stages_of(epi, mx, split) * stage_bytes(mx) + (staged(epi, mx, split) ? epi_warps(epi, mx, split) * kPlaceBytes : 0) + sizeof(Bars);
}
static_assert(smem_of(kEpiGateUp, true, 1) <= 227 * 1024 && smem_of(kEpiStore, false, 1) <= 227 * 1024 && smem_of(kEpiLinear, false, 1) <= 227 * 1024,
              "shared memory of one CTA");

MOE_DEV void store_cluster(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
// TMA load into this CTA whose bytes count on a barrier of the pair's first CTA.
MOE_DEV void tma_load_pair(void* dst, const CUtensorMap* m, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
      "[%4];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
MOE_DEV void store32(void* to, const uint32_t(&w)[8]) {  // 32-byte aligned
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(to), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
MOE_DEV void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }
MOE_DEV void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// The same with e4m3 operands and e8m0 scales in TMEM (32 values of k, one scale each).
MOE_DEV void mma_pair_mx(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb,
                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
      : "memory");
}
// 512 bytes of scales (32 rows of 16 bytes) from the same place in both CTAs'
// shared memory into 4 TMEM columns, repeated for the four lane quarters.
MOE_DEV void copy_scales_pair(uint32_t tmem, uint32_t saddr) {
  const uint64_t d = mx_scale_desc(saddr);
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(d) : "memory");
}
// One 512-byte scale tile, counted on a barrier of the pair's first CTA.
MOE_DEV void tma_load_scales_pair(void* dst, const CUtensorMap* m, int col, int row, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, "
      "%4}], [%5];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(0), "r"(col), "r"(row), "r"(bar)
      : "memory");
}
// Arrive on `bar` of both CTAs once this thread's earlier MMAs have finished.
MOE_DEV void commit_pair(uint64_t* bar, uint16_t both) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"(both)
      : "memory");
}

// Whether a phase has completed, without waiting.
MOE_DEV bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
// Whether `ok` holds in all 256 threads of the epilogue warps.
MOE_DEV bool all_of_256(bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.and.aligned.pred q, 1, 256, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(ok ? 1u : 0u)
      : "memory");
  return r != 0;
}
// `bytes` of this CTA's shared memory to another CTA of the cluster (addresses there: dst, bar).
MOE_DEV void copy_to_cta(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "r"(smem_u32(src)), "r"(bytes), "r"(bar)
               : "memory");
}
MOE_DEV bool aborted(const Bars* b) { return *reinterpret_cast<const volatile int*>(&b->abort_flag) != 0; }
MOE_DEV void set_abort(Bars* b) { *reinterpret_cast<volatile int*>(&b->abort_flag) = 1; }

// The j-th tile of a pair: its product, m-tile and n-tile; false past the last.
// A product's tiles are swept kGroupM m-tiles at a time, all n for each group,
// so that the pairs of one moment share operands in L2.
//
// MULTI: independent products in one launch, so that only one of them ends with
// idle pairs.  The heavy tiles (longer reduction) are dealt out first, round
// robin; the light tiles follow in the order in which pairs come free: the pairs
// that got one heavy tile less deal among themselves for the `early` rounds that
// a heavy tile lasts, then all deal.
struct Tile {
  int q, m, n;
};
template <bool MULTI>
MOE_DEV bool tile_of(const GemmParams& p, int pair, int pairs, int j, Tile& t) {
  int i;
  t.q = 0;
  if (!MULTI) {
    i = pair + j * pairs;
    if (i >= p.q[0].tiles) return false;
  } else {
    const int rem = p.heavy_tiles % pairs, mine = p.heavy_tiles / pairs + (pair < rem ? 1 : 0);
    int last;
    if (j < mine) {
      i = pair + j * pairs;
      last = p.heavy_count;
    } else {
      const int f = j - mine, fewer = rem ? pairs - rem : 0, skip = rem ? p.early : 0;  // pairs with a heavy tile less
      i = rem && pair >= rem && f < skip ? f * fewer + pair - rem
                                         : skip * fewer + (rem && pair >= rem ? f - skip : f) * pairs + pair;
      t.q = p.heavy_count;
      last = p.count;
    }
    while (t.q < last && i >= p.q[t.q].tiles) i -= p.q[t.q++].tiles;
    if (t.q >= last) return false;
  }
  const int mt = p.q[t.q].mt, nt = p.q[t.q].nt;
  const int per = kGroupM * nt, g = i / per, r = i - g * per;
  const int gm = min(kGroupM, mt - g * kGroupM);
  t.m = g * kGroupM + r % gm;
  t.n = r / gm;
  return true;
}

template <int EPI, bool A_MN, bool B_MN, bool MX, int SPLIT, bool MULTI>
__global__ void __launch_bounds__(threads_of(EPI, MX, SPLIT), 1)
    ffn_gemm_kernel(const __grid_constant__ GemmParams p) {
  constexpr int S = stages_of(EPI, MX, SPLIT);
  constexpr uint32_t kTx = stage_bytes(MX);        // bytes per CTA and k block
  static_assert(!MX || (!A_MN && !B_MN && EPI != kEpiGrad), "mx8: forward products only");
  constexpr int TN = EPI == kEpiGateUp ? kBN / 2 : kBN;  // result columns per tile
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = smem_raw + (-smem_u32(smem_raw) & 1023u);  // (the compiler still sees shared memory in it)
  uint8_t* scales = base + S * kStageBytes;  // mx8; else, where results are staged, the places
  constexpr bool kStaged = staged(EPI, MX, SPLIT);
  constexpr int E = epi_warps(EPI, MX, SPLIT), kBWarp = 2 + E;
  Bars* bar = reinterpret_cast<Bars*>(scales + (MX ? S * kScaleBytes : kStaged ? E * kPlaceBytes : 0));

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t crank = cluster_rank(), rank = crank & 1, lead = crank & ~1u;  // rank in the pair, its first CTA
  const int slot = SPLIT > 1 ? (int)crank >> 1 : 0;                             // the pair's part of the reduction
  const int pair = blockIdx.x / (2 * SPLIT), pairs = gridDim.x / (2 * SPLIT);   // (SPLIT: a cluster has one tile)
  static_assert(!MULTI || (EPI == kEpiStore && B_MN && !MX && SPLIT == 1), "MULTI: dx and the weights' gradients");
  Tile t;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 6; ++i) {
      mbar_init(&bar->full[i], 1);
      mbar_init(&bar->empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar->tfull[i], 1);
      mbar_init(&bar->tempty[i], 2 * E);
    }
    mbar_init(&bar->mma_done, 1);
    for (int i = 0; i < 4; ++i) mbar_init(&bar->free[i], 1);
    for (int i = 0; i < kEpiWarps; ++i) mbar_init(&bar->recv[i], 1);
    bar->abort_flag = 0;
    bar->any_abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&bar->tmem_base))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers and TMEM are ready
  tc_fence_after();
  const uint32_t tmem = bar->tmem_base;
  // Launched while the kernel before may still run: the setup above overlaps its end, everything below follows it.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");

  if (warp == 0 || warp >= kBWarp) {
    if (lane == 0) {
      const int role = warp == 0 ? 0 : warp - kBWarp + 1;
      tma_prefetch_desc(role == 0 ? &p.q[0].a : role == 1 ? &p.q[0].b : &p.as);
      bool ok = true;
      int issued = 0;
      for (int i = 0; ok && tile_of<MULTI>(p, pair, pairs, i, t); ++i) {
        const Product& q = p.q[MULTI ? t.q : 0];
        const bool a_mn = MULTI ? q.a_mn != 0 : A_MN;
        const int m = t.m, n = t.n, kb0 = slot * q.blocks / SPLIT, kb1 = (slot + 1) * q.blocks / SPLIT;
        const int arow = (2 * m + (int)rank) * kBM;
        // B's half: gate rows in the first CTA, up rows in the second
        const int brow = EPI == kEpiGateUp ? n * TN + (int)rank * q.N : n * TN + (int)rank * 128;
        for (int kb = kb0; kb < kb1; ++kb) {
          const int st = issued % S;
          if (!mbar_wait(&bar->empty[st], ((issued / S) & 1) ^ 1, p.ctl) || aborted(bar)) {
            set_abort(bar);
            ok = false;
            break;
          }
          const uint32_t fb = map_cta(&bar->full[st], lead);
          uint8_t* a = base + st * kStageBytes;
          uint8_t* b = a + kOpBytes;
          const int k = kb * (MX ? kRowBytes : kBK);
          if (role == 0) {
            if (rank == 0) mbar_expect_tx(&bar->full[st], 2 * kTx);  // everything, both CTAs'
            if (a_mn) {
              tma_load_pair(a, &q.a, arow, k, fb);
              tma_load_pair(a + kOpBytes / 2, &q.a, arow + 64, k, fb);
            } else {
              tma_load_pair(a, &q.a, k, arow, fb);
            }
          } else if (role == 1) {
            if (B_MN) {
              tma_load_pair(b, &q.b, brow, k, fb);
              tma_load_pair(b + kOpBytes / 2, &q.b, brow + 64, k, fb);
            } else {
              tma_load_pair(b, &q.b, k, brow, fb);
            }
          } else if (MX) {
            uint8_t* sc = scales + st * kScaleBytes;
            tma_load_scales_pair(sc, &p.as, kb, 2 * m + (int)rank, fb);
            tma_load_scales_pair(sc + 512, &p.bs0, kb, EPI == kEpiGateUp ? n : 2 * n, fb);
            tma_load_scales_pair(sc + 1024, &p.bs1, kb, EPI == kEpiGateUp ? n : 2 * n + 1, fb);
          }
          ++issued;
        }
      }
      bar->issued[rank][role] = issued;
    }
  } else if (warp == 1) {
    // Seeing that a block has landed takes a load from shared memory, which queues behind the operand reads of the MMAs
    // issued before it (some 300 cycles of a block's 512).
    const uint16_t both = (uint16_t)(3u << lead);  // the pair's CTAs in the cluster
    int it = 0, lt = 0;
    bool ok = true;
    if (p.ctl.stall && rank == 0) {  // test hook: nothing arrives there before the end
      if (lane == 0) ok = mbar_wait(&bar->mma_done, 0, p.ctl);
      ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
    }
    if constexpr (!MX) {
      if (rank == 0 && lane == 0) {
        bool ready = false;
        for (; ok && tile_of<MULTI>(p, pair, pairs, lt, t); ++lt) {
          const Product& q = p.q[MULTI ? t.q : 0];
          const bool a_mn = MULTI ? q.a_mn != 0 : A_MN;
          const uint32_t idesc = umma_idesc_bf16(2 * kBM, kBN) | (a_mn ? 1u << 15 : 0u) | (B_MN ? 1u << 16 : 0u);
          const int kb0 = slot * q.blocks / SPLIT, kb1 = (slot + 1) * q.blocks / SPLIT;
          const int acc = lt & 1;
          // the accumulator was read two tiles ago
          if (!mbar_wait(&bar->tempty[acc], ((lt >> 1) & 1) ^ 1, p.ctl) || aborted(bar)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d = tmem + acc * kBN;
          for (int kb = kb0; kb < kb1; ++kb, ++it) {
            const int st = it % S;
            if (!ready && (!mbar_wait(&bar->full[st], (it / S) & 1, p.ctl) || aborted(bar))) {
              ok = false;
              break;
            }
            // asked for before this block's MMAs
            ready = mbar_test(&bar->full[(it + 1) % S], ((it + 1) / S) & 1);
            tc_fence_after();
            const uint32_t a = smem_u32(base + st * kStageBytes), b = a + kOpBytes;
            const uint64_t da = a_mn ? desc_mn(a) : umma_desc_sw128(a), db = B_MN ? desc_mn(b) : umma_desc_sw128(b);
            // 16 k: 32 bytes along a K-major row, 16 rows of 128 bytes of an MN-major tile
            const uint64_t sa = a_mn ? 128 : 2, sb = B_MN ? 128 : 2;
#pragma unroll
            for (int j = 0; j < kBK / 16; ++j) mma_pair(d, da + j * sa, db + j * sb, idesc, kb != kb0 || j != 0);
            commit_pair(&bar->empty[st], both);
          }
          if (ok) commit_pair(&bar->tfull[acc], both);
        }
      }
    } else if (rank == 0) {
      // A block needs its data and a set of scale columns, which the MMAs of the block kScaleSets before it must have
      // left (tcgen05.cp and a later MMA keep their order, an MMA and a later tcgen05.cp need not).  Lanes 0-5 look at
      // the stages, lanes 8 on at the blocks before, all at once, and lane 0 issues what can go.  T = 4096, d = 4096, I =
      // 8192, a forward call: 340 us with two sets, 316 with three, 310 with four.
      for (; ok && tile_of<MULTI>(p, pair, pairs, lt, t); ++lt) {
        const Product& q = p.q[0];
        const int kb0 = slot * q.blocks / SPLIT, kb1 = (slot + 1) * q.blocks / SPLIT;
        const int acc = lt & 1;
        // the tile before has left the shared columns (which its epilogue warps reach only after the tile before that)
        if (lane == 0) ok = (lt == 0 || mbar_wait(&bar->tempty[0], (lt - 1) & 1, p.ctl)) && !aborted(bar);
        const uint32_t d = tmem + acc * (kBN - kSharedCols);
        for (int kb = kb0; kb < kb1;) {
          const int before = it + lane - 8 - kScaleSets;  // lanes 8 on: blocks it - kScaleSets ... it - 1
          bool yes = true;
          if (lane < S)
            yes = mbar_test(&bar->full[(it + lane) % S], ((it + lane) / S) & 1);
          else if (lane >= 8 && lane < 8 + kScaleSets && before >= 0)
            yes = mbar_test(&bar->empty[before % S], (before / S) & 1);
          const uint32_t seen = __ballot_sync(0xffffffffu, yes);
          int n = min(__ffs(~(seen & 0xffu)) - 1, __ffs(~(seen >> 8 & ((1u << kScaleSets) - 1u))) - 1);
          if (n == 0) {
            if (lane == 0)
              ok = ok && mbar_wait(&bar->full[it % S], (it / S) & 1, p.ctl) &&
                   (it < kScaleSets || mbar_wait(&bar->empty[(it - kScaleSets) % S], ((it - kScaleSets) / S) & 1, p.ctl)) &&
                   !aborted(bar);
            n = 1;
          }
          ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
          if (!ok) break;
          n = min(n, kb1 - kb);
          if (lane == 0) {
            tc_fence_after();
            for (int i = it; i < it + n; ++i) {
              const int st = i % S;
              const uint32_t a = smem_u32(base + st * kStageBytes);
              const uint64_t da = umma_desc_sw128(a), db = umma_desc_sw128(a + kOpBytes);
              const uint32_t sc = smem_u32(scales + st * kScaleBytes), ts = tmem + kScaleCol + i % kScaleSets * 12;
#pragma unroll
              for (int j = 0; j < 3; ++j) copy_scales_pair(ts + 4 * j, sc + 512 * j);
#pragma unroll
              for (int j = 0; j < 4; ++j)
                mma_pair_mx(d, da + j * 2, db + j * 2, umma_idesc_mx(2 * kBM, kBN, j), ts, ts + 4,
                            kb + i != kb0 + it || j != 0);
              commit_pair(&bar->empty[st], both);
            }
          }
          __syncwarp();
          kb += n;
          it += n;
        }
        if (ok && lane == 0) commit_pair(&bar->tfull[acc], both);
      }
    }
    if (rank == 0 && lane == 0) {
      if (!ok) set_abort(bar);
      // the MMAs issued so far are done before TMEM is freed and shared memory left
      asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                       smem_u32(&bar->mma_done))
                   : "memory");
      mbar_wait(&bar->mma_done, 0, drain_ctl(p.ctl));
    }
    __syncwarp();
  } else {
    const int ew = warp - 2, part = warp & 3, half = ew >> 2;
    const uint32_t lanes = (uint32_t)(part * 32) << 16;
    // 16 columns of a row as bf16; N is a multiple of 8, and of 16 where q.wide is set
    auto store16 = [&](const Product& q, uint16_t* to, int pitch, int row, int col, const float(&v)[16]) {
      if (row >= q.M) return;
      uint32_t w[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = pack_bf16x2(v[2 * e], v[2 * e + 1]);
      uint16_t* at = to + (size_t)row * pitch + col;
      if (q.wide) {
        if (col < q.N) store32(at, w);
      } else {
        if (col < q.N) *reinterpret_cast<uint4*>(at) = make_uint4(w[0], w[1], w[2], w[3]);
        if (col + 8 < q.N) *reinterpret_cast<uint4*>(at + 8) = make_uint4(w[4], w[5], w[6], w[7]);
      }
    };
    // 16 columns from column col on as 2 or 4 x 16 bytes, 8 columns at a time.
    auto load16 = [&](const Product& q, const void* from, bool wide, size_t at, int col, bool ok, uint4* to) {
      const uint4* v = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(from) + at * (wide ? 4 : 2));
      const int n = wide ? 4 : 2;
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (c < n) to[c] = ok && col + c * 16 / n < q.N ? v[c] : make_uint4(0, 0, 0, 0);
    };
    // What 16 columns of a row need besides their sums, asked for ahead of them.  grad: pre's values; linear: the
    // residual (first four) and the bias, as they lie in memory.
    constexpr int kIn = EPI == kEpiLinear ? 8 : 4;
    auto load_pre = [&](const Product& q, int row, int col, uint4(&in)[kIn]) {
      if constexpr (EPI == kEpiLinear) {
        if (p.res) load16(q, p.res, p.y32, (size_t)row * q.N + col, col, row < q.M, in);
        if (p.bias) load16(q, p.bias, !p.bias_bf16, col, col, true, in + 4);
      }
      if (EPI != kEpiGrad) return;
      const uint16_t* gp = p.pre + (size_t)row * 2 * q.N + col;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const bool ok = row < q.M && col + c * 8 < q.N;
        in[c] = ok ? *reinterpret_cast<const uint4*>(gp + c * 8) : make_uint4(0, 0, 0, 0);
        in[2 + c] = ok ? *reinterpret_cast<const uint4*>(gp + q.N + c * 8) : make_uint4(0, 0, 0, 0);
      }
    };
    auto activate = [&](float(&v)[16]) {  // linear
      with_act_or_none(p.act, [&](auto act) {
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
          const float2 a = act_value2<decltype(act)::value>(make_float2(v[e], v[e + 1]));
          v[e] = a.x, v[e + 1] = a.y;
        }
      });
    };
    // Values of 16 columns, as they lie in memory, added to v.
    auto add = [&](float(&v)[16], const uint4* from, bool wide) {
      const uint32_t* w = reinterpret_cast<const uint32_t*>(from);
      if (wide) {
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] += __uint_as_float(w[e]);
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] += e & 1 ? bf16_hi(w[e >> 1]) : bf16_lo(w[e >> 1]);
      }
    };
    // One row's results: 16 columns of a product or of dh, or gate and up values of 16 neurons
    // (grad: pre's 16 gate and up values of the row in `in`)
    auto finish = [&](const Product& q, int row, int col, float(&v)[16], const float(&u)[16], const uint4(&in)[kIn]) {
      if constexpr (EPI == kEpiLinear) {
        if (p.bias) add(v, in + 4, !p.bias_bf16);
        if (p.pre_out) store16(q, p.pre_out, q.N, row, col, v);
        activate(v);
        if (p.res) add(v, in, p.y32);
        if (!p.y32) {
          store16(q, q.y, q.N, row, col, v);
        } else if (row < q.M) {
          float* at = reinterpret_cast<float*>(q.y) + (size_t)row * q.N + col;
#pragma unroll
          for (int h = 0; h < 16; h += 8)
            if (col + h < q.N) {
              uint32_t w[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) w[e] = __float_as_uint(v[h + e]);
              if (p.wide32) {
                store32(at + h, w);
              } else {
                reinterpret_cast<uint4*>(at + h)[0] = make_uint4(w[0], w[1], w[2], w[3]);
                reinterpret_cast<uint4*>(at + h)[1] = make_uint4(w[4], w[5], w[6], w[7]);
              }
            }
        }
      } else if (EPI == kEpiStore) {
        store16(q, q.y, q.N, row, col, v);
      } else if (EPI == kEpiGateUp) {
        if (p.pre_out) {  // (the up half lies N columns further)
          store16(q, p.pre_out, 2 * q.N, row, col, v);
          store16(q, p.pre_out + q.N, 2 * q.N, row, col, u);
        }
        with_act(p.act, [&](auto act) {
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] = act_value<decltype(act)::value>(v[e]) * u[e];
        });
        store16(q, q.y, q.N, row, col, v);
      } else {
        float dg[16], du[16], h[16];
        const uint32_t gw[8] = {in[0].x, in[0].y, in[0].z, in[0].w, in[1].x, in[1].y, in[1].z, in[1].w};
        const uint32_t uw[8] = {in[2].x, in[2].y, in[2].z, in[2].w, in[3].x, in[3].y, in[3].z, in[3].w};
        with_act(p.act, [&](auto act) {
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float gv = e & 1 ? bf16_hi(gw[e >> 1]) : bf16_lo(gw[e >> 1]);
            const float uv = e & 1 ? bf16_hi(uw[e >> 1]) : bf16_lo(uw[e >> 1]);
            float a, da;
            act_and_grad<decltype(act)::value>(gv, a, da);
            dg[e] = v[e] * uv * da;
            du[e] = v[e] * a;
            h[e] = a * uv;
          }
        });
        store16(q, p.dpre, 2 * q.N, row, col, dg);
        store16(q, p.dpre + q.N, 2 * q.N, row, col, du);
        store16(q, q.y, q.N, row, col, h);
      }
    };
    // mx8 gate/up: one row's 32 neurons, a group
    auto finish_mx = [&](const Product& q, int row, int col, float(&h)[32], const float(&u)[32]) {
      uint32_t top = 0;
      with_act(p.act, [&](auto act) {
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          h[e] = act_value<decltype(act)::value>(h[e]) * u[e];
          top = max(top, mag_bits(h[e]));
        }
      });
      const uint32_t byte = mx_scale_byte(__uint_as_float(top));
      const float k = mx_inverse_scale(byte);
      if (row >= q.M || col >= q.N) return;
      uint32_t w[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = e4m3x4(h[4 * e] * k, h[4 * e + 1] * k, h[4 * e + 2] * k, h[4 * e + 3] * k);
      store32(p.hq + (size_t)row * q.N + col, w);
      p.hs[mx_scale_word(row, col / 128, mx_tile_cols(q.N)) + col / 32 % 4] = (uint8_t)byte;
    };

    auto release = [&](int acc) {  // an accumulator (mx8: the shared columns) is read
      tc_fence_before();
      __syncwarp();
      // relaxed: only the TMEM reads above come before it, which have completed (a release would first wait for the
      // rows stored so far, ~1 us)
      if (lane == 0)
        asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(
                         map_cta(&bar->tempty[MX ? 0 : acc], lead))
                     : "memory");
    };
    if constexpr (kStaged && EPI == kEpiStore) {
      // 64 columns at a time go through the warp's place, as bf16, to leave as 128 bytes of a row.  Against 32 bytes of
      // each of a warp's rows, a backward call (us): 41 tokens, 1256 to 11376 28.6 for 31.8; T = 387, 1976 to 7472 49 for
      // 53; T = 512, 4096 to 4096 33.9 for 35.5; T = 4096, 4096 to 16384 (long reductions) 640-665 for 640-650.  The gated block's
      // products: d = 4096, I = 16384, backward T = 16 147 for 174, T = 501 295 for 307, T = 4096 2050 for 2100, forward T = 512
      // 131 for 139; d = I = 2048, backward T = 501 39.7 for 42.3.
      uint4* const place = reinterpret_cast<uint4*>(scales + ew * kPlaceBytes);
      const int to = lane * 8 + (lane & 7);  // piece e of row `lane` at to ^ e
      const int r0 = lane >> 3, from = r0 * 8 + ((lane & 7) ^ r0);  // a thread's rows are r0 + 4 i: from + 32 i, odd i's ^ 4
      for (int lt = 0; tile_of<MULTI>(p, pair, pairs, lt, t); ++lt) {
        const int acc = lt & 1;
        const Product& q = p.q[MULTI ? t.q : 0];
        const int N = q.N, row = (2 * t.m + (int)rank) * kBM + part * 32 + r0;
        const int rows = q.M > row ? (q.M - row + 3) >> 2 : 0;  // of this thread
        uint16_t* const y = q.y + (size_t)row * N;
        if (!mbar_wait(&bar->tfull[acc], (lt >> 1) & 1, p.ctl) || aborted(bar)) {
          set_abort(bar);
          break;
        }
        tc_fence_after();
        __syncwarp();
        const uint32_t src = tmem + lanes + acc * kBN + half * 128;
#pragma unroll 1
        for (int g = 0; g < 2; ++g) {
          float v[64];
#pragma unroll
          for (int e = 0; e < 64; e += 16) tmem_ld16_async(src + g * 64 + e, v + e);
          tmem_ld_wait();
          if (g == 1) release(acc);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            place[to ^ e] = make_uint4(pack_bf16x2(v[8 * e], v[8 * e + 1]), pack_bf16x2(v[8 * e + 2], v[8 * e + 3]),
                                       pack_bf16x2(v[8 * e + 4], v[8 * e + 5]), pack_bf16x2(v[8 * e + 6], v[8 * e + 7]));
          __syncwarp();
          const int col = t.n * TN + half * 128 + g * 64 + (lane & 7) * 8;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (i < rows && col < N)
              *reinterpret_cast<uint4*>(y + col + (size_t)(4 * i) * N) = place[(from ^ (i & 1) * 4) + 32 * i];
          __syncwarp();
        }
      }
    } else if constexpr (kStaged) {
      // The sums of 32 columns at a time change hands through the warp's place in shared memory, so that a thread, which
      // reads a row of them, finishes 8 neighbouring columns (the same in every row) of every eighth row: bias, residual and
      // results then move 64 or 128 bytes of a row at a time, and a column's bias is read once.  (In the place the 16-byte
      // pieces of a row are swapped by the row: neither side finds a bank twice.)  What the next columns need is asked for
      // ahead of them, and the next tile's residual brought to L2.  All this waits more than it computes, so that sixteen
      // warps are worth a stage of the ring (whose memory their places take).  Against eight warps whose threads write their
      // own rows (us; T, in, out): 4719, 304, 15616 gelu 70 for 117, as it is 52 for 73, with an fp32 residual 133 for 160;
      // 4096, 1024, 4096 gelu and a residual 33.7 for 42.7; 16384, 1024, 4096 gelu, fp32 residual, pre 159 for 187; one
      // tile for a pair (777, 1000, 2744) 19.0 for 18.3.  Eight warps this way 93 (first), sixteen with 16 columns at a
      // time and all six stages 78.  A short reduction is bound by this epilogue (3.4-4.6 us a tile, of which ~1.6 are
      // accesses to shared memory; a tile of K = 304 multiplies for 1.4), from K = ~1000 on by the MMAs.
      const Product& q = p.q[0];
      const int M = q.M, N = q.N;
      const bool f32 = p.y32, bias_bf16 = p.bias_bf16;
      const uint8_t *res_in = static_cast<const uint8_t*>(p.res), *bias_in = static_cast<const uint8_t*>(p.bias);
      uint8_t* const y = reinterpret_cast<uint8_t*>(q.y);
      uint16_t* const pre_out = p.pre_out;
      const int size = f32 ? 4 : 2;
      float4* const place = reinterpret_cast<float4*>(scales + ew * kPlaceBytes);
      const int to = lane * 8 + (lane & 7);              // piece e of row `lane` at to ^ e
      const int r0 = lane >> 2, piece = (lane & 3) * 2;  // a thread's rows are r0 + 8 i: from + 64 i
      const int from = r0 * 8 + (piece ^ r0);            // the second piece at from ^ 1
      struct Group {  // a thread's part of 32 columns of a tile
        int rows;     // of its four rows how many there are (its 8 columns are there or not)
        size_t at;    // the first of its values in the matrix
      };
      auto row_of = [&](const Tile& t) { return (2 * t.m + (int)rank) * kBM + part * 32; };
      auto col_of = [&](const Tile& t) { return t.n * TN + half * 64; };
      auto group_of = [&](const Tile& t, int g) {
        const int row = row_of(t) + r0, col = col_of(t) + g * 32 + (lane & 3) * 8;
        return Group{col < N && row < M ? min((M - row + 7) >> 3, 4) : 0, (size_t)row * N + col};
      };
      uint4 res[8], bias[2];
      auto fetch_bias = [&](const Tile& t, int g) {
        const int col = col_of(t) + g * 32 + (lane & 3) * 8;
        if (!bias_in || col >= N) return;
        const uint4* b = reinterpret_cast<const uint4*>(bias_in + (size_t)col * (bias_bf16 ? 2 : 4));
        bias[0] = b[0];
        if (!bias_bf16) bias[1] = b[1];
      };
      auto fetch_row = [&](const Group& gr, int i, uint4* to) {
        if (!res_in || i >= gr.rows) return;
        const uint4* r = reinterpret_cast<const uint4*>(res_in + (gr.at + (size_t)(i * 8) * N) * size);
        to[0] = r[0];
        if (f32) to[1] = r[1];
      };
      auto prefetch = [&](const Tile& t) {  // the residual's 64 columns of row `lane`, by their first and last line
        const int row = row_of(t) + lane, col = col_of(t);
        if (!res_in || row >= M || col >= N) return;
        const uint8_t* r = res_in + ((size_t)row * N + col) * size;
        prefetch_l2(r);
        prefetch_l2(r + min(64, N - col) * size - 1);
      };
      Tile next;
      bool more = tile_of<MULTI>(p, pair, pairs, 0, next);
      Group ahead{};
      if (more) {
        ahead = group_of(next, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) fetch_row(ahead, i, res + 2 * i);
        prefetch(next);
      }
      for (int lt = 0; more; ++lt) {
        const int acc = lt & 1;
        t = next;
        more = tile_of<MULTI>(p, pair, pairs, lt + 1, next);
        if (more) prefetch(next);
        if (!mbar_wait(&bar->tfull[acc], (lt >> 1) & 1, p.ctl) || aborted(bar)) {
          set_abort(bar);
          break;
        }
        tc_fence_after();
        __syncwarp();
        const uint32_t src = tmem + lanes + acc * kBN + half * 64;
#pragma unroll 1
        for (int g = 0; g < 2; ++g) {
          const Group here = ahead;
          float v[32];
          tmem_ld16_async(src + g * 32, v);
          tmem_ld16_async(src + g * 32 + 16, v + 16);
          fetch_bias(t, g);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 8; ++e)
            place[to ^ e] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
          if (g == 1) release(acc);
          __syncwarp();
          ahead = g == 0 ? group_of(t, 1) : more ? group_of(next, 0) : Group{};
          const uint32_t bw[8] = {bias[0].x, bias[0].y, bias[0].z, bias[0].w, bias[1].x, bias[1].y, bias[1].z, bias[1].w};
          float2 b[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            b[e] = !bias_in    ? both(0.f)
                   : bias_bf16 ? bf16_two(bw[e])
                               : make_float2(__uint_as_float(bw[2 * e]), __uint_as_float(bw[2 * e + 1]));
          with_act_or_none(p.act, [&](auto a) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float4 lo = place[from + i * 64], hi = place[(from ^ 1) + i * 64];
              float2 x[4] = {{lo.x, lo.y}, {lo.z, lo.w}, {hi.x, hi.y}, {hi.z, hi.w}};
              const size_t at = here.at + (size_t)(i * 8) * N;
              auto packed = [&]() {
                return make_uint4(pack_bf16x2(x[0].x, x[0].y), pack_bf16x2(x[1].x, x[1].y), pack_bf16x2(x[2].x, x[2].y),
                                  pack_bf16x2(x[3].x, x[3].y));
              };
              const bool live = i < here.rows;
#pragma unroll
              for (int e = 0; e < 4; ++e) x[e] = add2(x[e], b[e]);
              if (pre_out && live) *reinterpret_cast<uint4*>(pre_out + at) = packed();
#pragma unroll
              for (int e = 0; e < 4; ++e) x[e] = act_value2<decltype(a)::value>(x[e]);
              if (res_in) {
                const uint4 l = res[2 * i], h = res[2 * i + 1];
                const uint32_t w[8] = {l.x, l.y, l.z, l.w, h.x, h.y, h.z, h.w};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  x[e] = add2(x[e], f32 ? make_float2(__uint_as_float(w[2 * e]), __uint_as_float(w[2 * e + 1]))
                                        : bf16_two(w[e]));
                fetch_row(ahead, i, res + 2 * i);
              }
              if (!live) continue;
              if (!f32) {
                *reinterpret_cast<uint4*>(y + at * 2) = packed();
              } else {
                float4* out = reinterpret_cast<float4*>(y + at * 4);
                out[0] = make_float4(x[0].x, x[0].y, x[1].x, x[1].y);
                out[1] = make_float4(x[2].x, x[2].y, x[3].x, x[3].y);
              }
            }
          });
          __syncwarp();
        }
      }
    } else if constexpr (SPLIT == 1) {
      int lt = 0;
      for (; tile_of<MULTI>(p, pair, pairs, lt, t); ++lt) {
        const Product& q = p.q[MULTI ? t.q : 0];
        const int m = t.m, n = t.n, acc = lt & 1;
        const int row = (2 * m + (int)rank) * kBM + part * 32 + lane;
        constexpr int kChunks = EPI == kEpiGateUp ? 4 : 8;  // of 16 columns (neurons), see below
        uint4 in[kIn];
        load_pre(q, row, n * TN + half * kChunks * 16, in);  // in flight while the product is waited for
        if (!mbar_wait(&bar->tfull[acc], (lt >> 1) & 1, p.ctl) || aborted(bar)) {
          set_abort(bar);
          break;
        }
        tc_fence_after();
        __syncwarp();
        const uint32_t src = tmem + lanes + acc * (MX ? kBN - kSharedCols : kBN);
        // mx8: the part with the shared columns first (the last columns of accumulator 0, the first of 1)
        const bool back = MX && acc == 0;
        const bool holds = !MX || half == (back ? 1 : 0);  // mx8: this warp reads shared columns
        if (!holds) release(acc);
        if (EPI == kEpiGateUp && MX) {
          // Two groups of 32 neurons.  The shared columns are up values (back) or gate values of both groups, so the
          // second group's are read with the first.
          auto column = [&](int i) { return half * 64 + (back ? 1 - i : i) * 32; };
          auto load = [&](float* v, int c) {
            tmem_ld16_async(src + c, v);
            tmem_ld16_async(src + c + 16, v + 16);
          };
          float g[32], u[32], next[32];
          load(g, column(0));
          load(u, 128 + column(0));
          load(next, (back ? 128 : 0) + column(1));
          tmem_ld_wait();
          if (holds) release(acc);
#pragma unroll 1
          for (int i = 0; i < 2; ++i) {
            finish_mx(q, row, n * TN + column(i), g, u);
            if (i == 0) {
              float other[32];
              load(other, (back ? 0 : 128) + column(1));
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                g[e] = back ? other[e] : next[e];
                u[e] = back ? next[e] : other[e];
              }
            }
          }
        } else {
          // 16 columns (neurons) at a time in a compact loop: straight-line code for the whole tile takes longer to
          // fetch than to run where a CTA has one tile or two
          constexpr int kShared = MX ? kSharedCols / 16 : kChunks;  // chunks after which the accumulator is released
          float v[16], u[16];
          auto load = [&](int i) {
            const int c = (half * kChunks + (back ? kChunks - 1 - i : i)) * 16;
            tmem_ld16_async(src + c, v);
            if (EPI == kEpiGateUp) tmem_ld16_async(src + 128 + c, u);
          };
          load(0);
#pragma unroll 1
          for (int i = 0; i < kChunks; ++i) {
            tmem_ld_wait();
            float x[16], y[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = v[e], y[e] = u[e];
            uint4 now[kIn];
#pragma unroll
            for (int e = 0; e < kIn; ++e) now[e] = in[e];
            if (holds && i == kShared - 1) release(acc);
            if (i + 1 < kChunks) {
              load(i + 1);
              load_pre(q, row, n * TN + (half * kChunks + i + 1) * 16, in);
            }
            finish(q, row, n * TN + (half * kChunks + (back ? kChunks - 1 - i : i)) * 16, x, y, now);
          }
        }
      }
    } else {
      // This warp's share of a pair's columns: W from a0 and W from b0 (gate/up: gate and up columns of W neurons).
      // (SPLIT == 3, of linear and its gradients: the 16 chunks of 16 columns go two or three to each of the six.)
      constexpr int W = SPLIT == 3 ? 24 : kBN / 4 / SPLIT, kSendBytes = 2 * W * 32 * 4;
      static_assert(SPLIT != 3 || EPI != kEpiGateUp, "columns of one range per warp");
      auto chunk0 = [](int o) { return o * 16 / 6; };
      auto width_of = [&](int owner) {  // columns of its share, both ranges
        return SPLIT == 3 ? (chunk0(owner * 2 + half + 1) - chunk0(owner * 2 + half)) * 16 : 2 * W;
      };
      auto a0_of = [&](int owner) {
        return SPLIT == 3           ? chunk0(owner * 2 + half) * 16
               : EPI == kEpiGateUp ? (owner * 2 + half) * W
                                   : (owner * 2 + half) * 2 * W;
      };
      auto b0_of = [&](int owner) { return a0_of(owner) + (EPI == kEpiGateUp ? kBN / 2 : W); };
      const uint32_t src = tmem + lanes;
      uint8_t* send = base;                                         // [SPLIT - 1][warp] x kSendBytes
      uint8_t* recv = base + (SPLIT - 1) * kEpiWarps * kSendBytes;  // the same, by sender
      static_assert(2 * (SPLIT - 1) * kEpiWarps * kSendBytes <= S * kStageBytes, "the exchange fits the ring");
      // Place of column c of row `lane`: 16-byte pieces of 4 columns, rows side by side.
      auto at = [&](uint8_t* buf, int c) { return reinterpret_cast<float4*>(buf + ((c >> 2) * 32 + lane) * 16); };
      bool ok = mbar_wait(&bar->tfull[0], 0, p.ctl) && !aborted(bar);
      if (lane == 0) mbar_expect_tx(&bar->recv[ew], (SPLIT - 1) * width_of(slot) * 128);
      __syncwarp();
      ok = all_of_256(ok);  // (all give up or none)
      if (ok) {
        tc_fence_after();
        // the pair's MMAs are done, so its ring's memory takes in the others' sums now
        if (warp == 2 && lane < SPLIT && lane != slot) arrive_cluster(map_cta(&bar->free[slot], 2 * lane + rank));
#pragma unroll 1
        for (int i = 1; i < SPLIT; ++i) {
          const int owner = (slot + i) % SPLIT;
          uint8_t* out = send + ((i - 1) * kEpiWarps + ew) * kSendBytes;
#pragma unroll 1
          for (int c = 0; c < width_of(owner); c += 16) {
            float v[16];
            tmem_ld16_async(src + (SPLIT == 3 || c < W ? a0_of(owner) + c : b0_of(owner) + c - W), v);
            tmem_ld_wait();
#pragma unroll
            for (int q = 0; q < 16; q += 4) *at(out, c + q) = make_float4(v[q], v[q + 1], v[q + 2], v[q + 3]);
          }
          fence_proxy_async_shared_cta();
          __syncwarp();
          if (lane == 0) {
            if (!mbar_wait(&bar->free[owner], 0, p.ctl)) {
              set_abort(bar);
            } else {
              const int by = slot < owner ? slot : slot - 1;  // this pair among the owner's senders
              const uint32_t to = (uint32_t)(2 * owner) + rank;
              copy_to_cta(map_cta(recv + (by * kEpiWarps + ew) * kSendBytes, to), out, width_of(owner) * 128,
                          map_cta(&bar->recv[ew], to));
            }
          }
          __syncwarp();
        }
        ok = mbar_wait(&bar->recv[ew], 0, p.ctl);
        if (!ok) mbar_wait(&bar->recv[ew], 0, drain_ctl(p.ctl));
        ok = __all_sync(0xffffffffu, ok);
      }
      if (!ok) {
        set_abort(bar);
      } else if (tile_of<MULTI>(p, pair, pairs, 0, t)) {
        const Product& q = p.q[0];
        const int m = t.m, n = t.n;
        const int row = (2 * m + (int)rank) * kBM + part * 32 + lane;
        // 16 columns' sums over the pairs in the order of k; place c in the exchange, TMEM column col
        auto sum16 = [&](int c, int col, float* v) {
#pragma unroll
          for (int k = 0; k < SPLIT; ++k) {
            float x[16];
            if (k == slot) {
              tmem_ld16_async(src + col, x);
              tmem_ld_wait();
            } else {
              uint8_t* in = recv + ((k < slot ? k : k - 1) * kEpiWarps + ew) * kSendBytes;
#pragma unroll
              for (int q = 0; q < 16; q += 4) {
                const float4 f = *at(in, c + q);
                x[q] = f.x, x[q + 1] = f.y, x[q + 2] = f.z, x[q + 3] = f.w;
              }
            }
#pragma unroll
            for (int q = 0; q < 16; ++q) v[q] = k == 0 ? x[q] : v[q] + x[q];
          }
        };
        const int a0 = a0_of(slot), b0 = b0_of(slot);
        if constexpr (EPI == kEpiGateUp && MX) {
          static_assert(W == 32, "a warp holds whole groups");
          float g[32], u[32];
          sum16(0, a0, g);
          sum16(16, a0 + 16, g + 16);
          sum16(32, b0, u);
          sum16(48, b0 + 16, u + 16);
          finish_mx(q, row, n * TN + a0, g, u);
        } else if (EPI == kEpiGateUp) {
          const uint4 none[kIn] = {};
#pragma unroll 1
          for (int c = 0; c < W; c += 16) {
            float g[16], u[16];
            sum16(c, a0 + c, g);
            sum16(W + c, b0 + c, u);
            finish(q, row, n * TN + a0 + c, g, u, none);
          }
        } else {
#pragma unroll 1
          for (int c = 0; c < width_of(slot); c += 16) {
            float v[16];
            uint4 in[kIn];
            load_pre(q, row, n * TN + a0 + c, in);
            sum16(c, a0 + c, v);
            finish(q, row, n * TN + a0 + c, v, v, in);
          }
        }
      }
    }
  }

  __syncthreads();
  // Leave together: the other CTA's shared memory is the target of remote
  // arrivals and of the MMAs' reads.  On the normal path every copy has landed
  // (an MMA waited for it).  After an abort, which every CTA of the cluster is
  // told, copies may be in flight: a pair's second CTA reports what its
  // producers have issued, and the first waits for both CTAs' copies block by
  // block, crediting a barrier with what never was.
  constexpr int kRoles = roles_of(MX);
  if (threadIdx.x == 0 && bar->abort_flag)
    for (uint32_t r = 0; r < 2 * SPLIT; ++r) store_cluster(map_cta(&bar->any_abort, r), 1u);
  cluster_sync();
  if (bar->any_abort) {
    if (threadIdx.x == 0 && rank == 1)
      for (int r = 0; r < kRoles; ++r) store_cluster(map_cta(&bar->issued[1][r], lead), bar->issued[1][r]);
    cluster_sync();
    if (threadIdx.x == 0 && rank == 0) {
      const DevCtl drain = drain_ctl(p.ctl);
      constexpr uint32_t bytes[3] = {kOpBytes, kOpBytes, kScaleBytes};
      int most = 0;
      for (int r = 0; r < 2 * kRoles; ++r) most = max(most, (int)bar->issued[r / kRoles][r % kRoles]);
      for (int j = max(0, most - S); j < most; ++j) {
        uint64_t* fb = &bar->full[j % S];
        uint32_t missing = 0;
        for (int r = 0; r < 2 * kRoles; ++r)
          if (j >= (int)bar->issued[r / kRoles][r % kRoles]) missing += bytes[r % kRoles];
        if (j >= (int)bar->issued[0][0]) mbar_expect_tx(fb, 2 * kTx);
        if (missing)
          asm volatile("mbarrier.complete_tx.relaxed.cluster.shared::cluster.b64 [%0], %1;" ::"r"(map_cta(fb, lead)),
                       "r"(missing)
                       : "memory");
        mbar_wait(fb, (j / S) & 1, drain);
      }
    }
    cluster_sync();
  }
  if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

// ------------------------------------------------------------------ host side
template <int EPI, bool A_MN, bool B_MN, bool MX, int SPLIT>
cudaLaunchConfig_t config(int clusters, cudaLaunchAttribute (&at)[2]) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * SPLIT * clusters);
  cfg.blockDim = dim3(threads_of(EPI, MX, SPLIT));
  cfg.dynamicSmemBytes = smem_of(EPI, MX, SPLIT);
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 2 * SPLIT;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cfg;
}

template <int EPI, bool A_MN, bool B_MN, bool MX, int SPLIT, bool MULTI = false>
cudaError_t launch(const GemmParams& p, int clusters, cudaStream_t st) {
  cudaLaunchAttribute at[2];
  cudaLaunchConfig_t cfg = config<EPI, A_MN, B_MN, MX, SPLIT>(clusters, at);
  cfg.stream = st;
  return cudaLaunchKernelEx(&cfg, ffn_gemm_kernel<EPI, A_MN, B_MN, MX, SPLIT, MULTI>, p);
}

bool aligned32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }

// A product's operands and sizes.  b_rows: rows of b (columns where it is MN-major).  Without y the sizes alone.
template <int EPI, bool A_MN, bool B_MN, bool MX>
bool set_product(const FfnEngine& e, Product& q, const void* a, const void* b, int M, int N, int K, uint64_t b_rows,
                 void* y) {
  constexpr int TN = EPI == kEpiGateUp ? kBN / 2 : kBN;
  q.M = M;
  q.N = N;
  q.K = K;
  q.a_mn = A_MN;
  q.wide = N % 16 == 0 && aligned32(y);
  q.y = static_cast<uint16_t*>(y);
  q.mt = (M + 2 * kBM - 1) / (2 * kBM);
  q.nt = (N + TN - 1) / TN;
  if ((long long)q.mt * q.nt > (1 << 28)) return false;
  q.tiles = q.mt * q.nt;
  q.blocks = (K + (MX ? 127 : 63)) / (MX ? 128 : 64);
  if (!y && EPI == kEpiStore) return true;
  if (MX) return make_code_map(e.encode, &q.a, a, K, M, 128) && make_code_map(e.encode, &q.b, b, K, b_rows, 128);
  // a K-major operand is [rows, K], an MN-major one [K, rows]
  return (A_MN ? make_bf16_map(e.encode, &q.a, a, M, K, M, 64, kBK)
               : make_bf16_map(e.encode, &q.a, a, K, M, K, kBK, kBM)) &&
         (B_MN ? make_bf16_map(e.encode, &q.b, b, b_rows, K, b_rows, 64, kBK)
               : make_bf16_map(e.encode, &q.b, b, K, b_rows, K, kBK, 128));
}

// Pairs that a tile's reduction is split over, and the time of the product, in
// k blocks: the least of rounds of tiles x time of a tile.  Measured (us for
// the two products of a forward call, all with 1, 2 or 4, against this choice
// for each): T = 128, d = 2048, I = 8192: 58.1, 50.4, 68.6 -> 34.8; T = 1024, d
// = 2048, I = 2048: 29.9, 36.2, 79.5 -> 27.1; T = 2048, d = 2048, I = 8192:
// 120.4, 223.5, 427.3 -> 120.7.
template <int EPI, bool MX>
int split_of(const FfnEngine& e, const Product& q, bool three, double* cost) {
  constexpr int kMost = MX && EPI == kEpiGateUp ? 2 : 4;  // mx8: a warp must keep whole groups of 32 neurons
  int split = 1;
  *cost = 1e30;
  for (int s = 1; s <= kMost && s <= q.blocks; s += three || s == 1 ? 1 : 2) {
    const int fit = s == 1 ? e.pairs : s == 2 ? e.pairs2 : s == 3 ? e.pairs3 : e.pairs4;  // clusters that run at a time
    if (fit < 1) break;
    const double rounds = (double)((q.tiles + fit - 1) / fit);
    const double c =
        rounds * ((q.blocks + s - 1) / s + kTileCost + (double)epilogue_cost(EPI) / s + (s > 1 ? kSplitCost : 0));
    if (c < *cost) *cost = c, split = s;
  }
  return split;
}

// Products that may be split over three pairs: linear and its gradients' (the feed-forward block's are not).
constexpr bool has_three(int epi, bool b_mn) { return epi == kEpiLinear || (epi == kEpiStore && b_mn); }

template <int EPI, bool A_MN, bool B_MN, bool MX>
cudaError_t run(const FfnEngine& e, GemmParams& p, cudaStream_t st, bool three = false) {
  p.ctl = e.ctl;
  double cost;
  const int split = split_of<EPI, MX>(e, p.q[0], three, &cost), tiles = p.q[0].tiles;
  if (split == 1) return launch<EPI, A_MN, B_MN, MX, 1>(p, tiles < e.pairs ? tiles : e.pairs, st);
  if (split == 2) return launch<EPI, A_MN, B_MN, MX, 2>(p, tiles, st);
  if constexpr (has_three(EPI, B_MN))
    if (split == 3) return launch<EPI, A_MN, B_MN, MX, 3>(p, tiles, st);
  if constexpr (!(MX && EPI == kEpiGateUp)) return launch<EPI, A_MN, B_MN, MX, 4>(p, tiles, st);
  return cudaErrorInvalidValue;
}

template <int EPI, bool A_MN, bool B_MN, bool MX, int SPLIT, bool MULTI = false>
cudaError_t prepare(int* clusters) {
  auto k = ffn_gemm_kernel<EPI, A_MN, B_MN, MX, SPLIT, MULTI>;
  cudaError_t err = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)smem_of(EPI, MX, SPLIT));
  if (err != cudaSuccess) return err;
  cudaLaunchAttribute at[2];
  cudaLaunchConfig_t cfg = config<EPI, A_MN, B_MN, MX, SPLIT>(1, at);
  cfg.numAttrs = 1;
  int n = 0;
  err = cudaOccupancyMaxActiveClusters(&n, k, &cfg);
  if (err == cudaSuccess && n < *clusters) *clusters = n;
  return err;
}
template <int EPI, bool A_MN, bool B_MN, bool MX>
cudaError_t prepare_splits(FfnEngine* e) {
  cudaError_t err = prepare<EPI, A_MN, B_MN, MX, 1>(&e->pairs);
  if (err == cudaSuccess) err = prepare<EPI, A_MN, B_MN, MX, 2>(&e->pairs2);
  if constexpr (has_three(EPI, B_MN))
    if (err == cudaSuccess) err = prepare<EPI, A_MN, B_MN, MX, 3>(&e->pairs3);
  if constexpr (!(MX && EPI == kEpiGateUp))
    if (err == cudaSuccess) err = prepare<EPI, A_MN, B_MN, MX, 4>(&e->pairs4);
  return err;
}

// The scales of rows row0, row0 + 1, ... of a matrix as a matrix of their own
// (row0 a multiple of 32 but not of 128, so that its tiles start elsewhere):
// one 4-byte word per thread.
__global__ void __launch_bounds__(256) shift_scales_kernel(const uint32_t* src, uint32_t* dst, int row0, int rows,
                                                           int tile_cols, size_t words) {
  const size_t at = (size_t)blockIdx.x * 256 + threadIdx.x;
  if (at >= words) return;
  // word `at` of dst: tile, then row % 32, then row / 32 % 4
  const size_t tile = at / 128, in = at % 128;
  const size_t row = tile / tile_cols * 128 + in % 4 * 32 + in / 4, col = tile % tile_cols;
  dst[at] = row < (size_t)rows ? src[mx_scale_word(row0 + row, col, tile_cols) / 4] : 0u;
}

}  // namespace

cudaError_t prepare_ffn_gemm(FfnEngine* e) {
  e->pairs = e->pairs2 = e->pairs3 = e->pairs4 = e->sms / 2;
  cudaError_t err = prepare_splits<kEpiGateUp, false, false, false>(e);
  if (err == cudaSuccess) err = prepare_splits<kEpiStore, false, false, false>(e);
  if (err == cudaSuccess) err = prepare_splits<kEpiGrad, false, true, false>(e);
  if (err == cudaSuccess) err = prepare_splits<kEpiStore, false, true, false>(e);
  if (err == cudaSuccess) err = prepare_splits<kEpiStore, true, true, false>(e);
  if (err == cudaSuccess) err = prepare<kEpiStore, true, true, false, 1, true>(&e->pairs);
  if (err == cudaSuccess) err = prepare_splits<kEpiLinear, false, false, false>(e);
  if (err == cudaSuccess) err = prepare_splits<kEpiGateUp, false, false, true>(e);
  if (err == cudaSuccess) err = prepare_splits<kEpiStore, false, false, true>(e);
  return err == cudaSuccess && e->pairs < 1 ? cudaErrorInvalidConfiguration : err;
}

cudaError_t launch_mx_up_scales(const FfnShape& s, const uint8_t* gate_up_s, uint8_t* up_s, cudaStream_t st) {
  const size_t words = mx_scale_bytes(s.I, s.d) / 4;
  shift_scales_kernel<<<(unsigned)((words + 255) / 256), 256, 0, st>>>(
      reinterpret_cast<const uint32_t*>(gate_up_s), reinterpret_cast<uint32_t*>(up_s), s.I, s.I, (int)mx_tile_cols(s.d),
      words);
  return cudaGetLastError();
}

cudaError_t launch_ffn_gate_up_mx(const FfnEngine& e, const FfnShape& s, const FfnForwardArgs& a, const uint8_t* up_s,
                                  uint8_t* hq, uint8_t* hs, cudaStream_t st) {
  GemmParams p{};
  p.act = s.act;
  p.hq = hq;
  p.hs = hs;
  const uint64_t tiles = (s.I + 127) / 128;
  if (!set_product<kEpiGateUp, false, false, true>(e, p.q[0], a.x, a.gate_up, s.T, s.I, s.d, 2 * (uint64_t)s.I,
                                                   nullptr) ||
      !make_scale_map(e.encode, &p.as, a.xs, s.d, (s.T + 127) / 128) ||
      !make_scale_map(e.encode, &p.bs0, a.gate_up_s, s.d, tiles) || !make_scale_map(e.encode, &p.bs1, up_s, s.d, tiles))
    return cudaErrorInvalidValue;
  return run<kEpiGateUp, false, false, true>(e, p, st);
}

cudaError_t launch_ffn_down_mx(const FfnEngine& e, const FfnShape& s, const uint8_t* hq, const uint8_t* hs,
                               const FfnForwardArgs& a, cudaStream_t st) {
  GemmParams p{};
  if (!set_product<kEpiStore, false, false, true>(e, p.q[0], hq, a.down, s.T, s.d, s.I, s.d, a.y) ||
      !make_scale_map(e.encode, &p.as, hs, s.I, (s.T + 127) / 128) ||
      !make_scale_map(e.encode, &p.bs0, a.down_s, s.I, (s.d + 127) / 128))
    return cudaErrorInvalidValue;
  p.bs1 = p.bs0;
  return run<kEpiStore, false, false, true>(e, p, st);
}

cudaError_t launch_ffn_gate_up(const FfnEngine& e, const FfnShape& s, const void* x, const void* gate_up, uint16_t* h,
                               uint16_t* pre, cudaStream_t st) {
  GemmParams p{};
  p.act = s.act;
  p.pre_out = pre;
  if (!set_product<kEpiGateUp, false, false, false>(e, p.q[0], x, gate_up, s.T, s.I, s.d, 2 * (uint64_t)s.I, h))
    return cudaErrorInvalidValue;
  if (!aligned32(pre)) p.q[0].wide = 0;
  return run<kEpiGateUp, false, false, false>(e, p, st);
}

cudaError_t launch_ffn_down(const FfnEngine& e, const FfnShape& s, const uint16_t* h, const void* down, void* y,
                            cudaStream_t st) {
  GemmParams p{};
  if (!set_product<kEpiStore, false, false, false>(e, p.q[0], h, down, s.T, s.d, s.I, s.d, y))
    return cudaErrorInvalidValue;
  return run<kEpiStore, false, false, false>(e, p, st);
}

cudaError_t launch_ffn_grad_h(const FfnEngine& e, const FfnShape& s, const FfnBackwardArgs& a, const FfnScratch& sc,
                              cudaStream_t st) {
  GemmParams p{};
  p.act = s.act;
  p.pre = a.pre;
  p.dpre = sc.dpre;
  if (!set_product<kEpiGrad, false, true, false>(e, p.q[0], a.dy, a.down, s.T, s.I, s.d, s.I, sc.h))
    return cudaErrorInvalidValue;
  return run<kEpiGrad, false, true, false>(e, p, st);
}

namespace {

// dx = dpre gate_up (K = 2I), dgate_up = dpre^T x and ddown = dy^T h (K = T).
// They do not depend on one another: they go into one launch, unless it is
// shorter to split dx's few tiles over clusters and to launch the other two
// after it, or to split each.  That is decided for all three, so that a gradient
// does not depend on which others are wanted.  d = 1024, I = 2816, a call with
// grad_h: T = 501 in one launch 45.4 us, dx first 39.3; T = 256 each by itself
// 38.6 us, dx first 33.6.  For few tokens launch_skinny_backward has done dx,
// and the others have one k block.
cudaError_t launch_grads(const FfnEngine& e, Product (&all)[3], bool few, bool three, int* launches, cudaStream_t st) {
  const bool dx_first = all[0].blocks >= all[1].blocks;  // the longer reduction

  // Times in k blocks.  One launch: at best even, at worst one light tile more, and no less than the heavy tiles' (a tile
  // after a pair's first costs less than kTileCost and its epilogue: they overlap).
  const int each = kNextTileCost, first = kTileCost + epilogue_cost(kEpiStore) - each;
  const long long weight_tiles = (long long)all[1].tiles + all[2].tiles;
  const long long heavy = dx_first ? all[0].tiles : weight_tiles, light = dx_first ? weight_tiles : all[0].tiles;
  const int ch = (dx_first ? all[0] : all[1]).blocks + each, cl = (dx_first ? all[1] : all[0]).blocks + each;
  double together = (double)(heavy * ch + light * cl) / e.pairs + cl;
  const double least = (double)((heavy + e.pairs - 1) / e.pairs) * ch;
  if (together < least) together = least;
  together += first;
  double c[3];
  int split[3];
  for (int i = 0; i < 3; ++i) {
    c[i] = 0, split[i] = 1;
    if (all[i].tiles) split[i] = split_of<kEpiStore, false>(e, all[i], three, &c[i]);
  }
  const double weights = (double)((weight_tiles + e.pairs - 1) / e.pairs) * (all[1].blocks + each) + first;
  // (these estimates are good to about a tenth, and one launch has less to go wrong)
  const double dx_apart = split[0] == 1 ? 1e30 : 1.12 * (c[0] + kLaunchCost + weights);
  // (two products that are not split gain nothing from a launch each: T = 2000, 2048 to 2048 31.8 us in one, 37.0 in two)
  const double apart = all[2].tiles         ? 1.12 * (c[0] + c[1] + c[2] + 2 * kLaunchCost)
                       : split[0] * split[1] > 1 ? 1.12 * (c[0] + c[1] + kLaunchCost)
                                                 : 1e30;
  const bool one = together <= dx_apart && together <= apart, two = !one && dx_apart <= apart;

  GemmParams p{};
  p.ctl = e.ctl;
  p.early = ch / cl;
  *launches = 0;
  if (few) {
    all[0].y = nullptr;
  } else if (two && all[0].y) {
    GemmParams dx{};
    dx.q[0] = all[0];
    const cudaError_t err = run<kEpiStore, false, true, false>(e, dx, st, three);
    if (err != cudaSuccess) return err;
    *launches = 1;
    all[0].y = nullptr;
  }
  auto add = [&](const Product& q) {
    if (q.y) p.q[p.count++] = q;
  };
  if (dx_first) add(all[0]);
  if (!dx_first) add(all[1]), add(all[2]);
  p.heavy_count = p.count;
  if (dx_first) add(all[1]), add(all[2]);
  if (!dx_first) add(all[0]);
  long long tiles = 0;
  for (int i = 0; i < p.count; ++i) {
    tiles += p.q[i].tiles;
    if (i < p.heavy_count) p.heavy_tiles = (int)tiles;
  }
  if (tiles > (1 << 28)) return cudaErrorInvalidValue;
  const int pairs = tiles < e.pairs ? (int)tiles : e.pairs;
  if (!p.count) return cudaSuccess;
  if (few || one || two) {
    ++*launches;
    if (p.count > 1) return launch<kEpiStore, true, true, false, 1, true>(p, pairs, st);
    return p.q[0].a_mn ? launch<kEpiStore, true, true, false, 1>(p, pairs, st)
                       : launch<kEpiStore, false, true, false, 1>(p, pairs, st);
  }
  *launches += p.count;
  cudaError_t err = cudaSuccess;
  for (int i = 0; i < p.count && err == cudaSuccess; ++i) {
    GemmParams one{};
    one.q[0] = p.q[i];
    err = one.q[0].a_mn ? run<kEpiStore, true, true, false>(e, one, st, three)
                        : run<kEpiStore, false, true, false>(e, one, st, three);
  }
  return err;
}

}  // namespace

cudaError_t launch_ffn_grads(const FfnEngine& e, const FfnShape& s, const FfnBackwardArgs& a, const FfnScratch& sc,
                             int* launches, cudaStream_t st) {
  Product all[3] = {};  // dx, dgate_up, ddown
  if (!set_product<kEpiStore, false, true, false>(e, all[0], sc.dpre, a.gate_up, s.T, s.d, 2 * s.I, s.d, a.dx) ||
      !set_product<kEpiStore, true, true, false>(e, all[1], sc.dpre, a.x, 2 * s.I, s.d, s.T, s.d, a.dgate_up) ||
      !set_product<kEpiStore, true, true, false>(e, all[2], a.dy, sc.h, s.d, s.I, s.T, s.I, a.ddown))
    return cudaErrorInvalidValue;
  return launch_grads(e, all, few_tokens(s), false, launches, st);
}

cudaError_t launch_linear_grads(const FfnEngine& e, const LinearShape& s, const uint16_t* dpre, const void* x,
                                const void* w, void* dx, void* dw, int* launches, cudaStream_t st) {
  Product all[3] = {};  // dx, dw
  if (!set_product<kEpiStore, false, true, false>(e, all[0], dpre, w, s.T, s.k, s.n, s.k, dx) ||
      !set_product<kEpiStore, true, true, false>(e, all[1], dpre, x, s.n, s.k, s.T, s.k, dw))
    return cudaErrorInvalidValue;
  return launch_grads(e, all, few_tokens(s, s.k), true, launches, st);
}

cudaError_t launch_linear_tiles(const FfnEngine& e, const LinearShape& s, const LinearForwardArgs& a, cudaStream_t st) {
  GemmParams p{};
  p.act = s.act;
  p.pre_out = a.pre;
  p.bias = a.bias;
  p.res = a.res;
  p.bias_bf16 = a.bias_dtype == MOE_BF16;
  p.y32 = a.y_dtype == MOE_F32;
  p.wide32 = aligned32(a.y);
  if (!set_product<kEpiLinear, false, false, false>(e, p.q[0], a.x, a.w, s.T, s.n, s.k, s.n, a.y))
    return cudaErrorInvalidValue;
  if (!aligned32(a.pre)) p.q[0].wide = 0;
  return run<kEpiLinear, false, false, false>(e, p, st, true);
}

}  // namespace moe
