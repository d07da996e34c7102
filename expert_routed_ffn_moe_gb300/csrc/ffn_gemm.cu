// The gated feed-forward block's matrix products on the 5th-generation tensor
// cores, for the forward and the backward pass.
//
//   gate_up   [g | u] = x gate_up^T; h = act(g) * u        (x, weights K-major)
//   down      y = h down^T
//   grad_h    dh = dy down; dpre = [dh u act'(g) | dh act(g)]; h = act(g) * u
//   dx        dx = dpre gate_up
//   dgate_up  dpre^T x
//   ddown     dy^T h
//
// One persistent kernel.  A pair of CTAs on neighbouring SMs (a cluster of two)
// computes a 256 x 256 tile with tcgen05.mma.cta_group::2: each CTA loads its
// own 128 rows of A and half of B's 256 rows, so a 64-deep k block costs each
// SM 32 KB of shared-memory fill for 256 cycles of MMA (a lone CTA's 128 x 256
// tile takes 48 KB for the same work).  Per CTA 11 warps (12 for mx8):
//   warps 0, 10, 11  TMA producers (one thread each) of a ring of k blocks,
//              128-byte swizzle: A, B, and mx8's scales.  One thread alone takes
//              longer for all of a k block's copies than its MMAs do;
//   warp 1     allocates all 512 TMEM columns: two fp32 accumulators of 256
//              columns; in the pair's first CTA one thread issues the MMAs;
//   warps 2-9  epilogue: two warps for each quarter of the TMEM lanes, each
//              taking one half of the columns, through a swizzled staging tile
//              per warp and TMA stores (which clip ragged edges).
// The epilogue of tile i overlaps the main loop of tile i + 1.  In the gate/up
// product B's first half holds gate rows and the second half the up rows of the
// same 128 neurons, so the activation finishes in the accumulator's columns.
//
// A product with fewer tiles than pairs splits the reduction over 2 or 4 pairs
// of one cluster (SPLIT).  Each pair ends with fp32 sums of the whole tile; the
// columns are divided among the pairs, every CTA sends its sums of the others'
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
// B's.  They take TMEM columns, so the two accumulators there share 32 columns:
// the epilogue reads those first and the next tile's MMAs may then start.  h is
// rounded to mx8 in the epilogue, where a thread holds a whole group of 32.
//
// Every wait is bounded; on expiry the kernel drains what it has in flight,
// frees TMEM and returns (see the end of the kernel).
#include "ffn_internal.h"

namespace moe {
namespace {

constexpr int kBM = 128;                    // rows of A per CTA
constexpr int kBN = 256;                    // accumulator columns
constexpr int kRowBytes = 128;              // a k block: 64 bf16 or 128 e4m3 values
constexpr int kBK = 64;                     // k block of bf16
constexpr int kOpBytes = 128 * kRowBytes;   // one operand's half tile: 16 KB
constexpr int kStageBytes = 2 * kOpBytes;   // per CTA
constexpr int kEpiWarps = 8;
constexpr int kBWarp = 2 + kEpiWarps, kScaleWarp = kBWarp + 1;  // producers of B and of the scales (A: warp 0)
constexpr int threads_of(bool mx) { return (mx ? kScaleWarp + 1 : kBWarp + 1) * 32; }
constexpr int kStoreBytes = 32 * 128;       // staging tile: 32 rows x 64 bf16
constexpr int kScaleBytes = 3 * 512;        // mx8 scales of a k block: A's 128 rows, B's 2 x 128
constexpr int kSharedCols = 32;             // mx8: accumulator columns that both tiles use
constexpr uint32_t kScaleCol = 2 * kBN - kSharedCols;  // mx8: TMEM columns of two k blocks' scales, 16 each
constexpr int kTileCost = 10, kSplitCost = 6; // of a tile besides its k blocks, in k blocks (~0.27 us), see run()
constexpr int kGroupM = 8;                  // m-tiles that share a sweep over n (L2 reuse)

enum { kEpiStore, kEpiGateUp, kEpiGrad };

struct GemmParams {
  CUtensorMap a, b;                // operands
  CUtensorMap out;                 // bf16 result: y / dx / dW, or h
  CUtensorMap out_g, out_u;        // the halves of pre (gate/up) or of dpre (grad)
  CUtensorMap as, bs0, bs1;        // mx8 scales: of A, and of the two 128-row halves of B
  uint8_t *hq, *hs;                // mx8 gate/up: codes and scales of h
  const uint16_t* pre;             // grad: [M, 2N] pre-activations
  uint16_t *y, *pre_out, *dpre;    // SPLIT: the result (or h), pre and dpre by address
  int M, N, K;                     // N: columns of the result (gate/up: neurons)
  int act;
  int store_pre;
  DevCtl ctl;
};

constexpr int stages_of(int epi, bool mx, int split = 1) { return split > 1 || (epi == kEpiStore && !mx) ? 6 : 5; }
constexpr int stage_bytes(bool mx) { return kStageBytes + (mx ? kScaleBytes : 0); }
// staging tiles per epilogue warp
constexpr int buffers_of(int epi, bool mx, int split = 1) { return split > 1 ? 0 : epi == kEpiStore ? 1 : (mx ? 0 : 2); }

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
  uint32_t issued[2][3];  // k blocks loaded by each CTA's producers of A, B and scales (first CTA: both's)
  uint32_t any_abort;     // some CTA of the cluster has given up
};

constexpr size_t smem_of(int epi, bool mx, int split = 1) {
  return 1024 + (size_t)stages_of(epi, mx, split) * stage_bytes(mx) +
         (size_t)kEpiWarps * buffers_of(epi, mx, split) * kStoreBytes + sizeof(Bars);
}
static_assert(smem_of(kEpiStore, false) <= 227 * 1024 && smem_of(kEpiGateUp, false) <= 227 * 1024 &&
                  smem_of(kEpiStore, true) <= 227 * 1024 && smem_of(kEpiGateUp, true) <= 227 * 1024 &&
                  smem_of(kEpiStore, true, 4) <= 227 * 1024,
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
MOE_DEV void tma_store(const CUtensorMap* m, int x, int y, const void* src) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                   reinterpret_cast<uint64_t>(m)),
               "r"(x), "r"(y), "r"(smem_u32(src))
               : "memory");
}
MOE_DEV void tma_store_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
template <int N>
MOE_DEV void tma_store_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
// Shared-memory matrix descriptor of an MN-major bf16 operand, 128-byte swizzle:
// each k is a 128-byte row of 64 elements along m (or n), 8 k rows make a
// 1024-byte atom; the next 64 elements along m lie `64 k rows` further.
MOE_DEV uint64_t desc_mn(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3ffffu) >> 4);
  d |= static_cast<uint64_t>((kBK * 128) >> 4) << 16;  // leading: from 64 elements of m to the next 64
  d |= static_cast<uint64_t>(1024 >> 4) << 32;         // stride: from 8 k rows to the next 8
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}
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

// Tile t of the sweep: kGroupM m-tiles at a time, all n for each group.
MOE_DEV void tile_of(int t, int mt, int nt, int& m, int& n) {
  const int per = kGroupM * nt, g = t / per, r = t - g * per;
  const int gm = min(kGroupM, mt - g * kGroupM);
  m = g * kGroupM + r % gm;
  n = r / gm;
}

// 16 bytes (8 bf16) into a swizzled staging tile: row `lane`, 16-byte column c.
MOE_DEV void stage16(uint8_t* tile, int lane, int c, uint4 v) {
  *reinterpret_cast<uint4*>(tile + lane * 128 + ((c ^ (lane & 7)) << 4)) = v;
}

template <int EPI, bool A_MN, bool B_MN, bool MX, int SPLIT>
__global__ void __launch_bounds__(threads_of(MX), 1)
    ffn_gemm_kernel(const __grid_constant__ GemmParams p) {
  constexpr int S = stages_of(EPI, MX, SPLIT), NB = buffers_of(EPI, MX, SPLIT);
  constexpr uint32_t kTx = stage_bytes(MX);        // bytes per CTA and k block
  constexpr int kDepth = MX ? kRowBytes : kBK;     // values of k per block
  static_assert(!MX || (!A_MN && !B_MN && EPI != kEpiGrad), "mx8: forward products only");
  constexpr int TN = EPI == kEpiGateUp ? kBN / 2 : kBN;  // result columns per tile
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* staging = base + S * kStageBytes;  // (the scales follow the staging tiles)
  uint8_t* scales = staging + kEpiWarps * NB * kStoreBytes;
  Bars* bar = reinterpret_cast<Bars*>(scales + (MX ? S * kScaleBytes : 0));

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t crank = cluster_rank(), rank = crank & 1, lead = crank & ~1u;  // rank in the pair, its first CTA
  const int slot = SPLIT > 1 ? (int)crank >> 1 : 0;                             // the pair's part of the reduction
  const int pair = blockIdx.x / (2 * SPLIT), pairs = gridDim.x / (2 * SPLIT);   // (SPLIT: a cluster has one tile)
  const int mt = (p.M + 2 * kBM - 1) / (2 * kBM), nt = (p.N + TN - 1) / TN, tiles = mt * nt;
  const int blocks = (p.K + kDepth - 1) / kDepth;
  const int kb0 = slot * blocks / SPLIT, kb1 = (slot + 1) * blocks / SPLIT;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 6; ++i) {
      mbar_init(&bar->full[i], 1);
      mbar_init(&bar->empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar->tfull[i], 1);
      mbar_init(&bar->tempty[i], 2 * kEpiWarps);
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
      const int role = warp == 0 ? 0 : warp - kBWarp + 1;  // A, B, scales
      tma_prefetch_desc(role == 0 ? &p.a : role == 1 ? &p.b : &p.as);
      bool ok = true;
      int issued = 0;
      for (int t = pair; t < tiles && ok; t += pairs) {
        int m, n;
        tile_of(t, mt, nt, m, n);
        const int arow = (2 * m + (int)rank) * kBM;
        // B's half: gate rows in the first CTA, up rows in the second
        const int brow = EPI == kEpiGateUp ? n * TN + (int)rank * p.N : n * TN + (int)rank * 128;
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
          const int k = kb * kDepth;
          if (role == 0) {
            if (rank == 0) mbar_expect_tx(&bar->full[st], 2 * kTx);  // everything, both CTAs'
            if (A_MN) {
              tma_load_pair(a, &p.a, arow, k, fb);
              tma_load_pair(a + kOpBytes / 2, &p.a, arow + 64, k, fb);
            } else {
              tma_load_pair(a, &p.a, k, arow, fb);
            }
          } else if (role == 1) {
            if (B_MN) {
              tma_load_pair(b, &p.b, brow, k, fb);
              tma_load_pair(b + kOpBytes / 2, &p.b, brow + 64, k, fb);
            } else {
              tma_load_pair(b, &p.b, k, brow, fb);
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
    if (rank == 0 && lane == 0) {
      constexpr uint32_t idesc = umma_idesc_bf16(2 * kBM, kBN) | (A_MN ? 1u << 15 : 0u) | (B_MN ? 1u << 16 : 0u);
      const uint16_t both = (uint16_t)(3u << lead);  // the pair's CTAs in the cluster
      int it = 0, lt = 0;
      bool ok = true, ready = false;
      if (p.ctl.stall && !mbar_wait(&bar->mma_done, 0, p.ctl)) {  // test hook: nothing arrives there before the end
        set_abort(bar);
        ok = false;
      }
      for (int t = pair; t < tiles && ok; t += pairs, ++lt) {
        const int acc = lt & 1;
        // bf16: the accumulator was read two tiles ago; mx8: the tile before has left the shared columns (which its
        // epilogue warps reach only after the tile before that)
        const bool free = MX ? lt == 0 || mbar_wait(&bar->tempty[0], (lt - 1) & 1, p.ctl)
                             : mbar_wait(&bar->tempty[acc], ((lt >> 1) & 1) ^ 1, p.ctl);
        if (!free || aborted(bar)) {
          set_abort(bar);
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem + acc * (MX ? kBN - kSharedCols : kBN);
        for (int kb = kb0; kb < kb1; ++kb, ++it) {
          const int st = it % S;
          if (!ready && (!mbar_wait(&bar->full[st], (it / S) & 1, p.ctl) || aborted(bar))) {
            set_abort(bar);
            ok = false;
            break;
          }
          // asked for before this block's MMAs: a load from shared memory queues behind their operand reads
          ready = mbar_test(&bar->full[(it + 1) % S], ((it + 1) / S) & 1);
          tc_fence_after();
          const uint32_t a = smem_u32(base + st * kStageBytes), b = a + kOpBytes;
          const uint64_t da = A_MN ? desc_mn(a) : umma_desc_sw128(a), db = B_MN ? desc_mn(b) : umma_desc_sw128(b);
          // 16 k: 32 bytes along a K-major row, 16 rows of 128 bytes of an MN-major tile
          constexpr uint64_t sa = A_MN ? 128 : 2, sb = B_MN ? 128 : 2;
          if (MX) {
            const uint32_t sc = smem_u32(scales + st * kScaleBytes), ts = tmem + kScaleCol + (it & 1) * 16;
#pragma unroll
            for (int j = 0; j < 3; ++j) copy_scales_pair(ts + 4 * j, sc + 512 * j);
#pragma unroll
            for (int j = 0; j < 4; ++j)
              mma_pair_mx(d, da + j * 2, db + j * 2, umma_idesc_mx(2 * kBM, kBN, j), ts, ts + 4, kb != kb0 || j != 0);
          } else {
#pragma unroll
            for (int j = 0; j < kBK / 16; ++j) mma_pair(d, da + j * sa, db + j * sb, idesc, kb != kb0 || j != 0);
          }
          commit_pair(&bar->empty[st], both);
        }
        if (ok) commit_pair(&bar->tfull[acc], both);
      }
      // the MMAs issued so far are done before TMEM is freed and shared memory left
      asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                       smem_u32(&bar->mma_done))
                   : "memory");
      mbar_wait(&bar->mma_done, 0, p.ctl);
    }
  } else if (SPLIT > 1) {
    // This warp's share of a pair's columns: W from a0 and W from b0 (gate/up: gate and up columns of W neurons).
    constexpr int W = kBN / 4 / SPLIT, kSendBytes = 2 * W * 32 * 4;
    const int ew = warp - 2, part = warp & 3, half = ew >> 2;
    auto a0_of = [&](int owner) { return EPI == kEpiGateUp ? (owner * 2 + half) * W : (owner * 2 + half) * 2 * W; };
    auto b0_of = [&](int owner) { return a0_of(owner) + (EPI == kEpiGateUp ? kBN / 2 : W); };
    const uint32_t src = tmem + ((uint32_t)(part * 32) << 16);
    uint8_t* send = base;                                            // [SPLIT - 1][warp] x kSendBytes
    uint8_t* recv = base + (SPLIT - 1) * kEpiWarps * kSendBytes;     // the same, by sender
    static_assert(2 * (SPLIT - 1) * kEpiWarps * kSendBytes <= S * kStageBytes, "the exchange fits the ring");
    // Place of column c of row `lane`: 16-byte pieces of 4 columns, rows side by side.
    auto at = [&](uint8_t* buf, int c) { return reinterpret_cast<float4*>(buf + ((c >> 2) * 32 + lane) * 16); };
    bool ok = mbar_wait(&bar->tfull[0], 0, p.ctl) && !aborted(bar);
    if (lane == 0) mbar_expect_tx(&bar->recv[ew], (SPLIT - 1) * kSendBytes);
    ok = all_of_256(ok);  // (all give up or none)
    if (ok) {
      tc_fence_after();
      // the pair's MMAs are done, so its ring's memory takes in the others' sums now
      if (warp == 2 && lane < SPLIT && lane != slot) arrive_cluster(map_cta(&bar->free[slot], 2 * lane + rank));
#pragma unroll 1
      for (int i = 1; i < SPLIT; ++i) {
        const int owner = (slot + i) % SPLIT;
        uint8_t* out = send + ((i - 1) * kEpiWarps + ew) * kSendBytes;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int c = 0; c < W; c += 16) {
            float v[16];
            tmem_ld16_async(src + (h ? b0_of(owner) : a0_of(owner)) + c, v);
            tmem_ld_wait();
#pragma unroll
            for (int q = 0; q < 16; q += 4) *at(out, h * W + c + q) = make_float4(v[q], v[q + 1], v[q + 2], v[q + 3]);
          }
        }
        fence_proxy_async_shared_cta();
        __syncwarp();
        if (lane == 0) {
          if (!mbar_wait(&bar->free[owner], 0, p.ctl)) {
            set_abort(bar);
          } else {
            const int by = slot < owner ? slot : slot - 1;  // this pair among the owner's senders
            const uint32_t to = (uint32_t)(2 * owner) + rank;
            copy_to_cta(map_cta(recv + (by * kEpiWarps + ew) * kSendBytes, to), out, kSendBytes,
                        map_cta(&bar->recv[ew], to));
          }
        }
      }
      ok = mbar_wait(&bar->recv[ew], 0, p.ctl);
      if (!ok) {
        DevCtl drain = p.ctl;
        drain.spin_limit = 1000000000LL;
        mbar_wait(&bar->recv[ew], 0, drain);
      }
      ok = __all_sync(0xffffffffu, ok);
    }
    if (!ok) {
      set_abort(bar);
    } else if (pair < tiles) {
      int m, n;
      tile_of(pair, mt, nt, m, n);
      const int row = (2 * m + (int)rank) * kBM + part * 32 + lane;
      constexpr int kPer = 16;  // columns of a (and of b) at a time
      uint32_t top = 0;         // mx8: the group's largest magnitude, and its values
      float hv[W];
#pragma unroll
      for (int c = 0; c < W; c += kPer) {
        float a[kPer], b[kPer];
#pragma unroll
        for (int k = 0; k < SPLIT; ++k) {  // in the order of k
          float x[kPer], y[kPer];
          if (k == slot) {
            tmem_ld16_async(src + a0_of(slot) + c, x);
            tmem_ld16_async(src + b0_of(slot) + c, y);
            tmem_ld_wait();
          } else {
            uint8_t* in = recv + ((k < slot ? k : k - 1) * kEpiWarps + ew) * kSendBytes;
#pragma unroll
            for (int q = 0; q < kPer; q += 4) {
              const float4 f = *at(in, c + q), g = *at(in, W + c + q);
              x[q] = f.x, x[q + 1] = f.y, x[q + 2] = f.z, x[q + 3] = f.w;
              y[q] = g.x, y[q + 1] = g.y, y[q + 2] = g.z, y[q + 3] = g.w;
            }
          }
#pragma unroll
          for (int q = 0; q < kPer; ++q) {
            a[q] = k == 0 ? x[q] : a[q] + x[q];
            b[q] = k == 0 ? y[q] : b[q] + y[q];
          }
        }
        auto store = [&](uint16_t* to, int pitch, int col, const float(&v)[kPer]) {
#pragma unroll
          for (int q = 0; q < kPer; q += 8)
            if (row < p.M && col + q < p.N)
              *reinterpret_cast<uint4*>(to + (size_t)row * pitch + col + q) =
                  make_uint4(pack_bf16x2(v[q], v[q + 1]), pack_bf16x2(v[q + 2], v[q + 3]),
                             pack_bf16x2(v[q + 4], v[q + 5]), pack_bf16x2(v[q + 6], v[q + 7]));
        };
        if (EPI == kEpiStore) {
          store(p.y, p.N, n * TN + a0_of(slot) + c, a);
          store(p.y, p.N, n * TN + b0_of(slot) + c, b);
        } else if (EPI == kEpiGateUp) {
          const int col = n * TN + a0_of(slot) + c;
          if (!MX && p.store_pre) {
            store(p.pre_out, 2 * p.N, col, a);
            // (the up half starts N columns further: pointer moved, column bound the same)
            store(p.pre_out + p.N, 2 * p.N, col, b);
          }
#pragma unroll
          for (int q = 0; q < kPer; ++q) a[q] = act_value(a[q], p.act) * b[q];
          if (!MX) {
            store(p.y, p.N, col, a);
          } else {  // W = 32: one group of 32 neurons, its second half follows
            static_assert(SPLIT == 1 || !MX || EPI != kEpiGateUp || W == 32, "a warp holds whole groups");
#pragma unroll
            for (int q = 0; q < kPer; ++q) {
              top = max(top, mag_bits(a[q]));
              hv[(c + q) % W] = a[q];
            }
          }
        } else {
          auto grads = [&](int col, const float(&dh)[kPer]) {
            float g[kPer], u[kPer], h[kPer];
#pragma unroll
            for (int q = 0; q < kPer; q += 8) {
              const bool in = row < p.M && col + q < p.N;
              const uint16_t* gp = p.pre + (size_t)row * 2 * p.N + col + q;
              const uint4 g4 = in ? *reinterpret_cast<const uint4*>(gp) : make_uint4(0, 0, 0, 0);
              const uint4 u4 = in ? *reinterpret_cast<const uint4*>(gp + p.N) : make_uint4(0, 0, 0, 0);
              const uint32_t gw[4] = {g4.x, g4.y, g4.z, g4.w}, uw[4] = {u4.x, u4.y, u4.z, u4.w};
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float gv = e & 1 ? bf16_hi(gw[e >> 1]) : bf16_lo(gw[e >> 1]);
                const float uv = e & 1 ? bf16_hi(uw[e >> 1]) : bf16_lo(uw[e >> 1]);
                float act, da;
                act_and_grad(gv, p.act, act, da);
                g[q + e] = dh[q + e] * uv * da;
                u[q + e] = dh[q + e] * act;
                h[q + e] = act * uv;
              }
            }
            store(p.dpre, 2 * p.N, col, g);
            store(p.dpre + p.N, 2 * p.N, col, u);
            store(p.y, p.N, col, h);
          };
          grads(n * TN + a0_of(slot) + c, a);
          grads(n * TN + b0_of(slot) + c, b);
        }
      }
      if (EPI == kEpiGateUp && MX) {
        const int col = n * TN + a0_of(slot);
        if (row < p.M && col < p.N) {
          const uint32_t byte = mx_scale_byte(__uint_as_float(top));
          const float k = mx_inverse_scale(byte);
          uint32_t w[8];
#pragma unroll
          for (int q = 0; q < 32; q += 4) {
            w[q >> 2] = e4m3x4(hv[q % W] * k, hv[(q + 1) % W] * k, hv[(q + 2) % W] * k, hv[(q + 3) % W] * k);
          }
          uint4* to = reinterpret_cast<uint4*>(p.hq + (size_t)row * p.N + col);
          to[0] = make_uint4(w[0], w[1], w[2], w[3]);
          to[1] = make_uint4(w[4], w[5], w[6], w[7]);
          p.hs[mx_scale_word(row, col / 128, mx_tile_cols(p.N)) + col / 32 % 4] = (uint8_t)byte;
        }
      }
    }
  } else {
    const int ew = warp - 2, part = warp & 3, half = ew >> 2;
    uint8_t* tile0 = staging + ew * NB * kStoreBytes;
    const uint32_t lanes = (uint32_t)(part * 32) << 16;
    int lt = 0, nbuf = 0;
    // a staging tile that no store reads any more
    auto next_tile = [&]() {
      if (lane == 0) tma_store_wait_read<(NB > 1 ? NB - 1 : 0)>();
      __syncwarp();
      return tile0 + (NB > 1 ? (nbuf++ % NB) * kStoreBytes : 0);
    };
    auto put_tile = [&](const CUtensorMap* map, const uint8_t* tile, int x, int y) {
      fence_proxy_async_shared_cta();
      __syncwarp();
      if (lane == 0) {
        if (x < p.N && y < p.M) tma_store(map, x, y, tile);
        tma_store_commit();  // also without a store, so that groups and staging tiles stay in step
      }
    };
    for (int t = pair; t < tiles; t += pairs, ++lt) {
      int m, n;
      tile_of(t, mt, nt, m, n);
      const int acc = lt & 1;
      const int y = (2 * m + (int)rank) * kBM + part * 32;
      if (!mbar_wait(&bar->tfull[acc], (lt >> 1) & 1, p.ctl) || aborted(bar)) {
        set_abort(bar);
        break;
      }
      tc_fence_after();
      __syncwarp();
      const uint32_t src = tmem + lanes + acc * (MX ? kBN - kSharedCols : kBN);
      // mx8: the part with the shared columns first (the last columns of accumulator 0, the first of 1)
      const int first = MX && acc == 0 ? 1 : 0;
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_cluster(map_cta(&bar->tempty[MX ? 0 : acc], lead));
      };
      if (EPI == kEpiStore) {
#pragma unroll 1
        for (int i = 0; i < 2; ++i) {  // two boxes of 64 columns
          const int c = i ^ first;
          uint32_t r[2][32];
          tmem_ld32_async(src + half * 128 + c * 64, r[0]);
          tmem_ld32_async(src + half * 128 + c * 64 + 32, r[1]);
          uint8_t* tile = next_tile();
          tmem_ld_wait();
          if (i == (MX ? 0 : 1)) release();
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              w[i] = pack_bf16x2(__uint_as_float(r[q >> 2][(q & 3) * 8 + 2 * i]),
                                 __uint_as_float(r[q >> 2][(q & 3) * 8 + 2 * i + 1]));
            stage16(tile, lane, q, make_uint4(w[0], w[1], w[2], w[3]));
          }
          put_tile(&p.out, tile, n * TN + half * 128 + c * 64, y);
        }
      } else if (EPI == kEpiGateUp && MX) {
        const int row = y + lane;
        uint32_t bytes = 0;  // the scales of this thread's two groups
#pragma unroll 1
        for (int i = 0; i < 2; ++i) {
          const int c = i ^ first, x = n * TN + half * 64 + c * 32;
          uint32_t g[32], u[32];
          tmem_ld32_async(src + half * 64 + c * 32, g);
          tmem_ld32_async(src + 128 + half * 64 + c * 32, u);
          tmem_ld_wait();
          if (i == 0) release();
          uint32_t top = 0;
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            g[e] = __float_as_uint(act_value(__uint_as_float(g[e]), p.act) * __uint_as_float(u[e]));
            top = max(top, g[e] & 0x7fffffffu);
          }
          const uint32_t byte = mx_scale_byte(__uint_as_float(top));
          const float k = mx_inverse_scale(byte);
          bytes |= byte << (8 * c);
          if (row < p.M && x < p.N) {
            uint4* q = reinterpret_cast<uint4*>(p.hq + (size_t)row * p.N + x);
#pragma unroll
            for (int o = 0; o < 2; ++o) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const uint32_t* v = &g[o * 16 + e * 4];
                w[e] = e4m3x4(__uint_as_float(v[0]) * k, __uint_as_float(v[1]) * k, __uint_as_float(v[2]) * k,
                              __uint_as_float(v[3]) * k);
              }
              q[o] = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
        }
        const int x = n * TN + half * 64;
        if (row < p.M && x < p.N) {  // the second group may lie past the last column: its byte stays 0
          if (x + 32 >= p.N) bytes &= 0xffu;
          *reinterpret_cast<uint16_t*>(p.hs + mx_scale_word(row, x / 128, mx_tile_cols(p.N)) + half * 2) =
              (uint16_t)bytes;
        }
      } else if (EPI == kEpiGateUp) {
        const int x = n * TN + half * 64;
        auto stage_all = [&](const CUtensorMap* map, auto&& value) {
          uint8_t* tile = next_tile();
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t g[32], u[32];
            tmem_ld32_async(src + half * 64 + c * 32, g);
            tmem_ld32_async(src + 128 + half * 64 + c * 32, u);
            tmem_ld_wait();
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint32_t w[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int e = q * 8 + 2 * i;
                w[i] = pack_bf16x2(value(__uint_as_float(g[e]), __uint_as_float(u[e])),
                                   value(__uint_as_float(g[e + 1]), __uint_as_float(u[e + 1])));
              }
              stage16(tile, lane, c * 4 + q, make_uint4(w[0], w[1], w[2], w[3]));
            }
          }
          put_tile(map, tile, x, y);
        };
        if (p.store_pre) {
          stage_all(&p.out_g, [](float g, float) { return g; });
          stage_all(&p.out_u, [](float, float u) { return u; });
        }
        const int act = p.act;
        stage_all(&p.out, [act](float g, float u) { return act_value(g, act) * u; });
        release();
      } else {
        // gradients of 128 neurons: dh in the accumulator, g and u from memory
#pragma unroll 1
        for (int c = 0; c < 2; ++c) {
          const int x = n * TN + half * 128 + c * 64;
          const int row = y + lane;
          uint32_t dg[32], du[32], hh[32];  // bf16 pairs
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            uint32_t r[32];
            tmem_ld32_async(src + half * 128 + c * 64 + q * 32, r);
            uint4 g4[4], u4[4];
            const uint16_t* gp = p.pre + (size_t)row * 2 * p.N + x + q * 32;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const bool in = row < p.M && x + q * 32 + i * 8 < p.N;
              g4[i] = in ? *reinterpret_cast<const uint4*>(gp + i * 8) : make_uint4(0, 0, 0, 0);
              u4[i] = in ? *reinterpret_cast<const uint4*>(gp + p.N + i * 8) : make_uint4(0, 0, 0, 0);
            }
            tmem_ld_wait();
            if (c == 1 && q == 1) release();
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const uint4 gv = g4[i >> 2], uv = u4[i >> 2];
              const uint32_t gw = (i & 3) == 0 ? gv.x : (i & 3) == 1 ? gv.y : (i & 3) == 2 ? gv.z : gv.w;
              const uint32_t uw = (i & 3) == 0 ? uv.x : (i & 3) == 1 ? uv.y : (i & 3) == 2 ? uv.z : uv.w;
              float a0, d0, a1, d1;
              act_and_grad(bf16_lo(gw), p.act, a0, d0);
              act_and_grad(bf16_hi(gw), p.act, a1, d1);
              const float h0 = __uint_as_float(r[2 * i]), h1 = __uint_as_float(r[2 * i + 1]);
              const float u0 = bf16_lo(uw), u1 = bf16_hi(uw);
              dg[q * 16 + i] = pack_bf16x2(h0 * u0 * d0, h1 * u1 * d1);
              du[q * 16 + i] = pack_bf16x2(h0 * a0, h1 * a1);
              hh[q * 16 + i] = pack_bf16x2(a0 * u0, a1 * u1);
            }
          }
          auto put = [&](const CUtensorMap* map, const uint32_t(&v)[32]) {
            uint8_t* tile = next_tile();
#pragma unroll
            for (int q = 0; q < 8; ++q)
              stage16(tile, lane, q, make_uint4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]));
            put_tile(map, tile, x, y);
          };
          put(&p.out_g, dg);
          put(&p.out_u, du);
          put(&p.out, hh);
        }
      }
    }
    if (lane == 0) tma_store_wait_read<0>();
  }

  __syncthreads();
  // Leave together: the other CTA's shared memory is the target of remote
  // arrivals and of the MMAs' reads.  On the normal path every copy has landed
  // (an MMA waited for it).  After an abort, which every CTA of the cluster is
  // told, copies may be in flight: a pair's second CTA reports what its
  // producers have issued, and the first waits for both CTAs' copies block by
  // block, crediting a barrier with what never was.
  constexpr int kRoles = MX ? 3 : 2;
  if (threadIdx.x == 0 && bar->abort_flag)
    for (uint32_t r = 0; r < 2 * SPLIT; ++r) store_cluster(map_cta(&bar->any_abort, r), 1u);
  cluster_sync();
  if (bar->any_abort) {
    if (threadIdx.x == 0 && rank == 1)
      for (int r = 0; r < kRoles; ++r) store_cluster(map_cta(&bar->issued[1][r], lead), bar->issued[1][r]);
    cluster_sync();
    if (threadIdx.x == 0 && rank == 0) {
      DevCtl drain = p.ctl;
      drain.spin_limit = 1000000000LL;
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
  cfg.blockDim = dim3(threads_of(MX));
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

template <int EPI, bool A_MN, bool B_MN, bool MX, int SPLIT>
cudaError_t launch(const GemmParams& p, int clusters, cudaStream_t st) {
  cudaLaunchAttribute at[2];
  cudaLaunchConfig_t cfg = config<EPI, A_MN, B_MN, MX, SPLIT>(clusters, at);
  cfg.stream = st;
  return cudaLaunchKernelEx(&cfg, ffn_gemm_kernel<EPI, A_MN, B_MN, MX, SPLIT>, p);
}

template <int EPI, bool A_MN, bool B_MN, bool MX>
cudaError_t run(const FfnEngine& e, GemmParams& p, const void* a, const void* b, uint64_t b_rows, void* out,
                cudaStream_t st) {
  bool ok;
  if (MX) {
    ok = make_code_map(e.encode, &p.a, a, p.K, p.M, 128) && make_code_map(e.encode, &p.b, b, p.K, b_rows, 128);
  } else {  // a K-major operand is [rows, K], an MN-major one [K, rows]
    ok = A_MN ? make_bf16_map(e.encode, &p.a, a, p.M, p.K, p.M, 64, kBK)
              : make_bf16_map(e.encode, &p.a, a, p.K, p.M, p.K, kBK, kBM);
    ok = ok && (B_MN ? make_bf16_map(e.encode, &p.b, b, b_rows, p.K, b_rows, 64, kBK)
                     : make_bf16_map(e.encode, &p.b, b, p.K, b_rows, p.K, kBK, 128));
  }
  p.ctl = e.ctl;
  constexpr int TN = EPI == kEpiGateUp ? kBN / 2 : kBN;
  const long long tiles = (long long)((p.M + 2 * kBM - 1) / (2 * kBM)) * ((p.N + TN - 1) / TN);
  if (tiles > 0x7fffffffLL) return cudaErrorInvalidValue;
  const int blocks = (p.K + (MX ? 127 : 63)) / (MX ? 128 : 64);
  // Pairs that a tile's reduction is split over: time of a pair ~ rounds of tiles x (k blocks + what a tile costs
  // besides them, in k blocks); a split adds the exchange.
  constexpr int kMost = MX && EPI == kEpiGateUp ? 2 : 4;  // mx8: a warp must keep whole groups of 32 neurons
  int split = 1;
  double best = 1e30;
  for (int s = 1; s <= kMost && s <= blocks; s *= 2) {
    const int fit = s == 1 ? e.pairs : s == 2 ? e.pairs2 : e.pairs4;  // clusters that run at a time
    if (fit < 1) break;
    const double rounds = (double)((tiles + fit - 1) / fit);
    const double cost = rounds * ((blocks + s - 1) / s + kTileCost + (s > 1 ? kSplitCost : 0));
    if (cost < best) best = cost, split = s;
  }
  if (split == 1) {
    ok = ok && (!out || make_bf16_map(e.encode, &p.out, out, p.N, p.M, p.N, 64, 32));
    if (EPI != kEpiStore && !MX) {
      uint16_t* pre = EPI == kEpiGrad ? p.dpre : p.pre_out;
      if (pre)
        ok = ok && make_bf16_map(e.encode, &p.out_g, pre, p.N, p.M, 2 * (uint64_t)p.N, 64, 32) &&
             make_bf16_map(e.encode, &p.out_u, pre + p.N, p.N, p.M, 2 * (uint64_t)p.N, 64, 32);
    }
  }
  if (!ok) return cudaErrorInvalidValue;
  p.y = static_cast<uint16_t*>(out);
  if (split == 1) return launch<EPI, A_MN, B_MN, MX, 1>(p, tiles < e.pairs ? (int)tiles : e.pairs, st);
  if (split == 2) return launch<EPI, A_MN, B_MN, MX, 2>(p, (int)tiles, st);
  if constexpr (kMost == 4) return launch<EPI, A_MN, B_MN, MX, 4>(p, (int)tiles, st);
  return cudaErrorInvalidValue;
}

template <int EPI, bool A_MN, bool B_MN, bool MX, int SPLIT>
cudaError_t prepare(int* clusters) {
  auto k = ffn_gemm_kernel<EPI, A_MN, B_MN, MX, SPLIT>;
  cudaError_t err = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_of(EPI, MX, SPLIT));
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
  e->pairs = e->pairs2 = e->pairs4 = e->sms / 2;
  cudaError_t err = prepare_splits<kEpiGateUp, false, false, false>(e);
  if (err == cudaSuccess) err = prepare_splits<kEpiStore, false, false, false>(e);
  if (err == cudaSuccess) err = prepare_splits<kEpiGrad, false, true, false>(e);
  if (err == cudaSuccess) err = prepare_splits<kEpiStore, false, true, false>(e);
  if (err == cudaSuccess) err = prepare_splits<kEpiStore, true, true, false>(e);
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
  p.M = s.T;
  p.N = s.I;
  p.K = s.d;
  p.act = s.act;
  p.hq = hq;
  p.hs = hs;
  const uint64_t tiles = (s.I + 127) / 128;
  if (!make_scale_map(e.encode, &p.as, a.xs, s.d, (s.T + 127) / 128) ||
      !make_scale_map(e.encode, &p.bs0, a.gate_up_s, s.d, tiles) || !make_scale_map(e.encode, &p.bs1, up_s, s.d, tiles))
    return cudaErrorInvalidValue;
  return run<kEpiGateUp, false, false, true>(e, p, a.x, a.gate_up, 2 * (uint64_t)s.I, nullptr, st);
}

cudaError_t launch_ffn_down_mx(const FfnEngine& e, const FfnShape& s, const uint8_t* hq, const uint8_t* hs,
                               const FfnForwardArgs& a, cudaStream_t st) {
  GemmParams p{};
  p.M = s.T;
  p.N = s.d;
  p.K = s.I;
  const uint64_t tiles = (s.d + 127) / 128;
  if (!make_scale_map(e.encode, &p.as, hs, s.I, (s.T + 127) / 128) ||
      !make_scale_map(e.encode, &p.bs0, a.down_s, s.I, tiles))
    return cudaErrorInvalidValue;
  p.bs1 = p.bs0;
  return run<kEpiStore, false, false, true>(e, p, hq, a.down, s.d, a.y, st);
}

cudaError_t launch_ffn_gate_up(const FfnEngine& e, const FfnShape& s, const void* x, const void* gate_up, uint16_t* h,
                               uint16_t* pre, cudaStream_t st) {
  GemmParams p{};
  p.M = s.T;
  p.N = s.I;
  p.K = s.d;
  p.act = s.act;
  p.store_pre = pre != nullptr;
  p.pre_out = pre;
  return run<kEpiGateUp, false, false, false>(e, p, x, gate_up, 2 * (uint64_t)s.I, h, st);
}

cudaError_t launch_ffn_down(const FfnEngine& e, const FfnShape& s, const uint16_t* h, const void* down, void* y,
                            cudaStream_t st) {
  GemmParams p{};
  p.M = s.T;
  p.N = s.d;
  p.K = s.I;
  return run<kEpiStore, false, false, false>(e, p, h, down, s.d, y, st);
}

cudaError_t launch_ffn_grad_h(const FfnEngine& e, const FfnShape& s, const uint16_t* dy, const uint16_t* down,
                              const uint16_t* pre, uint16_t* dpre, uint16_t* h, cudaStream_t st) {
  GemmParams p{};
  p.M = s.T;
  p.N = s.I;
  p.K = s.d;
  p.act = s.act;
  p.pre = pre;
  p.dpre = dpre;
  return run<kEpiGrad, false, true, false>(e, p, dy, down, s.I, h, st);
}

cudaError_t launch_ffn_dx(const FfnEngine& e, const FfnShape& s, const uint16_t* dpre, const uint16_t* gate_up,
                          uint16_t* dx, cudaStream_t st) {
  GemmParams p{};
  p.M = s.T;
  p.N = s.d;
  p.K = 2 * s.I;
  return run<kEpiStore, false, true, false>(e, p, dpre, gate_up, s.d, dx, st);
}

cudaError_t launch_ffn_weight_grad(const FfnEngine& e, const uint16_t* a, int M, const uint16_t* b, int N, int T,
                                   uint16_t* dw, cudaStream_t st) {
  GemmParams p{};
  p.M = M;
  p.N = N;
  p.K = T;
  return run<kEpiStore, true, true, false>(e, p, a, b, N, dw, st);
}

}  // namespace moe
