// The gated feed-forward block for few tokens (see few_tokens()): the products
// that read the weights, bound by reading them once.
//
// The weight rows are the tensor cores' 128 rows and the tokens their N columns
// (D[row, token] = W x^T, N = T rounded up to 16, 32 or 64), so no MMA work and
// no shared memory goes to rows that do not exist, and one multiply per weight
// row block serves every token.  128 x 128-byte weight blocks and the matching x
// blocks go through a TMA ring.  A thread takes ~0.3 us to wait for a stage and
// to issue its copies, about as long as 16 KB take at an SM's share of the
// memory rate, so four warps share that: 0 and 6 bring the even and odd steps'
// weights, 7 and 8 their x blocks.  Warps 1 and 9 issue the even and odd steps'
// MMAs, into accumulators of their own: a wait for a stage queues behind the
// shared-memory operand reads of the MMAs before it, and one thread alone got
// through 16 KB per 0.30 us (0.40 us with mx8's scales), less than an SM's share
// of the memory rate.  Warps 2-5 read the accumulators (one weight row per
// thread).
//
// A tile of 128 weight rows belongs to a cluster of 1, 2, 4 or 8 CTAs, each of
// which streams a contiguous part of the row's length.  A power of two keeps the
// places of tokens and parts to shifts, but does not fill the device: where the
// rows are 2048 or a higher power of two there are 128 CTAs for 152 SMs, 86 for
// 11008 rows, 80 for 5120, 64 for 1024.  The parts meet in distributed shared memory: token t's are pushed to
// the cluster's CTA t mod C, which adds them in the order of k and finishes the
// token.  The result depends on the shape and the number of SMs, never on
// timing, and nothing goes through memory.
//
// In the gate/up product a tile is 128 neurons: the blocks of its gate and up
// rows alternate into two accumulators, and the activation, the product and
// h's rounding (with mx8: a group of 32 neurons is one warp) finish here.
//
// The two kernels overlap by programmatic launch: the down kernel's CTAs start
// beside the gate/up kernel's (one of each fits an SM), fill their rings with
// weights and only then wait for h.  A gate/up CTA that has asked for its last
// weights pulls its share of down's into L2, so memory stays busy while the
// gate/up product is summed up.
//
// The backward call's two are the same on the weights transposed, which are read
// where they lie (64 k rows of 128 neighbouring weight columns, an MN-major A):
// dh = dy down, whose finish reads pre and leaves dpre and h, and dx = dpre
// gate_up.  A backward call at T = 16, all three gradients, against these two as
// products of the pair kernel (us): d = 2048, I = 2048: 27 against 35; d = 1024,
// I = 2816: 20 against 35; d = 4096, I = 16384: 174 against 225.
#include "ffn_internal.h"

namespace moe {
namespace {

constexpr int kRows = 128;                 // weight rows of a tile
constexpr int kBlockBytes = kRows * 128;   // a weight block: 128 rows x 128 bytes of k
constexpr int kThreads = 320;
constexpr int kMaxCluster = 8;
constexpr int kMaxStages = 6;

// kLinear, kLinearDx: the product with its epilogue and its dx, calls of one such kernel
enum { kDown, kGateUp, kLinear, kGradH, kDx, kLinearDx };
constexpr bool first_of(int kind) { return kind != kDown && kind != kDx; }  // of a call's two kernels
constexpr bool w_mn(int kind) { return kind >= kGradH; }  // the weights lie [K, rows]

struct SkinnyParams {
  CUtensorMap w, x;                // weights; x, h, dy or dpre [T, K]
  CUtensorMap next;                // the first kernel: the weights of the second, next_rows x next_K (0: there is none)
  int next_rows, next_K;
  CUtensorMap ws, us, xs;          // mx8 scales: of the rows (gate), of the up rows, of x or h
  uint16_t *h, *pre, *y;           // y: of down or linear, or dx
  const void *bias, *res;          // linear: or NULL
  int bias_bf16, y32;              // linear: the bias is bf16; y and res are fp32
  uint16_t* dpre;
  uint8_t *hq, *hs;
  int T, N, K;                     // N: neurons (gate/up, grad_h) or columns of y
  int act;
  int log_cluster;                 // CTAs per tile: 1 << log_cluster
  DevCtl ctl;
};

constexpr int stage_bytes(bool mx, int nt) { return kBlockBytes + nt * 128 + (mx ? 1024 : 0); }
constexpr int exchange_bytes(int kind, int nt) { return nt * (kind == kGateUp ? 2 : 1) * kRows * 4; }
// Stages of the ring.  An even number: the even and the odd steps then have
// stages of their own, so that each stage's phases are waited for by one thread
// in their order (a wait by parity for a phase after the next would return at
// once).  A CTA of a call's first and one of its second kernel fit an SM together.
constexpr int stages_of(int kind, int nt) { return first_of(kind) && nt <= 16 ? 6 : 4; }
// Accumulators; mx8: and 8 columns of scales per stage, so that they are overwritten only when the MMAs that read them
// are done, like the stage itself.
constexpr uint32_t tmem_cols(bool mx, int kind, int nt) {
  const int need = 2 * nt + (mx ? 8 * stages_of(kind, nt) : 0);
  return need <= 32 ? 32 : need <= 64 ? 64 : need <= 128 ? 128 : 256;
}
// With 64 tokens the exchange lies in the ring's memory, so that two CTAs still
// fit an SM: the cluster's CTAs tell one another when their MMAs are done with it
// (1 - 1.5 us).
constexpr bool in_ring(int nt) { return nt > 32; }

struct __align__(8) Bars {
  uint64_t full[kMaxStages], empty[kMaxStages], tfull, mma_done;
  uint64_t parts;  // all parts of this CTA's tokens have been pushed here
  uint64_t ready;  // in_ring: all of the cluster's CTAs take parts in now
  uint32_t tmem_base;
  int abort_flag;
  int issued[2][2];  // by the producers of weights and of tokens, of even and odd steps
};
constexpr size_t smem_of(bool mx, int kind, int nt) {
  return 1024 + (size_t)stages_of(kind, nt) * stage_bytes(mx, nt) + (in_ring(nt) ? 0 : exchange_bytes(kind, nt)) +
         sizeof(Bars);
}
constexpr bool share_an_sm(bool mx, int first, int second, int nt) {  // 228 KB, 1 KB of it the system's for each CTA
  return smem_of(mx, first, nt) + smem_of(mx, second, nt) + 2048 <= 228 * 1024;
}
constexpr bool all_share(int nt) {
  return share_an_sm(false, kGateUp, kDown, nt) && share_an_sm(true, kGateUp, kDown, nt) &&
         share_an_sm(false, kGradH, kDx, nt);
}
static_assert(all_share(16) && all_share(32) && all_share(64), "shared memory");

MOE_DEV bool aborted(const Bars* b) { return *reinterpret_cast<const volatile int*>(&b->abort_flag) != 0; }
MOE_DEV void set_abort(Bars* b) { *reinterpret_cast<volatile int*>(&b->abort_flag) = 1; }

MOE_DEV void mma_mx(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
      : "memory");
}
// 512 bytes of scales into 4 TMEM columns, repeated for the four lane quarters.
MOE_DEV void copy_scales(uint32_t tmem, uint32_t saddr) {
  const uint64_t d = mx_scale_desc(saddr);
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(d) : "memory");
}
MOE_DEV void tma_load_scales(void* dst, const CUtensorMap* m, int col, int row, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(0), "r"(col), "r"(row), "r"(smem_u32(bar))
      : "memory");
}

MOE_DEV void tma_prefetch_2d(const CUtensorMap* m, int x, int y) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global [%0, {%1, %2}];" ::"l"(reinterpret_cast<uint64_t>(m)), "r"(x),
               "r"(y)
               : "memory");
}
// Bounded wait for arrivals of other CTAs of the cluster and the stores before them.
MOE_DEV bool mbar_wait_cluster(uint64_t* bar, uint32_t parity, const DevCtl& c) {
  const bool ok = mbar_wait(bar, parity, c);
  asm volatile("fence.acq_rel.cluster;" ::: "memory");
  return ok;
}

template <bool MX, int KIND, int NT>
__global__ void __launch_bounds__(kThreads, 1) ffn_skinny_kernel(const __grid_constant__ SkinnyParams p) {
  constexpr bool GATE = KIND == kGateUp, FIRST = first_of(KIND), W_MN = w_mn(KIND);
  static_assert(stages_of(KIND, NT) % 2 == 0 && stages_of(KIND, NT) <= kMaxStages, "see stages_of");
  static_assert(!MX || !W_MN, "mx8: forward products only");
  static_assert(!in_ring(NT) || exchange_bytes(KIND, NT) <= stages_of(KIND, NT) * stage_bytes(MX, NT), "the exchange");
  constexpr int S = stages_of(KIND, NT), kStage = stage_bytes(MX, NT);
  constexpr uint32_t kCols = tmem_cols(MX, KIND, NT);
  constexpr int kDepth = MX ? 128 : 64;  // values of k per block
  constexpr int kParts = GATE ? 2 : 1;   // weight blocks per k block
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  // weight blocks, then x blocks, then scales (1024-byte aligned tiles first), then the exchange
  uint8_t* xs0 = base + S * kBlockBytes;
  uint8_t* sc0 = xs0 + S * NT * 128;
  float* exchange = reinterpret_cast<float*>(base + (in_ring(NT) ? 0 : S * kStage));
  Bars* bar = reinterpret_cast<Bars*>(base + S * kStage + (in_ring(NT) ? 0 : exchange_bytes(KIND, NT)));

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank(), C = 1 << p.log_cluster;
  const int unit = blockIdx.x >> p.log_cluster;
  const int KB = (p.K + kDepth - 1) / kDepth;
  const int kb0 = (int)((long long)rank * KB >> p.log_cluster);
  const int steps = ((int)((long long)(rank + 1) * KB >> p.log_cluster) - kb0) * kParts;

  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(&bar->full[i], 2);  // the weights' and the tokens' producer
      mbar_init(&bar->empty[i], 1);
    }
    mbar_init(&bar->tfull, 2);
    mbar_init(&bar->mma_done, 2);
    mbar_init(&bar->parts, 4 * C);
    mbar_init(&bar->ready, C);
    bar->abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(&bar->tmem_base, kCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar->tmem_base;
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");  // waited for before the first push

  if (warp == 0 || (warp > 5 && warp < 9)) {
    if (lane == 0) {
      const bool tokens = warp > 6;
      const int odd = warp == 6 || warp == 8 ? 1 : 0;
      const uint64_t once = policy_evict_first(), keep = policy_evict_last();
      const int row0 = unit * kRows;
      auto load = [&](int s) {
        const int st = s % S, kb = kb0 + s / kParts, which = s % kParts;
        if (tokens) {
          mbar_expect_tx(&bar->full[st], NT * 128 + (MX ? 512 : 0));
          tma_load_2d(xs0 + st * NT * 128, &p.x, kb * kDepth, 0, &bar->full[st], keep);
          if (MX) tma_load_scales(sc0 + st * 1024 + 512, &p.xs, kb, 0, &bar->full[st]);
        } else {
          mbar_expect_tx(&bar->full[st], kBlockBytes + (MX ? 512 : 0));
          uint8_t* w = base + st * kBlockBytes;
          if (W_MN) {
            tma_load_2d(w, &p.w, row0, kb * kDepth, &bar->full[st], once);
            tma_load_2d(w + kBlockBytes / 2, &p.w, row0 + kRows / 2, kb * kDepth, &bar->full[st], once);
          } else {
            tma_load_2d(w, &p.w, kb * kDepth, row0 + which * p.N, &bar->full[st], once);
          }
          if (MX) tma_load_scales(sc0 + st * 1024, which ? &p.us : &p.ws, kb, unit, &bar->full[st]);
        }
      };
      // first kernel: the one before may have written anything; second: only its x, so the weights do not wait
      if (FIRST || tokens) asm volatile("griddepcontrol.wait;" ::: "memory");
      if (FIRST) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
      int s = odd;
      for (; s < steps; s += 2) {
        // (the second kernel's weights: the ring is full until h is there, and a wait's limit is not for the first kernel)
        if (!FIRST && s == S + odd) asm volatile("griddepcontrol.wait;" ::: "memory");
        if (s >= S && (!mbar_wait(&bar->empty[s % S], ((s / S) & 1) ^ 1, p.ctl) || aborted(bar))) {
          set_abort(bar);
          break;
        }
        load(s);
      }
      if (FIRST && !tokens) {
        const int nkb = (p.next_K + kDepth - 1) / kDepth, blocks = (p.next_rows + kRows - 1) / kRows * nkb;
        for (int b = 2 * blockIdx.x + odd; b < blocks; b += 2 * gridDim.x) {
          const int k = b % nkb * kDepth, row = b / nkb * kRows;
          if (W_MN) {
            tma_prefetch_2d(&p.next, row, k);
            if (row + kRows / 2 < p.next_rows) tma_prefetch_2d(&p.next, row + kRows / 2, k);
          } else {
            tma_prefetch_2d(&p.next, k, row);
          }
        }
      }
      if (!FIRST) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
      bar->issued[tokens][odd] = s;  // steps odd, odd + 2, ... below s
    }
  } else if (warp == 1 || warp == 9) {
    if (lane == 0) {
      const int odd = warp == 9 ? 1 : 0;
      bool ok = true;
      // Waits' limits are for what this kernel does: they begin when the kernel before has ended.
      asm volatile("griddepcontrol.wait;" ::: "memory");
      if (p.ctl.stall && !mbar_wait(&bar->mma_done, 0, p.ctl)) {  // test hook: nothing arrives there before the end
        set_abort(bar);
        ok = false;
      }
      const uint32_t d = tmem + odd * NT;  // gate/up: even steps are gate blocks, odd ones up blocks
      for (int s = odd; s < steps && ok; s += 2) {
        const int st = s % S;
        if (!mbar_wait(&bar->full[st], (s / S) & 1, p.ctl) || aborted(bar)) {
          set_abort(bar);
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t w = smem_u32(base + st * kBlockBytes);
        const uint64_t da = W_MN ? desc_mn(w) : umma_desc_sw128(w);
        const uint64_t db = umma_desc_sw128(smem_u32(xs0 + st * NT * 128));
        if (MX) {
          const uint32_t ts = tmem + 2 * NT + st * 8, sc = smem_u32(sc0 + st * 1024);
          copy_scales(ts, sc);
          copy_scales(ts + 4, sc + 512);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            mma_mx(d, da + j * 2, db + j * 2, umma_idesc_mx(kRows, NT, j), ts, ts + 4, s > odd || j != 0);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            umma_bf16(d, da + j * (W_MN ? 128 : 2), db + j * 2, umma_idesc_bf16(kRows, NT) | (W_MN ? 1u << 15 : 0u),
                      s > odd || j != 0);
        }
        umma_commit(&bar->empty[st]);
      }
      if (ok) umma_commit(&bar->tfull);
      umma_commit(&bar->mma_done);  // the MMAs issued so far are done before TMEM is freed
      mbar_wait(&bar->mma_done, 0, drain_ctl(p.ctl));
    }
  }
  __syncwarp();
  // every CTA of the cluster has set up its barriers: pushes may begin
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (warp >= 2 && warp <= 5) {
    const int part = warp & 3, row = part * 32 + lane;  // this thread's weight row of the tile
    const int T = p.T, own = (T + C - 1) >> p.log_cluster;  // tokens per CTA
    const int n = unit * kRows + row;
    const bool in = n < p.N;
    // The results of n tokens t, t + step, ...: values v (gate/up: of the gate), up values u.  No branch between the tokens, so
    // that their activations' latencies overlap.
    auto finish = [&](int t, int step, auto& v, const auto& u) {
      constexpr int n_tok = sizeof(v) / sizeof(float);
      if (GATE) {
        with_act(p.act, [&](auto act) {
#pragma unroll
          for (int i = 0; i < n_tok; ++i) {
            const float g = v[i];
            const size_t at = (size_t)(t + i * step) * 2 * p.N + n;
            if (!MX && p.pre && in && t + i * step < T) {
              p.pre[at] = __bfloat16_as_ushort(__float2bfloat16_rn(g));
              p.pre[at + p.N] = __bfloat16_as_ushort(__float2bfloat16_rn(u[i]));
            }
            v[i] = act_value<decltype(act)::value>(g) * u[i];
          }
        });
      }
      if constexpr (KIND == kGradH) {
        uint16_t g[n_tok], up[n_tok];
#pragma unroll
        for (int i = 0; i < n_tok; ++i) {
          const size_t at = (size_t)(t + i * step) * 2 * p.N + n;
          const bool is = in && t + i * step < T;
          g[i] = is ? p.pre[at] : (uint16_t)0;
          up[i] = is ? p.pre[at + p.N] : (uint16_t)0;
        }
        with_act(p.act, [&](auto act) {
#pragma unroll
          for (int i = 0; i < n_tok; ++i) {
            const float uv = __bfloat162float(__ushort_as_bfloat16(up[i]));
            float a, da;
            act_and_grad<decltype(act)::value>(__bfloat162float(__ushort_as_bfloat16(g[i])), a, da);
            const size_t row = t + i * step, at = row * 2 * p.N + n;
            if (in && row < T) {
              p.dpre[at] = __bfloat16_as_ushort(__float2bfloat16_rn(v[i] * uv * da));
              p.dpre[at + p.N] = __bfloat16_as_ushort(__float2bfloat16_rn(v[i] * a));
              p.h[row * p.N + n] = __bfloat16_as_ushort(__float2bfloat16_rn(a * uv));
            }
          }
        });
      } else if constexpr (KIND == kLinear) {
        const float b = !p.bias || !in ? 0.f
                        : p.bias_bf16  ? __bfloat162float(static_cast<const __nv_bfloat16*>(p.bias)[n])
                                       : static_cast<const float*>(p.bias)[n];
        float r[n_tok];
#pragma unroll
        for (int i = 0; i < n_tok; ++i) {
          const size_t at = (size_t)(t + i * step) * p.N + n;
          const bool is = p.res && in && t + i * step < T;
          r[i] = !is ? 0.f : p.y32 ? static_cast<const float*>(p.res)[at]
                                   : __bfloat162float(static_cast<const __nv_bfloat16*>(p.res)[at]);
        }
        with_act_or_none(p.act, [&](auto act) {
#pragma unroll
          for (int i = 0; i < n_tok; ++i) {
            const size_t at = (size_t)(t + i * step) * p.N + n;
            v[i] += b;
            if (p.pre && in && t + i * step < T) p.pre[at] = __bfloat16_as_ushort(__float2bfloat16_rn(v[i]));
            v[i] = act_value<decltype(act)::value>(v[i]) + r[i];
          }
        });
#pragma unroll
        for (int i = 0; i < n_tok; ++i) {
          const size_t at = (size_t)(t + i * step) * p.N + n;
          if (in && t + i * step < T) {
            if (p.y32)
              reinterpret_cast<float*>(p.y)[at] = v[i];
            else
              p.y[at] = __bfloat16_as_ushort(__float2bfloat16_rn(v[i]));
          }
        }
      } else if (GATE && MX) {
        uint32_t byte[n_tok];  // N is a multiple of 32: the warp's group is all in or all out
#pragma unroll
        for (int i = 0; i < n_tok; ++i)
          byte[i] = mx_scale_byte(__uint_as_float(__reduce_max_sync(0xffffffffu, mag_bits(v[i]))));
#pragma unroll
        for (int i = 0; i < n_tok; ++i) {
          const int ti = t + i * step;
          if (in && ti < T) {
            p.hq[(size_t)ti * p.N + n] = (uint8_t)e4m3x2(v[i] * mx_inverse_scale(byte[i]), 0.f);
            if (lane == 0) p.hs[mx_scale_word(ti, unit, mx_tile_cols(p.N)) + part] = (uint8_t)byte[i];
          }
        }
      } else {
        uint16_t* out = GATE ? p.h : p.y;
#pragma unroll
        for (int i = 0; i < n_tok; ++i)
          if (in && t + i * step < T)
            out[(size_t)(t + i * step) * p.N + n] = __bfloat16_as_ushort(__float2bfloat16_rn(v[i]));
      }
    };
    asm volatile("griddepcontrol.wait;" ::: "memory");  // (long over: the sums contain what the producers waited for)
    bool ok = mbar_wait(&bar->tfull, 0, p.ctl) && !aborted(bar);
    if (in_ring(NT) && C > 1) {
      // (all loads of this CTA have landed and been read; one that gives up does not arrive, and then nobody pushes)
      ok = __all_sync(0xffffffffu, ok);
      if (ok && warp == 2 && lane < C) arrive_cluster(map_cta(&bar->ready, lane));
      ok = ok && mbar_wait_cluster(&bar->ready, 0, p.ctl);
    }
    if (!__all_sync(0xffffffffu, ok)) {
      set_abort(bar);
    } else {
      tc_fence_after();
      const uint32_t src = tmem + ((uint32_t)(part * 32) << 16);
#pragma unroll 1
      for (int t0 = 0; t0 < T; t0 += 16) {
        float v[16], u[16];
        tmem_ld16_async(src + t0, v);
        tmem_ld16_async(src + NT + t0, u);
        tmem_ld_wait();
        if (!GATE && steps > 1) {
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] += u[i];
        }
        if (C == 1) {
          finish(t0, 1, v, u);
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int t = t0 + i;
            if (t < T) {
              const uint32_t at =
                  map_cta(exchange + ((rank * own + (t >> p.log_cluster)) * kParts) * kRows + row, t & (C - 1));
              asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(v[i]) : "memory");
              if (GATE) asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at + kRows * 4), "f"(u[i]) : "memory");
            }
          }
        }
      }
      if (C > 1) {
        asm volatile("fence.acq_rel.cluster;" ::: "memory");
        __syncwarp();
        if (lane < C) arrive_cluster(map_cta(&bar->parts, lane));
        ok = rank >= T || mbar_wait_cluster(&bar->parts, 0, p.ctl);
        if (!__all_sync(0xffffffffu, ok)) {
          set_abort(bar);
        } else {
#pragma unroll 1
          for (int i0 = 0; rank + i0 * C < T; i0 += 4) {  // four of this CTA's tokens, parts in the order of k
            float v[4] = {}, u[4] = {};
#pragma unroll 2
            for (int c = 0; c < C; ++c)
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float* q = exchange + ((c * own + min(i0 + j, own - 1)) * kParts) * kRows + row;
                v[j] += q[0];
                if (GATE) u[j] += q[kRows];
              }
            finish(rank + i0 * C, C, v, u);
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, kCols);
  if (threadIdx.x == 0 && bar->abort_flag) {
    // After an abort copies may be in flight (otherwise an MMA has waited for each): the last step of every stage
    // that anyone has issued must land before the CTA leaves.
    const DevCtl drain = drain_ctl(p.ctl);
    for (int st = 0; st < S; ++st)
      for (int j = st + (steps - 1) / S * S; j >= 0; j -= S) {
        const bool w = j < bar->issued[0][j & 1], t = j < bar->issued[1][j & 1];
        if (!w && !t) continue;
        if (!w || !t) mbar_arrive(&bar->full[st]);  // for the producer that did not get there
        mbar_wait(&bar->full[st], (j / S) & 1, drain);
        break;
      }
  }
  cluster_sync();  // no CTA leaves while another may still push to it
}

// ------------------------------------------------------------------ host side
// CTAs per tile: as many as keep the tiles' CTAs on different SMs (a power of
// two, 8 at most, and no more than there are k blocks).
int cluster_of(int tiles, int KB, int sms) {
  int c = 1;
  while (c < kMaxCluster && 2 * c * tiles <= sms && 2 * c <= KB) c *= 2;
  return c;
}

template <bool MX, int KIND, int NT>
cudaLaunchConfig_t config(int tiles, int C, cudaLaunchAttribute (&at)[2]) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(tiles * C);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem_of(MX, KIND, NT);
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = C;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cfg;
}
// Clusters of 8 on SMs of their own: half of what runs at a time, where two CTAs share an SM.
template <bool MX, int KIND, int NT>
cudaError_t lone_clusters(int* lone) {
  cudaLaunchAttribute at[2];
  cudaLaunchConfig_t cfg = config<MX, KIND, NT>(1, kMaxCluster, at);
  cfg.numAttrs = 1;
  int n = 0, per = 0;
  cudaError_t err = cudaOccupancyMaxActiveClusters(&n, ffn_skinny_kernel<MX, KIND, NT>, &cfg);
  if (err == cudaSuccess)
    err = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, ffn_skinny_kernel<MX, KIND, NT>, kThreads, cfg.dynamicSmemBytes);
  *lone = err == cudaSuccess && per > 0 ? n / per : 0;
  return err;
}
template <bool MX, int KIND, int NT>
cudaError_t run(const FfnEngine& e, SkinnyParams p, cudaStream_t st) {
  const int depth = MX ? 128 : 64;
  const int tiles = (p.N + kRows - 1) / kRows;
  int C = cluster_of(tiles, (p.K + depth - 1) / depth, e.sms);
  if constexpr (KIND == kLinear || KIND == kLinearDx) {
    // A call is this kernel alone, and clusters of 8 that have to share SMs, as they find no eight free ones in their part
    // of the device, cost more than they bring: 16 tiles (T = 16, d = 4096 to 2048) 13.6 us with 8, 9.0 with 4; 8 tiles
    // (4096 to 1024) 6.8 with 8, 8.0 with 4.
    static ByDevice known;
    if (C == 8 && tiles > once_per_device(known, lone_clusters<MX, KIND, NT>)) C = 4;
  }
  p.log_cluster = C == 8 ? 3 : C >> 1;
  cudaLaunchAttribute at[2];
  cudaLaunchConfig_t cfg = config<MX, KIND, NT>(tiles, C, at);
  cfg.stream = st;
  return cudaLaunchKernelEx(&cfg, ffn_skinny_kernel<MX, KIND, NT>, p);
}
template <bool MX, int KIND>
cudaError_t run_nt(const FfnEngine& e, const SkinnyParams& p, cudaStream_t st) {
  return p.T <= 16   ? run<MX, KIND, 16>(e, p, st)
         : p.T <= 32 ? run<MX, KIND, 32>(e, p, st)
                     : run<MX, KIND, 64>(e, p, st);
}
template <bool MX, int KIND, int NT>
cudaError_t prepare() {
  cudaError_t err = cudaFuncSetAttribute(ffn_skinny_kernel<MX, KIND, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)smem_of(MX, KIND, NT));
  // the SM keeps all its shared memory open, so that the other kernel's CTA fits beside this one's
  if (err == cudaSuccess)
    err = cudaFuncSetAttribute(ffn_skinny_kernel<MX, KIND, NT>, cudaFuncAttributePreferredSharedMemoryCarveout,
                               cudaSharedmemCarveoutMaxShared);
  return err;
}
template <bool MX, int KIND>
cudaError_t prepare_nt() {
  cudaError_t err = prepare<MX, KIND, 16>();
  if (err == cudaSuccess) err = prepare<MX, KIND, 32>();
  if (err == cudaSuccess) err = prepare<MX, KIND, 64>();
  return err;
}

uint32_t token_rows(int T) { return T <= 16 ? 16 : T <= 32 ? 32 : 64; }

SkinnyParams params(const FfnEngine& e, const FfnShape& s, int kind) {
  SkinnyParams p{};
  p.T = s.T;
  p.N = first_of(kind) ? s.I : s.d;
  p.K = first_of(kind) ? s.d : kind == kDx ? 2 * s.I : s.I;
  p.act = s.act;
  p.ctl = e.ctl;
  return p;
}

}  // namespace

cudaError_t prepare_ffn_skinny() {
  cudaError_t err = prepare_nt<false, kDown>();
  if (err == cudaSuccess) err = prepare_nt<false, kGateUp>();
  if (err == cudaSuccess) err = prepare_nt<true, kDown>();
  if (err == cudaSuccess) err = prepare_nt<true, kGateUp>();
  if (err == cudaSuccess) err = prepare_nt<false, kGradH>();
  if (err == cudaSuccess) err = prepare_nt<false, kDx>();
  if (err == cudaSuccess) err = prepare_nt<false, kLinear>();
  if (err == cudaSuccess) err = prepare_nt<false, kLinearDx>();
  return err;
}

cudaError_t launch_skinny_forward(const FfnEngine& e, const FfnShape& s, bool mx, const FfnForwardArgs& a,
                                  const uint8_t* up_s, const FfnScratch& sc, cudaStream_t st) {
  SkinnyParams g = params(e, s, kGateUp), d = params(e, s, kDown);
  const uint32_t nt = token_rows(s.T);
  bool ok;
  if (mx) {
    const uint64_t it = (s.I + 127) / 128, dt = (s.d + 127) / 128;
    ok = make_code_map(e.encode, &g.w, a.gate_up, s.d, 2 * (uint64_t)s.I, kRows) &&
         make_code_map(e.encode, &g.x, a.x, s.d, s.T, nt) && make_scale_map(e.encode, &g.ws, a.gate_up_s, s.d, it) &&
         make_scale_map(e.encode, &g.us, up_s, s.d, it) && make_scale_map(e.encode, &g.xs, a.xs, s.d, 1) &&
         make_code_map(e.encode, &d.w, a.down, s.I, s.d, kRows) && make_code_map(e.encode, &d.x, sc.hq, s.I, s.T, nt) &&
         make_scale_map(e.encode, &d.ws, a.down_s, s.I, dt) && make_scale_map(e.encode, &d.xs, sc.hs, s.I, 1);
    d.us = d.ws;
    g.hq = sc.hq;
    g.hs = sc.hs;
  } else {
    ok = make_bf16_map(e.encode, &g.w, a.gate_up, s.d, 2 * (uint64_t)s.I, s.d, 64, kRows) &&
         make_bf16_map(e.encode, &g.x, a.x, s.d, s.T, s.d, 64, nt) &&
         make_bf16_map(e.encode, &d.w, a.down, s.I, s.d, s.I, 64, kRows) &&
         make_bf16_map(e.encode, &d.x, sc.h, s.I, s.T, s.I, 64, nt);
    g.h = sc.h;
    g.pre = static_cast<uint16_t*>(a.pre);
  }
  d.y = static_cast<uint16_t*>(a.y);
  g.next = d.w;
  g.next_rows = s.d;
  g.next_K = s.I;
  if (!ok) return cudaErrorInvalidValue;
  cudaError_t err = mx ? run_nt<true, kGateUp>(e, g, st) : run_nt<false, kGateUp>(e, g, st);
  if (err == cudaSuccess) err = mx ? run_nt<true, kDown>(e, d, st) : run_nt<false, kDown>(e, d, st);
  return err;
}

cudaError_t launch_skinny_backward(const FfnEngine& e, const FfnShape& s, const FfnBackwardArgs& a,
                                   const FfnScratch& sc, cudaStream_t st) {
  SkinnyParams g = params(e, s, kGradH), d = params(e, s, kDx);
  const uint32_t nt = token_rows(s.T);
  const uint64_t I2 = 2 * (uint64_t)s.I;
  bool ok = make_bf16_map(e.encode, &g.w, a.down, s.I, s.d, s.I, 64, 64) &&
            make_bf16_map(e.encode, &g.x, a.dy, s.d, s.T, s.d, 64, nt);
  if (a.dx) {
    ok = ok && make_bf16_map(e.encode, &d.w, a.gate_up, s.d, I2, s.d, 64, 64) &&
         make_bf16_map(e.encode, &d.x, sc.dpre, I2, s.T, I2, 64, nt);
    g.next = d.w;
    g.next_rows = d.N;
    g.next_K = d.K;
  }
  if (!ok) return cudaErrorInvalidValue;
  g.pre = const_cast<uint16_t*>(a.pre);  // (read)
  g.dpre = sc.dpre;
  g.h = sc.h;
  d.y = a.dx;
  cudaError_t err = run_nt<false, kGradH>(e, g, st);
  if (err == cudaSuccess && a.dx) err = run_nt<false, kDx>(e, d, st);
  return err;
}

cudaError_t launch_linear_stream(const FfnEngine& e, const LinearShape& s, const LinearForwardArgs& a, cudaStream_t st) {
  SkinnyParams p{};
  p.T = s.T;
  p.N = s.n;
  p.K = s.k;
  p.act = s.act;
  p.ctl = e.ctl;
  p.y = static_cast<uint16_t*>(a.y);
  p.pre = a.pre;
  p.bias = a.bias;
  p.res = a.res;
  p.bias_bf16 = a.bias_dtype == MOE_BF16;
  p.y32 = a.y_dtype == MOE_F32;
  if (!make_bf16_map(e.encode, &p.w, a.w, s.k, s.n, s.k, 64, kRows) ||
      !make_bf16_map(e.encode, &p.x, a.x, s.k, s.T, s.k, 64, token_rows(s.T)))
    return cudaErrorInvalidValue;
  return run_nt<false, kLinear>(e, p, st);
}

cudaError_t launch_linear_dx_stream(const FfnEngine& e, const LinearShape& s, const uint16_t* dpre, const void* w,
                                    void* dx, cudaStream_t st) {
  SkinnyParams p{};
  p.T = s.T;
  p.N = s.k;
  p.K = s.n;
  p.ctl = e.ctl;
  p.y = static_cast<uint16_t*>(dx);
  if (!make_bf16_map(e.encode, &p.w, w, s.k, s.n, s.k, 64, 64) ||
      !make_bf16_map(e.encode, &p.x, dpre, s.n, s.T, s.n, 64, token_rows(s.T)))
    return cudaErrorInvalidValue;
  return run_nt<false, kLinearDx>(e, p, st);
}

}  // namespace moe
