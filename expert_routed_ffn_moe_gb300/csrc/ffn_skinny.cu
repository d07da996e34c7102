// The gated feed-forward block for few tokens (T <= 64): both products bound by
// reading the weights once.
//
// The weight rows are the tensor cores' 128 rows and the tokens their N columns
// (D[row, token] = W x^T, N = T rounded up to 16, 32 or 64), so no MMA work and
// no shared memory goes to rows that do not exist, and one multiply per weight
// row block serves every token.  One CTA per SM; warp 0 streams 128 x 128-byte
// weight blocks and the matching x block through a TMA ring, warp 1 issues the
// MMAs, warps 2-5 read the accumulators (one weight row per thread).
//
// The blocks of all row tiles, laid end to end, are cut into one equal
// contiguous share per CTA whatever the shape, so every SM streams the same
// number of bytes.  A row tile that is cut is summed through memory: each CTA
// leaves its fp32 part in its own slot, and the last to arrive (a ticket per
// tile) adds the parts in the order of k -- the result depends on the shape
// and the number of SMs alone, never on timing, and no CTA waits for another.
//
// In the gate/up product a unit is 128 neurons: the blocks of its gate and up
// rows alternate into two accumulators, and the activation, the product and
// h's rounding (with mx8: a group of 32 neurons is one warp) finish here.
//
// The down kernel is launched with programmatic stream serialization: its CTAs
// start beside the gate/up kernel's, fill their rings with weights, and wait
// for h only then.  Both together fit an SM's shared memory and TMEM.
#include "ffn_internal.h"

namespace moe {
namespace {

constexpr int kRows = 128;                 // weight rows of a tile
constexpr int kBlockBytes = kRows * 128;   // a weight block: 128 rows x 128 bytes of k
constexpr int kThreads = 192;
constexpr int kSmemEach = 113 * 1024;      // so that two CTAs share an SM

struct SkinnyParams {
  CUtensorMap w, x;                // weights [rows, K]; x or h [T, K]
  CUtensorMap ws, us, xs;          // mx8 scales: of the rows (gate), of the up rows, of x or h
  uint16_t *h, *pre, *y;
  uint8_t *hq, *hs;
  float* parts;                    // [CTAs][2][(gate, up) x T x 128]
  unsigned* tickets;               // one per unit, 0 between launches
  int T, N, K;                     // N: neurons (gate/up) or rows of down
  int act;
  DevCtl ctl;
};

constexpr int stage_bytes(bool mx, int nt) { return kBlockBytes + nt * 128 + (mx ? 1024 : 0); }
constexpr int stages_of(bool mx, int nt) {
  const int n = (kSmemEach - 2048) / stage_bytes(mx, nt);
  return n > 8 ? 8 : n;
}
constexpr int accs_of(int nt) { return nt <= 32 ? 2 : 1; }  // accumulator sets
constexpr int acc_cols(bool gate, int nt) { return (gate ? 2 : 1) * nt; }
constexpr uint32_t tmem_cols(bool mx, bool gate, int nt) {
  const int need = accs_of(nt) * acc_cols(gate, nt) + (mx ? 16 : 0);
  return need <= 32 ? 32 : need <= 64 ? 64 : need <= 128 ? 128 : 256;
}

struct __align__(8) Bars {
  uint64_t full[8], empty[8], tfull[2], tempty[2], mma_done;
  uint32_t tmem_base;
  int abort_flag;
  int last;
};
constexpr size_t smem_of(bool mx, int nt) {
  return 1024 + (size_t)stages_of(mx, nt) * stage_bytes(mx, nt) + sizeof(Bars);
}
static_assert(smem_of(false, 16) <= kSmemEach && smem_of(true, 16) <= kSmemEach && smem_of(false, 64) <= kSmemEach &&
                  smem_of(true, 64) <= kSmemEach && stages_of(true, 64) >= 4,
              "two CTAs per SM");

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

// Whether `ok` holds in all 128 threads of the epilogue warps.
MOE_DEV bool all_of_128(bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.and.aligned.pred q, 1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(ok ? 1u : 0u)
      : "memory");
  return r != 0;
}

// The share of CTA c: k blocks [begin, end) of the units' blocks laid end to end.
struct Share {
  int begin, end;
};
MOE_DEV Share share_of(int c, int ctas, int total) {
  return Share{(int)((long long)c * total / ctas), (int)((long long)(c + 1) * total / ctas)};
}
// The CTA whose share holds block b.
MOE_DEV int cta_of(int b, int ctas, int total) {
  int c = (int)(((long long)b * ctas + ctas - 1) / total);
  while (c > 0 && share_of(c, ctas, total).begin > b) --c;
  while (share_of(c, ctas, total).end <= b) ++c;
  return c;
}

template <bool MX, bool GATE, int NT>
__global__ void __launch_bounds__(kThreads, 2) ffn_skinny_kernel(const __grid_constant__ SkinnyParams p) {
  constexpr int S = stages_of(MX, NT), kStage = stage_bytes(MX, NT), NACC = accs_of(NT), kAccCols = acc_cols(GATE, NT);
  constexpr uint32_t kCols = tmem_cols(MX, GATE, NT);
  constexpr int kDepth = MX ? 128 : 64;  // values of k per block
  constexpr int kParts = GATE ? 2 : 1;   // accumulators, and weight blocks per k block
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  // weight blocks, then x blocks, then scales (1024-byte aligned tiles first)
  uint8_t* xs0 = base + S * kBlockBytes;
  uint8_t* sc0 = xs0 + S * NT * 128;
  Bars* bar = reinterpret_cast<Bars*>(base + S * kStage);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int KB = (p.K + kDepth - 1) / kDepth, units = (p.N + kRows - 1) / kRows;
  const int total = units * KB, ctas = gridDim.x;
  const Share sh = share_of(blockIdx.x, ctas, total);

  if (threadIdx.x == 0) {
    for (int i = 0; i < 8; ++i) {
      mbar_init(&bar->full[i], 1);
      mbar_init(&bar->empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar->tfull[i], 1);
      mbar_init(&bar->tempty[i], 128);
    }
    mbar_init(&bar->mma_done, 1);
    bar->abort_flag = 0;
    bar->last = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(&bar->tmem_base, kCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar->tmem_base;
  // the down kernel may start now: it touches nothing of this launch before it has waited for its end
  if (GATE) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (warp == 0) {
    if (lane == 0) {
      const uint64_t once = policy_evict_first(), keep = policy_evict_last();
      const int steps = (sh.end - sh.begin) * kParts;
      auto weights = [&](int s) {  // the weight block of step s and its scales
        const int st = s % S, b = sh.begin + s / kParts, which = s % kParts;
        const int unit = b / KB, kb = b - unit * KB;
        mbar_expect_tx(&bar->full[st], kStage);
        tma_load_2d(base + st * kBlockBytes, &p.w, kb * kDepth, unit * kRows + which * p.N, &bar->full[st], once);
        if (MX) tma_load_scales(sc0 + st * 1024, which ? &p.us : &p.ws, kb, unit, &bar->full[st]);
      };
      auto tokens = [&](int s) {
        const int st = s % S, b = sh.begin + s / kParts, kb = b % KB;
        tma_load_2d(xs0 + st * NT * 128, &p.x, kb * kDepth, 0, &bar->full[st], keep);
        if (MX) tma_load_scales(sc0 + st * 1024 + 512, &p.xs, kb, 0, &bar->full[st]);
      };
      const int ahead = steps < S ? steps : S;
      for (int s = 0; s < ahead; ++s) weights(s);
      // the kernel before (whose output x or h is) has finished; without programmatic launch this returns at once
      asm volatile("griddepcontrol.wait;" ::: "memory");
      for (int s = 0; s < ahead; ++s) tokens(s);
      int s = ahead;
      for (; s < steps; ++s) {
        if (!mbar_wait(&bar->empty[s % S], ((s / S) & 1) ^ 1, p.ctl) || aborted(bar)) {
          set_abort(bar);
          break;
        }
        weights(s);
        tokens(s);
      }
      // the copies land before the CTA leaves
      DevCtl drain = p.ctl;
      drain.spin_limit = 1000000000LL;
      for (int j = s > S ? s - S : 0; j < s; ++j) mbar_wait(&bar->full[j % S], (j / S) & 1, drain);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      int s = 0, lt = 0;
      bool ok = true;
      if (p.ctl.stall && !mbar_wait(&bar->mma_done, 0, p.ctl)) {  // test hook: nothing arrives there before the end
        set_abort(bar);
        ok = false;
      }
      for (int b = sh.begin; b < sh.end && ok; ++lt) {
        const int unit = b / KB, stop = min(sh.end, (unit + 1) * KB), acc = lt % NACC;
        if (!mbar_wait(&bar->tempty[acc], ((lt / NACC) & 1) ^ 1, p.ctl) || aborted(bar)) {
          set_abort(bar);
          break;
        }
        tc_fence_after();
        const int first = b;
        for (; b < stop && ok; ++b) {
#pragma unroll
          for (int which = 0; which < kParts; ++which, ++s) {
            const int st = s % S;
            if (!mbar_wait(&bar->full[st], (s / S) & 1, p.ctl) || aborted(bar)) {
              set_abort(bar);
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t d = tmem + acc * kAccCols + which * NT;
            const uint64_t da = umma_desc_sw128(smem_u32(base + st * kBlockBytes));
            const uint64_t db = umma_desc_sw128(smem_u32(xs0 + st * NT * 128));
            if (MX) {
              const uint32_t ts = tmem + NACC * kAccCols + (s & 1) * 8, sc = smem_u32(sc0 + st * 1024);
              copy_scales(ts, sc);
              copy_scales(ts + 4, sc + 512);
#pragma unroll
              for (int j = 0; j < 4; ++j)
                mma_mx(d, da + j * 2, db + j * 2, umma_idesc_mx(kRows, NT, j), ts, ts + 4, b != first || j != 0);
            } else {
#pragma unroll
              for (int j = 0; j < 4; ++j)
                umma_bf16(d, da + j * 2, db + j * 2, umma_idesc_bf16(kRows, NT), b != first || j != 0);
            }
            umma_commit(&bar->empty[st]);
          }
        }
        if (ok) umma_commit(&bar->tfull[acc]);
      }
      umma_commit(&bar->mma_done);  // the MMAs issued so far are done before TMEM is freed
      mbar_wait(&bar->mma_done, 0, p.ctl);
    }
  } else {
    const int part = warp & 3, row = part * 32 + lane;  // this thread's weight row of the tile
    const int T = p.T;
    int lt = 0;
    // One unit's results for the tokens from t0 on: gate (or down) values v, up values u.
    auto finish = [&](int unit, int t0, const auto& v, const auto& u) {
      const int n = unit * kRows + row;
      const bool in = n < p.N;
#pragma unroll
      for (int i = 0; i < (int)(sizeof(v) / sizeof(float)); ++i) {
        const int t = t0 + i;
        if (t >= T) break;
        if (!GATE) {
          if (in) p.y[(size_t)t * p.N + n] = __bfloat16_as_ushort(__float2bfloat16_rn(v[i]));
          continue;
        }
        const float h = act_value(v[i], p.act) * u[i];
        if (MX) {
          // N is a multiple of 32: the warp's group is all in or all out
          const uint32_t byte = mx_scale_byte(__uint_as_float(__reduce_max_sync(0xffffffffu, mag_bits(h))));
          if (in) {
            p.hq[(size_t)t * p.N + n] = (uint8_t)e4m3x2(h * mx_inverse_scale(byte), 0.f);
            if (lane == 0) p.hs[mx_scale_word(t, unit, mx_tile_cols(p.N)) + part] = (uint8_t)byte;
          }
        } else if (in) {
          p.h[(size_t)t * p.N + n] = __bfloat16_as_ushort(__float2bfloat16_rn(h));
          if (p.pre) {
            p.pre[(size_t)t * 2 * p.N + n] = __bfloat16_as_ushort(__float2bfloat16_rn(v[i]));
            p.pre[(size_t)t * 2 * p.N + p.N + n] = __bfloat16_as_ushort(__float2bfloat16_rn(u[i]));
          }
        }
      }
    };
    const size_t slot = (size_t)kParts * T * kRows;  // floats of a part
    for (int b = sh.begin; b < sh.end; ++lt) {
      const int unit = b / KB, lo = unit * KB, hi = lo + KB;
      const int begin = b, end = min(sh.end, hi), acc = lt % NACC;
      b = end;
      // the four warps give up together or not at all: they meet at barriers below
      if (!all_of_128(mbar_wait(&bar->tfull[acc], (lt / NACC) & 1, p.ctl) && !aborted(bar))) {
        set_abort(bar);
        break;
      }
      tc_fence_after();
      const bool whole = begin == lo && end == hi;
      // a part is this CTA's first (its share begins inside the unit) or its last
      float* mine = p.parts + ((size_t)blockIdx.x * 2 + (begin > lo ? 0 : 1)) * slot;
      const uint32_t src = tmem + ((uint32_t)(part * 32) << 16) + acc * kAccCols;
#pragma unroll 1
      for (int t0 = 0; t0 < T; t0 += 16) {
        float v[16], u[16];
        tmem_ld16_async(src + t0, v);
        if (GATE) tmem_ld16_async(src + NT + t0, u);
        tmem_ld_wait();
        if (whole) {
          finish(unit, t0, v, u);
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            if (t0 + i >= T) break;
            __stcg(mine + (size_t)(t0 + i) * kRows + row, v[i]);
            if (GATE) __stcg(mine + (size_t)(T + t0 + i) * kRows + row, u[i]);
          }
        }
      }
      tc_fence_before();
      mbar_arrive(&bar->tempty[acc]);
      if (whole) continue;
      __threadfence();
      asm volatile("bar.sync 1, 128;" ::: "memory");
      const int c0 = cta_of(lo, ctas, total), c1 = cta_of(hi - 1, ctas, total);
      if (threadIdx.x == 64) {
        const bool last = atomicAdd(&p.tickets[unit], 1u) == (unsigned)(c1 - c0);
        if (last) p.tickets[unit] = 0u;  // for the next launch
        bar->last = last;
      }
      asm volatile("bar.sync 1, 128;" ::: "memory");
      if (!bar->last) continue;  // (written again only after the next unit's first bar.sync)
      __threadfence();
      // The parts lie in the slots of CTAs c0 .. c1: c0's begins the unit (slot 1), the others' begin inside it.
      // kTogether of them are read at a time, so that a part's latency is paid once per kTogether, and added in
      // the order of k.
      constexpr int kTogether = 4;
      const float* p0 = p.parts + ((size_t)c0 * 2 + 1) * slot + row;
      auto part_of = [&](int c) { return c == c0 ? p0 : p.parts + (size_t)c * 2 * slot + row; };
#pragma unroll 1
      for (int t0 = 0; t0 < T; t0 += 8) {
        float v[8], u[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = u[i] = 0.f;
#pragma unroll 1
        for (int c = c0; c <= c1; c += kTogether) {
          float a[kTogether][8], e[kTogether][8];
#pragma unroll
          for (int q = 0; q < kTogether; ++q)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const bool on = c + q <= c1 && t0 + i < T;
              const float* from = part_of(c + q) + (size_t)(t0 + i) * kRows;
              a[q][i] = on ? __ldcg(from) : 0.f;
              e[q][i] = GATE && on ? __ldcg(from + (size_t)T * kRows) : 0.f;
            }
#pragma unroll
          for (int q = 0; q < kTogether; ++q)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              v[i] += a[q][i];
              u[i] += e[q][i];
            }
        }
        finish(unit, t0, v, u);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, kCols);
}

// ------------------------------------------------------------------ host side
template <bool MX, bool GATE, int NT>
cudaError_t run(const FfnEngine& e, const SkinnyParams& p, cudaStream_t st) {
  const int depth = MX ? 128 : 64;
  const int total = (p.K + depth - 1) / depth * ((p.N + kRows - 1) / kRows);
  // at least 128 KB of weights per CTA, or a share is shorter than its latency
  const int least = GATE ? 4 : 8;
  int ctas = (total + least - 1) / least;
  if (ctas > e.sms) ctas = e.sms;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem_of(MX, NT);
  cfg.stream = st;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = GATE ? 0 : 1;
  return cudaLaunchKernelEx(&cfg, ffn_skinny_kernel<MX, GATE, NT>, p);
}
template <bool MX, bool GATE>
cudaError_t run_nt(const FfnEngine& e, const SkinnyParams& p, cudaStream_t st) {
  return p.T <= 16 ? run<MX, GATE, 16>(e, p, st) : p.T <= 32 ? run<MX, GATE, 32>(e, p, st) : run<MX, GATE, 64>(e, p, st);
}
template <bool MX, bool GATE, int NT>
cudaError_t prepare() {
  return cudaFuncSetAttribute(ffn_skinny_kernel<MX, GATE, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (int)smem_of(MX, NT));
}
template <bool MX, bool GATE>
cudaError_t prepare_nt() {
  cudaError_t err = prepare<MX, GATE, 16>();
  if (err == cudaSuccess) err = prepare<MX, GATE, 32>();
  if (err == cudaSuccess) err = prepare<MX, GATE, 64>();
  return err;
}

uint32_t token_rows(int T) { return T <= 16 ? 16 : T <= 32 ? 32 : 64; }

SkinnyParams params(const FfnEngine& e, const FfnShape& s, const FfnScratch& sc, bool gate) {
  SkinnyParams p{};
  p.T = s.T;
  p.N = gate ? s.I : s.d;
  p.K = gate ? s.d : s.I;
  p.act = s.act;
  p.parts = sc.parts;
  p.tickets = sc.tickets;
  p.ctl = e.ctl;
  return p;
}

}  // namespace

size_t skinny_part_bytes(int sms, int tokens) {
  return (size_t)sms * 2 * 2 * (tokens < kSkinnyTokens ? tokens : kSkinnyTokens) * kRows * 4;
}
int skinny_tickets(int d, int inter) { return ((d > inter ? d : inter) + kRows - 1) / kRows; }

cudaError_t prepare_ffn_skinny() {
  cudaError_t err = prepare_nt<false, false>();
  if (err == cudaSuccess) err = prepare_nt<false, true>();
  if (err == cudaSuccess) err = prepare_nt<true, false>();
  if (err == cudaSuccess) err = prepare_nt<true, true>();
  return err;
}

cudaError_t launch_skinny_forward(const FfnEngine& e, const FfnShape& s, bool mx, const FfnForwardArgs& a,
                                  const uint8_t* up_s, const FfnScratch& sc, cudaStream_t st) {
  SkinnyParams g = params(e, s, sc, true), d = params(e, s, sc, false);
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
  if (!ok) return cudaErrorInvalidValue;
  cudaError_t err = mx ? run_nt<true, true>(e, g, st) : run_nt<false, true>(e, g, st);
  if (err == cudaSuccess) err = mx ? run_nt<true, false>(e, d, st) : run_nt<false, false>(e, d, st);
  return err;
}

}  // namespace moe
