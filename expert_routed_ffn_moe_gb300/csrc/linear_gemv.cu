// The product with its epilogue for one to four tokens: y = act(x w^T + bias) + residual.
//
// Bound by reading the weights once, on the CUDA cores: each 16 bytes of weights are 8
// multiply-adds per token, below what the SMs can do, and rows can be dealt out to all
// of them evenly, which tiles of 128 rows cannot (4096 rows are 32 tiles).  A block of 8
// warps per SM; a group of 1 to 8 of its warps has a contiguous range of rows, eight at a
// time, and its warps take the rows' length in turn, 512 columns each (two times 16 bytes
// per lane).  Weights come through each warp's own ring of three steps in shared memory
// by bulk copies, a row's 1024 bytes each (loads into registers one step ahead do not
// cover the memory's latency, 17.2 us below, and 16-byte copies cost more instructions
// than the sums, 16.2).  A warp's sums of eight rows meet by nine exchanges, the group's
// warps' in shared memory, in order; then one thread finishes each result.
//
// One token, 8192 to 4096 (67 MB): 14.5 us, some 4.6 of it for the launch, the first data
// and the end, the rest at the measured copy rate; 4096 to 16384 24.1 us.
#include "ops_internal.h"
#include "rows_common.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32, kRows = 8, kCols = 512, kSteps = 3;
constexpr int kPieces = kCols / 256;  // of 8 columns per lane
constexpr int kStepBytes = kRows * kCols * 2;  // of a warp
constexpr size_t kRingBytes = (size_t)kWarps * kSteps * kStepBytes;

struct GemvArgs {
  const __nv_bfloat16 *x, *w;
  LinearForwardArgs f;
  int K, N, act;
  int log_split;  // warps of a group: 1 << log_split
  DevCtl ctl;
};

MOE_DEV void bulk_copy(uint32_t to, const void* from, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(to),
               "l"(from), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}
// Sums over the warp of eight values: lane l gets that of value l / 4.
MOE_DEV float warp_sum8(const float (&v)[8]) {
  const int lane = threadIdx.x & 31;
  float a[4], b[2];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool up = (lane & 16) != 0;
    a[i] = (up ? v[i + 4] : v[i]) + __shfl_xor_sync(0xffffffffu, up ? v[i] : v[i + 4], 16);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const bool up = (lane & 8) != 0;
    b[i] = (up ? a[i + 2] : a[i]) + __shfl_xor_sync(0xffffffffu, up ? a[i] : a[i + 2], 8);
  }
  const bool up = (lane & 4) != 0;
  float c = (up ? b[1] : b[0]) + __shfl_xor_sync(0xffffffffu, up ? b[0] : b[1], 4);
  c += __shfl_xor_sync(0xffffffffu, c, 2);
  return c + __shfl_xor_sync(0xffffffffu, c, 1);
}

template <int T>
__global__ void __launch_bounds__(kThreads, 1) linear_gemv_kernel(const __grid_constant__ GemvArgs a) {
  __shared__ float part[2][kWarps][T][kRows];
  __shared__ uint64_t full[kWarps][kSteps], never;
  extern __shared__ __align__(128) uint8_t ring[];  // [kWarps][kSteps][kRows][kCols]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane < kSteps) mbar_init(&full[warp][lane], 1);
  if (threadIdx.x == 0) mbar_init(&never, 1);
  fence_mbar_init();
  __syncthreads();
  follow();

  const int split = 1 << a.log_split, groups = kWarps >> a.log_split;
  const int group = warp >> a.log_split, sub = warp & (split - 1);
  const int all = gridDim.x * groups;
  auto first_row = [&](int g) { return (int)((long long)a.N * (blockIdx.x * groups + g) / all); };
  const int r0 = first_row(group), r1 = first_row(group + 1);
  const int chunks = ((a.N + all - 1) / all + kRows - 1) / kRows;  // (the same for all: the block has barriers)
  const int stride = split * kCols, segs = (a.K + stride - 1) / stride;
  const int c0 = sub * kCols;
  uint8_t* mine = ring + warp * kSteps * kStepBytes;
  bool ok = true;
  if (a.ctl.stall) ok = mbar_wait(&never, 0, a.ctl);  // test hook: nothing arrives there

  // The copies of the next step: eight rows' 512 columns, as far as there are any.
  int ahead_chunk = 0, ahead_seg = 0, ahead_slot = 0, issued = 0;
  auto issue = [&]() {
    if (ahead_chunk >= chunks) return;
    const int row = r0 + ahead_chunk * kRows, c = c0 + ahead_seg * stride;
    const int rows = max(0, min(kRows, r1 - row)), bytes = max(0, min(kCols, a.K - c)) * 2;
    uint64_t* bar = &full[warp][ahead_slot];
    if (lane == 0) mbar_expect_tx(bar, rows * bytes);
    __syncwarp();
    if (lane < rows && bytes)
      bulk_copy(smem_u32(mine + ahead_slot * kStepBytes) + lane * kCols * 2, a.w + (size_t)(row + lane) * a.K + c, bytes, bar);
    ++issued;
    if (++ahead_seg == segs) ahead_seg = 0, ++ahead_chunk;
    if (++ahead_slot == kSteps) ahead_slot = 0;
  };
  if (ok) {
#pragma unroll
    for (int i = 0; i < kSteps; ++i) issue();
  }
  int slot = 0, parity = 0, used = 0;

  // What this thread finishes of every eight rows: row i_out of group g, token t_out.
  const int g = threadIdx.x / (T * kRows), t_out = threadIdx.x / kRows % T, i_out = threadIdx.x % kRows;
  static_assert(kWarps * T * kRows <= kThreads, "a thread per result");
  const int g0 = first_row(g) + i_out, g1 = g < groups ? first_row(g + 1) : 0;
  const LinearForwardArgs& f = a.f;
  for (int chunk = 0; chunk < chunks; ++chunk) {
    // its bias and residual, asked for before the sums are there
    const int n = g0 + chunk * kRows;
    const size_t at = (size_t)t_out * a.N + n;
    float bias = 0.f, res = 0.f;
    if (n < g1) {
      if (f.bias)
        bias = f.bias_dtype == MOE_BF16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(f.bias)[n])
                                        : static_cast<const float*>(f.bias)[n];
      if (f.res)
        res = f.y_dtype == MOE_BF16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(f.res)[at])
                                    : static_cast<const float*>(f.res)[at];
    }
    float2 acc[T][kRows];
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
      for (int i = 0; i < kRows; ++i) acc[t][i] = make_float2(0.f, 0.f);
    for (int seg = 0; seg < segs; ++seg) {
      const int c = c0 + seg * stride + lane * 8;
      uint4 x[kPieces][T];
#pragma unroll
      for (int q = 0; q < kPieces; ++q)
#pragma unroll
        for (int t = 0; t < T; ++t)
          if (c + q * 256 < a.K) x[q][t] = *reinterpret_cast<const uint4*>(a.x + (size_t)t * a.K + c + q * 256);
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&full[warp][slot], parity, a.ctl));
      if (!ok) continue;
      ++used;
#pragma unroll
      for (int q = 0; q < kPieces; ++q) {
        if (c + q * 256 >= a.K) continue;
        const uint4* w = reinterpret_cast<const uint4*>(mine + slot * kStepBytes) + q * 32 + lane;
        float2 xf[T][4];
#pragma unroll
        for (int t = 0; t < T; ++t) {
          const uint4 v = x[q][t];
          xf[t][0] = bf16_two(v.x), xf[t][1] = bf16_two(v.y), xf[t][2] = bf16_two(v.z), xf[t][3] = bf16_two(v.w);
        }
#pragma unroll
        for (int i = 0; i < kRows; ++i) {  // (rows past the group's last are not used)
          const uint4 v = w[i * (kCols / 8)];
          const float2 vf[4] = {bf16_two(v.x), bf16_two(v.y), bf16_two(v.z), bf16_two(v.w)};
#pragma unroll
          for (int t = 0; t < T; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[t][i] = fma2(vf[e], xf[t][e], acc[t][i]);
        }
      }
      __syncwarp();
      issue();  // (into the step just read)
      if (++slot == kSteps) slot = 0, parity ^= 1;
    }
    float(&to)[kWarps][T][kRows] = part[chunk & 1];
#pragma unroll
    for (int t = 0; t < T; ++t) {
      float v[kRows];
#pragma unroll
      for (int i = 0; i < kRows; ++i) v[i] = acc[t][i].x + acc[t][i].y;
      const float s = warp_sum8(v);
      if ((lane & 3) == 0) to[warp][t][lane >> 2] = s;
    }
    __syncthreads();  // (a part's memory is written again two chunks later, after the next barrier)
    if (n < g1) {
      float v = 0.f;
      for (int s = 0; s < split; ++s) v += to[g * split + s][t_out][i_out];
      v += bias;
      if (f.pre) f.pre[at] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
      with_act_or_none(a.act, [&](auto act) { v = act_value<decltype(act)::value>(v); });
      v += res;
      if (f.y_dtype == MOE_BF16)
        put(static_cast<__nv_bfloat16*>(f.y) + at, v);
      else
        put(static_cast<float*>(f.y) + at, v);
    }
  }
  // after a wait that ran out: what is still in flight lands before the block leaves
  for (; used < issued; ++used) mbar_wait(&full[warp][used % kSteps], used / kSteps & 1, drain_ctl(a.ctl));
}

template <int T>
cudaError_t launch(const GemvArgs& a, int grid, cudaStream_t st) {
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t err = allow_once(linear_gemv_kernel<T>, kRingBytes, allowed);
  return err != cudaSuccess ? err : launch_after(linear_gemv_kernel<T>, grid, dim3(kThreads), kRingBytes, st, a);
}

}  // namespace

cudaError_t launch_linear_gemv(const FfnEngine& e, const LinearShape& s, const LinearForwardArgs& f, cudaStream_t st) {
  GemvArgs a{static_cast<const __nv_bfloat16*>(f.x), static_cast<const __nv_bfloat16*>(f.w), f, s.k, s.n, s.act, 0, e.ctl};
  while ((1 << a.log_split) < kWarps && (kCols << (a.log_split + 1)) <= s.k) ++a.log_split;
  const int groups = kWarps >> a.log_split;
  int grid = (s.n + groups - 1) / groups;
  if (grid > e.sms) grid = e.sms;
  switch (s.T) {
    case 1: return launch<1>(a, grid, st);
    case 2: return launch<2>(a, grid, st);
    case 3: return launch<3>(a, grid, st);
    case 4: return launch<4>(a, grid, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace moe
