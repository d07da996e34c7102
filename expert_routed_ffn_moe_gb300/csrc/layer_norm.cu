// Layer norm with the residual's addition.
//
//   s = x + residual;  y = (s - mean(s)) * rsqrt(mean((s - mean(s))^2) + eps) * w + b
//
// Bound by memory: one pass over the rows, which stay in registers from their
// arrival to the output.  The variance is the mean of the squared distances from the
// mean, in a second sum over the registers (the difference of mean(s^2) and
// mean(s)^2 would lose what a row's offset takes of fp32's 24 bits).  A row belongs
// to R threads with 8 or 16 values each, R following from the width alone; blocks
// walk over rows.
//
// Two kernels.  Where rows are aligned a thread asks for its part of the next row
// before it finishes the present one, in registers, and reads weight and bias again
// for every row, from L1: the more warps fit an SM the better.  Other rows (see
// Windows) come through a ring in shared memory, and weight and bias, which do not
// lie on the windows' boundaries, are held in registers.
#include "layer_norm.cuh"

namespace moe {
namespace {

// Weight or bias of 8 columns, as param_of().
MOE_DEV F8 param8(const void* p, int dtype, int c, float otherwise) {
  if (p) return dtype == MOE_BF16 ? load8(static_cast<const __nv_bfloat16*>(p) + c) : load8(static_cast<const float*>(p) + c);
  F8 f;
#pragma unroll
  for (int i = 0; i < 8; ++i) f.v[i] = otherwise;
  return f;
}

// C chunks of 8 columns per thread.
template <typename XT, typename ST, int R, int C>
__global__ void __launch_bounds__(R == 32 ? 128 : R) layer_norm_kernel(LayerNormArgs a) {
  __shared__ float red[2][1][32];
  follow();
  constexpr int kRows = R == 32 ? 4 : 1;
  const int tid = R == 32 ? threadIdx.x & 31 : threadIdx.x;
  const XT* x_in = static_cast<const XT*>(a.x);
  const ST* r_in = static_cast<const ST*>(a.res);
  ST* s_out = static_cast<ST*>(a.s);
  const int stride = gridDim.x * kRows;
  const float inv_d = 1.0f / (float)a.d;

  Raw<XT> x[C];
  Raw<ST> res[C];
#pragma unroll
  for (int j = 0; j < C; ++j) {
    x[j].zero();
    res[j].zero();
  }
  auto load_row = [&](int row) {
    const size_t lo = (size_t)row * a.d;
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const int c = (tid + j * R) * 8;
      if (c < a.d) {
        x[j].load(x_in + lo + c);
        if (r_in) res[j].load(r_in + lo + c);
      }
    }
  };
  int row = blockIdx.x * kRows + (R == 32 ? threadIdx.x >> 5 : 0);
  if (row < a.T) load_row(row);
  for (; row < a.T; row += stride) {
    const size_t lo = (size_t)row * a.d;
    F8 s[C];
    float sum[1] = {0.f};
#pragma unroll
    for (int j = 0; j < C; ++j) {
      s[j] = x[j].get();
      const F8 r = res[j].get();
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        s[j].v[i] += r.v[i];  // (0 past the width)
        sum[0] += s[j].v[i];
      }
    }
    if (row + stride < a.T) load_row(row + stride);  // in flight while this row is finished
    if (s_out) {
#pragma unroll
      for (int j = 0; j < C; ++j) {
        const int c = (tid + j * R) * 8;
        if (c < a.d) store8(s_out + lo + c, s[j]);
      }
    }
    row_sums<R>(sum, &red[0]);
    const float mean = sum[0] * inv_d;
    sum[0] = 0.f;
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const bool in = (tid + j * R) * 8 < a.d;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        s[j].v[i] = in ? s[j].v[i] - mean : 0.f;
        sum[0] += s[j].v[i] * s[j].v[i];
      }
    }
    row_sums<R>(sum, &red[1]);
    const float rstd = rsqrtf(sum[0] * inv_d + a.eps);
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const int c = (tid + j * R) * 8;
      if (c < a.d) {
        const F8 w = param8(a.w, a.w_dtype, c, 1.f), b = param8(a.b, a.w_dtype, c, 0.f);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[j].v[i] = s[j].v[i] * rstd * w.v[i] + b.v[i];
        if (a.y_dtype == MOE_BF16)
          store8(static_cast<__nv_bfloat16*>(a.y) + lo + c, s[j]);
        else
          store8(static_cast<float*>(a.y) + lo + c, s[j]);
      }
    }
  }
}

template <typename XT, typename ST, int R, int C>
cudaError_t launch(const LayerNormArgs& a, cudaStream_t st) {
  constexpr int kBlock = R == 32 ? 128 : R, kRows = kBlock / R;
  const auto kernel = layer_norm_kernel<XT, ST, R, C>;
  int grid = (a.T + kRows - 1) / kRows;
  if (grid > 128) {  // (fewer blocks than SMs need no look at what is resident)
    static ByDevice known;
    const int resident = resident_blocks(kernel, kBlock, 0, known);
    if (grid > resident) grid = resident;
  }
  return launch_after(kernel, grid, dim3(kBlock), 0, st, a);
}
template <typename XT, typename ST>
cudaError_t aligned(const LayerNormArgs& a, cudaStream_t st) {
  if (a.d <= 512) return launch<XT, ST, 32, 2>(a, st);
  if (a.d <= 1024) return launch<XT, ST, 128, 1>(a, st);
  if (a.d <= 1536) return launch<XT, ST, 96, 2>(a, st);
  if (a.d <= 2048) return launch<XT, ST, 128, 2>(a, st);
  if (a.d <= 2560) return launch<XT, ST, 160, 2>(a, st);
  if (a.d <= 4096) return launch<XT, ST, 256, 2>(a, st);
  if (a.d <= 6144) return launch<XT, ST, 384, 2>(a, st);
  if (a.d <= 8192) return launch<XT, ST, 512, 2>(a, st);
  return launch<XT, ST, 1024, 2>(a, st);
}

// Rows of the ring: three, or what fits a block's shared memory.
template <typename XT, typename ST, int R>
constexpr int kStagesOf = [] {
  const int row = ln_rows(R) * 16 * R * (int)(sizeof(XT) + sizeof(ST)), most = (R <= 768 ? 220 / (768 / ln_block(R)) - 2 : 220) * 1024 / row;
  return most < 3 ? most : 3;
}();

template <typename XT, typename ST, int R>
__global__ void __launch_bounds__(ln_block(R), R <= 768 ? 768 / ln_block(R) : 1) layer_norm_odd_kernel(LayerNormArgs a) {
  constexpr int kRows = ln_rows(R), S = kStagesOf<XT, ST, R>;
  constexpr int kX = 16 * R * (int)sizeof(XT), kSlot = kX + 16 * R * (int)sizeof(ST);  // bytes of a row of x, of both
  constexpr bool HOLD = R < 1024;  // weight and bias in registers (else read again for every row, from L1)
  __shared__ RowRed<R, 1> red[2];
  extern __shared__ float4 ring4[];  // [kRows][S] rows of x and of the residual
  follow();
  const int tid = threadIdx.x % R, group = threadIdx.x / R;
  const int stride = gridDim.x * kRows, first = blockIdx.x * kRows + group;
  const Windows<R, true> win(tid, first, a.d);
  const size_t n = (size_t)a.T * a.d;
  const float inv_d = 1.0f / (float)a.d;
  uint8_t* x_sm = reinterpret_cast<uint8_t*>(ring4) + group * S * kSlot + tid * 16;
  uint8_t* r_sm = reinterpret_cast<uint8_t*>(ring4) + group * S * kSlot + kX + tid * 16;
  auto issue = [&](int it, int slot) {  // the copies of the group's it-th row
    const long long row = first + (long long)it * stride;
    if (row < a.T) {
      const size_t lo = (size_t)row * a.d;
#pragma unroll
      for (int o = 0; o < 2; ++o)
        if (win.in[o]) {
          win.copy(smem_u32(x_sm) + slot * kSlot, static_cast<const XT*>(a.x), lo, o, n);
          if (a.res)
            win.copy(smem_u32(r_sm) + slot * kSlot, static_cast<const ST*>(a.res), lo, o, n);
        }
    }
    copies_end();
  };
#pragma unroll
  for (int i = 0; i < S; ++i) issue(i, i);
  F8 w[2], b[2];
  if (HOLD) {
#pragma unroll
    for (int o = 0; o < 2; ++o) {
      w[o] = param_of(win, a.w, a.w_dtype, o, 1.f);
      b[o] = param_of(win, a.b, a.w_dtype, o, 0.f);
    }
  }
  int it = 0, slot = 0;
  for (int base = blockIdx.x * kRows; base < a.T; base += stride, ++it) {  // (the rows of a block end together)
    const int row = base + group;
    const bool live = kRows == 1 || row < a.T;
    const size_t lo = (size_t)row * a.d;
    copies_wait<S - 1>();
    F8 s[2];
    float sum[1] = {0.f};
#pragma unroll
    for (int o = 0; o < 2; ++o)
      if (win.in[o] && live) {
        s[o] = win.template take<XT>(x_sm + slot * kSlot, o);
        if (a.res) {
          const F8 r = win.template take<ST>(r_sm + slot * kSlot, o);
#pragma unroll
          for (int i = 0; i < 8; ++i) s[o].v[i] += r.v[i];
        }
        win.mask(o, s[o]);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[0] += s[o].v[i];
        if (a.s) win.store(static_cast<ST*>(a.s), lo, o, s[o]);
      }
    issue(it + S, slot);  // (this thread has read what lay there)
    if (++slot == S) slot = 0;
    ln_row_sums<R>(sum, red[0]);
    const float mean = sum[0] * inv_d;
    sum[0] = 0.f;
#pragma unroll
    for (int o = 0; o < 2; ++o)
      if (win.in[o]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) s[o].v[i] -= mean;
        win.mask(o, s[o]);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[0] += s[o].v[i] * s[o].v[i];
      }
    ln_row_sums<R>(sum, red[1]);
    const float rstd = rsqrtf(sum[0] * inv_d + a.eps);
#pragma unroll
    for (int o = 0; o < 2; ++o)
      if (win.in[o] && live) {
        const F8 wo = HOLD ? w[o] : param_of(win, a.w, a.w_dtype, o, 1.f);
        const F8 bo = HOLD ? b[o] : param_of(win, a.b, a.w_dtype, o, 0.f);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[o].v[i] = s[o].v[i] * rstd * wo.v[i] + bo.v[i];
        if (a.y_dtype == MOE_BF16)
          win.store(static_cast<__nv_bfloat16*>(a.y), lo, o, s[o]);
        else
          win.store(static_cast<float*>(a.y), lo, o, s[o]);
      }
  }
  copies_wait<0>();
}

template <typename XT, typename ST>
struct Odd {
  template <int R>
  struct Launch {
    static cudaError_t run(const LayerNormArgs& a, cudaStream_t st) {
      constexpr int kBlock = ln_block(R), kRows = ln_rows(R);
      constexpr size_t smem = (size_t)kRows * kStagesOf<XT, ST, R> * 16 * R * (sizeof(XT) + sizeof(ST));
      const auto kernel = layer_norm_odd_kernel<XT, ST, R>;
      static std::atomic<uint64_t> allowed{0};
      const cudaError_t err = allow_once(kernel, smem, allowed);
      if (err != cudaSuccess) return err;
      int grid = (a.T + kRows - 1) / kRows;
      if (grid > 128) {
        static ByDevice known;
        const int resident = resident_blocks(kernel, kBlock, smem, known) / 8 * 8;  // (see Windows)
        if (grid > resident) grid = resident;
      }
      if (!steps_of_eight(a.T, grid * kRows)) return cudaErrorInvalidValue;
      return launch_after(kernel, grid, dim3(kBlock), smem, st, a);
    }
  };
};
template <typename XT, typename ST>
cudaError_t typed(const LayerNormArgs& a, cudaStream_t st) {
  return a.d % 8 == 0 ? aligned<XT, ST>(a, st) : by_width<Odd<XT, ST>::template Launch>(a, st);
}

}  // namespace

cudaError_t launch_layer_norm(const LayerNormArgs& a, cudaStream_t st) {
  if (a.x_dtype == MOE_BF16)
    return a.s_dtype == MOE_BF16 ? typed<__nv_bfloat16, __nv_bfloat16>(a, st) : typed<__nv_bfloat16, float>(a, st);
  return a.s_dtype == MOE_BF16 ? typed<float, __nv_bfloat16>(a, st) : typed<float, float>(a, st);
}

}  // namespace moe
