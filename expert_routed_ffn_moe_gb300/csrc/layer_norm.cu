// Layer norm with the residual's addition.
//
//   s = x + residual;  y = (s - mean(s)) * rsqrt(mean((s - mean(s))^2) + eps) * w + b
//
// Bound by memory: one pass over the rows, which stay in registers from their
// load to the output.  The variance is the mean of the squared distances from the
// mean, in a second sum over the registers (the difference of mean(s^2) and
// mean(s)^2 would lose what a row's offset takes of fp32's 24 bits); with several
// rows in flight per SM the second sum's time is hidden.  A row belongs to R
// threads with 16 values each (8 for narrow ones): R follows from the width
// alone.  Blocks walk over rows and ask for the next one before they finish the
// present one.  Weight and bias are read again for every row, from L1.
//
// Widths that are a multiple of 8 move in chunks of 8 columns (16-byte loads of
// bf16, two of fp32).  For other widths, whose rows are not aligned, a chunk is
// one column: neighbouring threads read neighbouring values, and a thread has
// the same columns in every row, whatever the row's alignment.
#include "layer_norm.cuh"

namespace moe {
namespace {

template <typename XT, typename ST, int R, int C, int VEC>
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

  Chunk<XT, VEC> x[C];
  Chunk<ST, VEC> res[C];
#pragma unroll
  for (int j = 0; j < C; ++j) {
    x[j].zero();
    res[j].zero();
  }
  auto load_row = [&](int row) {
    const size_t lo = (size_t)row * a.d;
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const int c = (tid + j * R) * VEC;
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
    float s[C][VEC], sum[1] = {0.f};
#pragma unroll
    for (int j = 0; j < C; ++j)
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        s[j][i] = x[j].get(i) + res[j].get(i);  // (0 past the width)
        sum[0] += s[j][i];
      }
    if (row + stride < a.T) load_row(row + stride);  // in flight while this row is finished
    if (s_out) {
#pragma unroll
      for (int j = 0; j < C; ++j) {
        const int c = (tid + j * R) * VEC;
        if (c < a.d) Chunk<ST, VEC>::store(s_out + lo + c, s[j]);
      }
    }
    row_sums<R>(sum, &red[0]);
    const float mean = sum[0] * inv_d;
    sum[0] = 0.f;
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const bool in = (tid + j * R) * VEC < a.d;
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        s[j][i] = in ? s[j][i] - mean : 0.f;
        sum[0] += s[j][i] * s[j][i];
      }
    }
    row_sums<R>(sum, &red[1]);
    const float rstd = rsqrtf(sum[0] * inv_d + a.eps);
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const int c = (tid + j * R) * VEC;
      if (c < a.d) {
        float w[VEC], b[VEC];
        load_param<VEC>(w, a.w, a.w_dtype, c, 1.f);
        load_param<VEC>(b, a.b, a.w_dtype, c, 0.f);
#pragma unroll
        for (int i = 0; i < VEC; ++i) w[i] = s[j][i] * rstd * w[i] + b[i];
        if (a.y_dtype == MOE_BF16)
          Chunk<__nv_bfloat16, VEC>::store(static_cast<__nv_bfloat16*>(a.y) + lo + c, w);
        else
          Chunk<float, VEC>::store(static_cast<float*>(a.y) + lo + c, w);
      }
    }
  }
}

template <typename XT, typename ST, int R, int C, int VEC>
cudaError_t launch(const LayerNormArgs& a, cudaStream_t st) {
  constexpr int kBlock = R == 32 ? 128 : R, kRows = kBlock / R;
  const auto kernel = layer_norm_kernel<XT, ST, R, C, VEC>;
  int grid = (a.T + kRows - 1) / kRows;
  if (grid > 128) {  // (fewer blocks than SMs need no look at what is resident)
    static const int resident = resident_blocks(kernel, kBlock, 0);
    if (grid > resident) grid = resident;
  }
  return launch_after(kernel, grid, dim3(kBlock), 0, st, a);
}
template <typename XT, typename ST, int VEC>
cudaError_t by_width(const LayerNormArgs& a, cudaStream_t st) {
  if (a.d <= 512) return launch<XT, ST, 32, 16 / VEC, VEC>(a, st);
  if (a.d <= 1024) return launch<XT, ST, 128, 8 / VEC, VEC>(a, st);
  if (a.d <= 2048) return launch<XT, ST, 128, 16 / VEC, VEC>(a, st);
  if (a.d <= 4096) return launch<XT, ST, 256, 16 / VEC, VEC>(a, st);
  if (a.d <= 8192) return launch<XT, ST, 512, 16 / VEC, VEC>(a, st);
  return launch<XT, ST, 1024, 16 / VEC, VEC>(a, st);
}
template <typename XT, typename ST>
cudaError_t typed(const LayerNormArgs& a, cudaStream_t st) {
  return a.d % 8 == 0 ? by_width<XT, ST, 8>(a, st) : by_width<XT, ST, 1>(a, st);
}

}  // namespace

cudaError_t launch_layer_norm(const LayerNormArgs& a, cudaStream_t st) {
  if (a.x_dtype == MOE_BF16)
    return a.s_dtype == MOE_BF16 ? typed<__nv_bfloat16, __nv_bfloat16>(a, st) : typed<__nv_bfloat16, float>(a, st);
  return a.s_dtype == MOE_BF16 ? typed<float, __nv_bfloat16>(a, st) : typed<float, float>(a, st);
}

}  // namespace moe
