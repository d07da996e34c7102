// Root-mean-square norm with the residual's addition, its gradients, and the
// rounding of a matrix to mx8.
//
//   forward   s = x + residual;  y = s * rsqrt(mean(s^2) + eps) * w
//   backward  n = s * rstd, g = dy * w:  dx = rstd * (g - n * mean(g * n)) + ds,
//             dw = sum over rows of dy * n
//
// Both are bound by memory: one pass over the rows, which stay in registers
// between the reduction and the output (s is never read back).  A row belongs
// to R threads, each holding C chunks of 8 neighbouring columns (16-byte loads
// of bf16, two of fp32); R and C follow from the width alone (row_layout).  All
// sums are fp32: 8 C columns per thread, then a shuffle tree, then the warps'
// sums in order.  y is computed from the unrounded s and rounded once.
//
// A width that is not a multiple of 8 leaves rows unaligned; the chunks are
// then the aligned 16-byte windows of the whole matrix that cover the row, with
// the neighbours' columns masked, so the loads stay wide (ODD).
#include "ffn_internal.h"

namespace moe {
namespace {

struct F8 {
  float v[8];
};

template <typename T>
MOE_DEV F8 load8(const T* p);
template <>
MOE_DEV F8 load8<float>(const float* p) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  return F8{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}
template <>
MOE_DEV F8 load8<__nv_bfloat16>(const __nv_bfloat16* p) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  return F8{{bf16_lo(a.x), bf16_hi(a.x), bf16_lo(a.y), bf16_hi(a.y), bf16_lo(a.z), bf16_hi(a.z), bf16_lo(a.w),
             bf16_hi(a.w)}};
}
MOE_DEV void store8(float* p, const F8& f) {
  reinterpret_cast<float4*>(p)[0] = make_float4(f.v[0], f.v[1], f.v[2], f.v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(f.v[4], f.v[5], f.v[6], f.v[7]);
}
MOE_DEV void store8(__nv_bfloat16* p, const F8& f) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(f.v[0], f.v[1]), pack_bf16x2(f.v[2], f.v[3]),
                                            pack_bf16x2(f.v[4], f.v[5]), pack_bf16x2(f.v[6], f.v[7]));
}
MOE_DEV float to_f(float v) { return v; }
MOE_DEV float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
MOE_DEV void put(float* p, float v) { *p = v; }
MOE_DEV void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// The chunk of 8 columns at e of a matrix of n values; columns outside [lo, hi) read 0.
template <typename T, bool ODD>
MOE_DEV F8 load_chunk(const T* p, size_t e, size_t n, size_t lo, size_t hi) {
  if (!ODD) return load8(p + e);
  F8 f;
  if (e + 8 <= n) {
    f = load8(p + e);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f.v[i] = e + i < n ? to_f(p[e + i]) : 0.f;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (e + i < lo || e + i >= hi) f.v[i] = 0.f;
  return f;
}
template <typename T, bool ODD>
MOE_DEV void store_chunk(T* p, size_t e, size_t lo, size_t hi, const F8& f) {
  if (!ODD || (e >= lo && e + 8 <= hi)) {
    store8(p + e, f);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (e + i >= lo && e + i < hi) put(p + e + i, f.v[i]);
  }
}

// The sum over the R threads of a row, in every one of them.
template <int R>
MOE_DEV float row_sum(float v, float* red) {
  v = warp_sum(v);
  if (R == 32) return v;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) red[warp] = v;
  __syncthreads();
  return warp_sum(lane < R / 32 ? red[lane] : 0.f);
}

// The scale and the codes of this thread's 8 columns of a group of 32 (4
// neighbouring lanes hold the group; every lane of the warp takes part).
MOE_DEV uint2 quantize8(const F8& f, uint32_t& byte) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, mag_bits(f.v[i]));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  byte = mx_scale_byte(__uint_as_float(m));
  const float k = mx_inverse_scale(byte);
  return make_uint2(e4m3x4(f.v[0] * k, f.v[1] * k, f.v[2] * k, f.v[3] * k),
                    e4m3x4(f.v[4] * k, f.v[5] * k, f.v[6] * k, f.v[7] * k));
}
// The four scale bytes of 16 neighbouring lanes (128 columns), in the first of them.
MOE_DEV uint32_t gather_scales(uint32_t byte) {
  const uint32_t b1 = __shfl_down_sync(0xffffffffu, byte, 4), b2 = __shfl_down_sync(0xffffffffu, byte, 8),
                 b3 = __shfl_down_sync(0xffffffffu, byte, 12);
  return byte | (b1 << 8) | (b2 << 16) | (b3 << 24);
}

template <typename XT, typename ST, int R, int C, bool ODD>
__global__ void __launch_bounds__(R == 32 ? 128 : R) norm_kernel(NormArgs a) {
  __shared__ float red[32];
  constexpr int kRows = R == 32 ? 4 : 1;
  const int row = blockIdx.x * kRows + (R == 32 ? threadIdx.x >> 5 : 0);
  const int tid = R == 32 ? threadIdx.x & 31 : threadIdx.x;
  const size_t tile_cols = mx_tile_cols(a.d);
  if (row >= a.T) {
    // rows that only pad the last scale tile
    if (a.y_dtype == MOE_MX8 && row < (a.T + 127) / 128 * 128)
      for (size_t w = tid; w < tile_cols; w += R)
        *reinterpret_cast<uint32_t*>(a.scales + mx_scale_word(row, w, tile_cols)) = 0u;
    return;
  }
  const size_t n = (size_t)a.T * a.d, lo = (size_t)row * a.d, hi = lo + a.d;
  const size_t c0 = lo / 8;
  const int chunks = (int)((hi + 7) / 8 - c0);
  const XT* x = static_cast<const XT*>(a.x);
  const ST* res = static_cast<const ST*>(a.res);
  ST* s_out = static_cast<ST*>(a.s);

  F8 s[C];
#pragma unroll
  for (int j = 0; j < C; ++j) {
    const int c = tid + j * R;
    if (c < chunks) {
      s[j] = load_chunk<XT, ODD>(x, (c0 + c) * 8, n, lo, hi);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) s[j].v[i] = 0.f;
    }
  }
  if (res) {
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const int c = tid + j * R;
      if (c < chunks) {
        const F8 r = load_chunk<ST, ODD>(res, (c0 + c) * 8, n, lo, hi);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[j].v[i] += r.v[i];
      }
    }
  }
  float ss = 0.f;
#pragma unroll
  for (int j = 0; j < C; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) ss += s[j].v[i] * s[j].v[i];
  if (s_out) {
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const int c = tid + j * R;
      if (c < chunks) store_chunk<ST, ODD>(s_out, (c0 + c) * 8, lo, hi, s[j]);
    }
  }
  const float rstd = rsqrtf(row_sum<R>(ss, red) / (float)a.d + a.eps);
#pragma unroll
  for (int j = 0; j < C; ++j) {
    const int c = tid + j * R;
    const bool in = c < chunks;
    const size_t e = (c0 + c) * 8;
    F8 y;
    if (in) {
      F8 w;
      if (!ODD) {
        w = a.w_dtype == MOE_BF16 ? load8(static_cast<const __nv_bfloat16*>(a.w) + c * 8)
                                  : load8(static_cast<const float*>(a.w) + c * 8);
      } else {  // the weight's columns are not aligned with the windows
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const bool ok = e + i >= lo && e + i < hi;
          const int k = ok ? (int)(e + i - lo) : 0;
          const float v = a.w_dtype == MOE_BF16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.w)[k])
                                                : static_cast<const float*>(a.w)[k];
          w.v[i] = ok ? v : 0.f;
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) y.v[i] = s[j].v[i] * rstd * w.v[i];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) y.v[i] = 0.f;
    }
    if (a.y_dtype == MOE_MX8) {
      uint32_t byte;
      const uint2 q = quantize8(y, byte);
      if (!in) byte = 0u;  // groups past the last column
      const uint32_t word = gather_scales(byte);
      if (in) *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.y) + e) = q;
      if (in && c % 16 == 0) *reinterpret_cast<uint32_t*>(a.scales + mx_scale_word(row, c / 16, tile_cols)) = word;
    } else if (in) {
      if (a.y_dtype == MOE_BF16)
        store_chunk<__nv_bfloat16, ODD>(static_cast<__nv_bfloat16*>(a.y), e, lo, hi, y);
      else
        store_chunk<float, ODD>(static_cast<float*>(a.y), e, lo, hi, y);
    }
  }
}

// Gradients.  A block walks rows blockIdx.x, + gridDim.x, ...; every thread
// keeps the weight gradient of its own columns in registers over all of them
// and leaves it in row blockIdx.x of `partial`, which norm_grad_sum_kernel adds
// up in a fixed order (no atomics: the result does not depend on timing).  The
// columns of a thread must be the same for every row, so rows of odd width are
// read one column at a time (neighbouring threads, neighbouring columns).
template <typename ST, int R, int C, bool ODD>
__global__ void __launch_bounds__(R) norm_grad_kernel(NormGradArgs a) {
  __shared__ float red[2][32];
  const int tid = threadIdx.x;
  const ST* s_in = static_cast<const ST*>(a.s);
  const ST* dy_in = static_cast<const ST*>(a.dy);
  const ST* ds_in = static_cast<const ST*>(a.ds);
  ST* dx = static_cast<ST*>(a.dx);
  // column of value i of chunk j: 8 (tid + j R) + i, or tid + (8 j + i) R
  auto column = [&](int j, int i) { return ODD ? tid + (8 * j + i) * R : (tid + j * R) * 8 + i; };
  F8 acc[C];
#pragma unroll
  for (int j = 0; j < C; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[j].v[i] = 0.f;
  auto load_weight = [&](int j) {
    F8 w;
    if (!ODD && column(j, 0) < a.d) {
      w = a.w_dtype == MOE_BF16 ? load8(static_cast<const __nv_bfloat16*>(a.w) + column(j, 0))
                                : load8(static_cast<const float*>(a.w) + column(j, 0));
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int k = column(j, i);
        w.v[i] = k >= a.d ? 0.f
                          : (a.w_dtype == MOE_BF16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.w)[k])
                                                   : static_cast<const float*>(a.w)[k]);
      }
    }
    return w;
  };
  auto load_row = [&](const ST* p, size_t lo, F8(&f)[C]) {
#pragma unroll
    for (int j = 0; j < C; ++j) {
      if (ODD) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[j].v[i] = column(j, i) < a.d ? to_f(p[lo + column(j, i)]) : 0.f;
      } else if (column(j, 0) < a.d) {
        f[j] = load8(p + lo + column(j, 0));
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[j].v[i] = 0.f;
      }
    }
  };
  for (int row = blockIdx.x, it = 0; row < a.T; row += gridDim.x, ++it) {
    const size_t lo = (size_t)row * a.d;
    F8 s[C], dy[C];
    load_row(s_in, lo, s);
    load_row(dy_in, lo, dy);
    float ss = 0.f, sg = 0.f;
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const F8 w = load_weight(j);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        ss += s[j].v[i] * s[j].v[i];
        sg += s[j].v[i] * dy[j].v[i] * w.v[i];
      }
    }
    ss = warp_sum(ss);
    sg = warp_sum(sg);
    if (R > 32) {
      const int warp = tid >> 5, lane = tid & 31;
      __syncthreads();  // the previous row's sums have been read
      if (lane == 0) {
        red[0][warp] = ss;
        red[1][warp] = sg;
      }
      __syncthreads();
      ss = warp_sum(lane < R / 32 ? red[0][lane] : 0.f);
      sg = warp_sum(lane < R / 32 ? red[1][lane] : 0.f);
    }
    const float rstd = rsqrtf(ss / (float)a.d + a.eps);
    const float k = sg * rstd / (float)a.d;  // mean(g n)
    if (dx) {
      F8 o[C];
      if (ds_in) {
        load_row(ds_in, lo, o);
      } else {
#pragma unroll
        for (int j = 0; j < C; ++j)
#pragma unroll
          for (int i = 0; i < 8; ++i) o[j].v[i] = 0.f;
      }
#pragma unroll
      for (int j = 0; j < C; ++j) {
        const F8 w = load_weight(j);
#pragma unroll
        for (int i = 0; i < 8; ++i) o[j].v[i] += rstd * (dy[j].v[i] * w.v[i] - s[j].v[i] * rstd * k);
        if (ODD) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (column(j, i) < a.d) put(dx + lo + column(j, i), o[j].v[i]);
        } else if (column(j, 0) < a.d) {
          store8(dx + lo + column(j, 0), o[j]);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < C; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[j].v[i] += dy[j].v[i] * (s[j].v[i] * rstd);
  }
  if (a.dw) {
#pragma unroll
    for (int j = 0; j < C; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (column(j, i) < a.d) a.partial[(size_t)blockIdx.x * a.d + column(j, i)] = acc[j].v[i];
  }
}

// dw[c] = the sum of the blocks' partial gradients: 32 columns per block, 8
// threads per column over every 8th partial row, then the eight in order.
__global__ void __launch_bounds__(256) norm_grad_sum_kernel(const float* partial, int rows, int d, void* dw,
                                                            int w_dtype) {
  __shared__ float part[8][32];
  const int c = blockIdx.x * 32 + threadIdx.x;
  float v = 0.f;
  if (c < d)
    for (int r = threadIdx.y; r < rows; r += 8) v += partial[(size_t)r * d + c];
  part[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.y == 0 && c < d) {
    for (int i = 1; i < 8; ++i) v += part[i][threadIdx.x];
    if (w_dtype == MOE_BF16)
      static_cast<__nv_bfloat16*>(dw)[c] = __float2bfloat16_rn(v);
    else
      static_cast<float*>(dw)[c] = v;
  }
}

// One thread per 8 columns; cols is a multiple of 32.
template <typename T>
__global__ void __launch_bounds__(256) mx_quantize_kernel(const T* v, int rows, int cols, uint8_t* codes,
                                                          uint8_t* scales) {
  const size_t tile_cols = mx_tile_cols(cols);
  const size_t per_row = tile_cols * 16;  // chunks of a row, padded to whole scale words
  const size_t at = (size_t)blockIdx.x * 256 + threadIdx.x;
  const size_t row = at / per_row, c = at % per_row;
  const size_t all = (size_t)(rows + 127) / 128 * 128;
  if (row >= all) return;  // whole warps: all * per_row is a multiple of 32
  const bool in = row < (size_t)rows && c * 8 < (size_t)cols;
  F8 f;
  if (in) {
    f = load8(v + row * cols + c * 8);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f.v[i] = 0.f;
  }
  uint32_t byte;
  const uint2 q = quantize8(f, byte);
  if (!in) byte = 0u;
  const uint32_t word = gather_scales(byte);
  if (in) *reinterpret_cast<uint2*>(codes + row * cols + c * 8) = q;
  if (c % 16 == 0) *reinterpret_cast<uint32_t*>(scales + mx_scale_word(row, c / 16, tile_cols)) = word;
}

// Threads per row: the fewest (a power of two, 32 at least) that hold the row
// in at most 4 chunks of 8 columns each.
int row_threads(int chunks) {
  int r = 32;
  while (r < 1024 && r * 4 < chunks) r *= 2;
  return r;
}

template <typename XT, typename ST, int R, int C>
cudaError_t norm_odd(const NormArgs& a, cudaStream_t st) {
  const int rows = a.y_dtype == MOE_MX8 ? (a.T + 127) / 128 * 128 : a.T;
  const int grid = R == 32 ? (rows + 3) / 4 : rows;
  const int block = R == 32 ? 128 : R;
  if (a.d % 8 == 0)
    norm_kernel<XT, ST, R, C, false><<<grid, block, 0, st>>>(a);
  else
    norm_kernel<XT, ST, R, C, true><<<grid, block, 0, st>>>(a);
  return cudaGetLastError();
}
template <typename XT, typename ST>
cudaError_t norm_typed(const NormArgs& a, cudaStream_t st) {
  const int chunks = a.d % 8 == 0 ? a.d / 8 : (a.d + 7) / 8 + 1;  // an unaligned row may touch one window more
  switch (row_threads(chunks)) {
    case 32:
      if (chunks <= 32) return norm_odd<XT, ST, 32, 1>(a, st);
      return norm_odd<XT, ST, 32, 4>(a, st);
    case 64: return norm_odd<XT, ST, 64, 4>(a, st);
    case 128: return norm_odd<XT, ST, 128, 4>(a, st);
    case 256: return norm_odd<XT, ST, 256, 4>(a, st);
    case 512: return norm_odd<XT, ST, 512, 4>(a, st);
    default: return norm_odd<XT, ST, 1024, 4>(a, st);  // the widest odd rows
  }
}

template <typename ST, int R, int C>
cudaError_t grad_odd(const NormGradArgs& a, cudaStream_t st) {
  const int grid = a.T < kNormPartials ? a.T : kNormPartials;
  if (a.d % 8 == 0)
    norm_grad_kernel<ST, R, C, false><<<grid, R, 0, st>>>(a);
  else
    norm_grad_kernel<ST, R, C, true><<<grid, R, 0, st>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !a.dw) return e;
  norm_grad_sum_kernel<<<(a.d + 31) / 32, dim3(32, 8), 0, st>>>(a.partial, grid, a.d, a.dw, a.w_dtype);
  return cudaGetLastError();
}
template <typename ST>
cudaError_t grad_typed(const NormGradArgs& a, cudaStream_t st) {
  const int chunks = (a.d + 7) / 8;
  switch (row_threads(chunks)) {
    case 32:
      if (chunks <= 32) return grad_odd<ST, 32, 1>(a, st);
      return grad_odd<ST, 32, 4>(a, st);
    case 64: return grad_odd<ST, 64, 4>(a, st);
    case 128: return grad_odd<ST, 128, 4>(a, st);
    case 256: return grad_odd<ST, 256, 4>(a, st);
    default: return grad_odd<ST, 512, 4>(a, st);
  }
}

}  // namespace

cudaError_t launch_norm(const NormArgs& a, cudaStream_t st) {
  if (a.x_dtype == MOE_BF16)
    return a.s_dtype == MOE_BF16 ? norm_typed<__nv_bfloat16, __nv_bfloat16>(a, st)
                                 : norm_typed<__nv_bfloat16, float>(a, st);
  return a.s_dtype == MOE_BF16 ? norm_typed<float, __nv_bfloat16>(a, st) : norm_typed<float, float>(a, st);
}

cudaError_t launch_norm_backward(const NormGradArgs& a, cudaStream_t st) {
  return a.dtype == MOE_BF16 ? grad_typed<__nv_bfloat16>(a, st) : grad_typed<float>(a, st);
}

cudaError_t launch_mx_quantize(const void* v, int dtype, int rows, int cols, uint8_t* codes, uint8_t* scales,
                               cudaStream_t st) {
  const size_t n = (size_t)(rows + 127) / 128 * 128 * mx_tile_cols(cols) * 16;
  const size_t grid = (n + 255) / 256;
  if (grid > 0x7fffffffu) return cudaErrorInvalidValue;
  if (dtype == MOE_BF16)
    mx_quantize_kernel<<<(unsigned)grid, 256, 0, st>>>(static_cast<const __nv_bfloat16*>(v), rows, cols, codes, scales);
  else
    mx_quantize_kernel<<<(unsigned)grid, 256, 0, st>>>(static_cast<const float*>(v), rows, cols, codes, scales);
  return cudaGetLastError();
}

}  // namespace moe
