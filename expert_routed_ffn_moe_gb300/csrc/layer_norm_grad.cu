// Gradients of the layer norm.
//
//   c = s - mean(s), rstd = rsqrt(mean(c^2) + eps), n = c rstd, g = dy w
//   dx = rstd * (g - mean(g) - n * mean(g n)) + ds
//   dw = sum over the rows of dy n,  db = sum over the rows of dy
//
// Bound by memory: one pass over s, dy and ds, rows in registers, as in the
// forward pass; mean(s) and mean(g) come from one sum over the row's threads,
// mean(c^2) and mean(g c) from a second.  A thread has the same columns in every
// row and keeps their dw and db in registers (in shared memory where a block of
// 1024 threads has 64 registers each, see kAccShared).  A block leaves the sums
// over its rows in `partial`, which a second kernel adds up in a fixed order: no
// atomics, the result does not depend on timing.
#include "layer_norm.cuh"

namespace moe {
namespace {

// Gradients of weight and bias in shared memory: where registers do not hold them beside the rows.
template <typename T, int R>
constexpr bool kAccShared = R == 1024;
// The next row asked for while this one is finished: where registers hold both.
template <typename T, int R>
constexpr bool kAhead = R < 1024 && (sizeof(T) == 2 || R < 512);

template <int VEC>
MOE_DEV void add_shared(float* p, const float (&f)[VEC]) {
  if constexpr (VEC == 8) {
    F8 t = load8(p);
#pragma unroll
    for (int i = 0; i < 8; ++i) t.v[i] += f[i];
    store8(p, t);
  } else {
    *p += f[0];
  }
}

template <typename ST, int R, int C, int VEC>
__global__ void __launch_bounds__(R == 32 ? 128 : R) layer_norm_grad_kernel(LayerNormGradArgs a) {
  constexpr bool SHARED = kAccShared<ST, R>, AHEAD = kAhead<ST, R>;
  __shared__ float red[2][2][32];
  // SHARED: [2][d] sums; R == 32: the warps' sums at the end, [4][2][d]
  extern __shared__ float4 sums4[];
  float* sums = reinterpret_cast<float*>(sums4);
  follow();
  constexpr int kRows = R == 32 ? 4 : 1;
  const int tid = R == 32 ? threadIdx.x & 31 : threadIdx.x, group = R == 32 ? threadIdx.x >> 5 : 0;
  const int stride = gridDim.x * kRows;
  const ST* s_in = static_cast<const ST*>(a.s);
  const ST* dy_in = static_cast<const ST*>(a.dy);
  const ST* ds_in = static_cast<const ST*>(a.ds);
  ST* dx = static_cast<ST*>(a.dx);
  const float inv_d = 1.0f / (float)a.d;

  Chunk<ST, VEC> rs[C], rdy[C], rds[C];
#pragma unroll
  for (int j = 0; j < C; ++j) {
    rs[j].zero();
    rdy[j].zero();
    rds[j].zero();
  }
  auto load_row = [&](int row) {
    const size_t lo = (size_t)row * a.d;
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const int c = (tid + j * R) * VEC;
      if (c < a.d) {
        rs[j].load(s_in + lo + c);
        rdy[j].load(dy_in + lo + c);
        if (ds_in && dx) rds[j].load(ds_in + lo + c);
      }
    }
  };
  float dw[SHARED ? 1 : C][VEC], db[SHARED ? 1 : C][VEC];
  if (SHARED) {
    for (int k = threadIdx.x; k < 2 * a.d; k += R) sums[k] = 0.f;
    __syncthreads();
  } else {
#pragma unroll
    for (int j = 0; j < (SHARED ? 1 : C); ++j)
#pragma unroll
      for (int i = 0; i < VEC; ++i) dw[j][i] = db[j][i] = 0.f;
  }

  int row = blockIdx.x * kRows + group;
  if (row < a.T) load_row(row);
  for (; row < a.T; row += stride) {
    const size_t lo = (size_t)row * a.d;
    Chunk<ST, VEC> cs[C], cdy[C], cds[C];
    float sum[2] = {0.f, 0.f};  // s and g
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const int c = (tid + j * R) * VEC;
      cs[j] = rs[j];
      cdy[j] = rdy[j];
      cds[j] = rds[j];
      if (c < a.d) {
        float w[VEC];
        load_param<VEC>(w, a.w, a.w_dtype, c, 1.f);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          sum[0] += cs[j].get(i);
          sum[1] += cdy[j].get(i) * w[i];
        }
      }
    }
    if (AHEAD && row + stride < a.T) load_row(row + stride);
    row_sums<R>(sum, &red[0]);
    const float mean = sum[0] * inv_d, g_mean = sum[1] * inv_d;
    sum[0] = sum[1] = 0.f;  // c^2 and g c
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const int c = (tid + j * R) * VEC;
      if (c < a.d) {
        float w[VEC];
        load_param<VEC>(w, a.w, a.w_dtype, c, 1.f);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const float v = cs[j].get(i) - mean;
          sum[0] += v * v;
          sum[1] += cdy[j].get(i) * w[i] * v;
        }
      }
    }
    row_sums<R>(sum, &red[1]);
    const float rstd = rsqrtf(sum[0] * inv_d + a.eps);
    const float gn_mean = sum[1] * rstd * inv_d;
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const int c = (tid + j * R) * VEC;
      if (c < a.d) {
        float w[VEC], n[VEC];
        load_param<VEC>(w, a.w, a.w_dtype, c, 1.f);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const float dy = cdy[j].get(i);
          n[i] = (cs[j].get(i) - mean) * rstd;
          w[i] = rstd * (dy * w[i] - g_mean - n[i] * gn_mean) + cds[j].get(i);
          n[i] *= dy;
        }
        if (dx) Chunk<ST, VEC>::store(dx + lo + c, w);
        if (SHARED) {
          add_shared<VEC>(sums + c, n);
#pragma unroll
          for (int i = 0; i < VEC; ++i) n[i] = cdy[j].get(i);
          add_shared<VEC>(sums + a.d + c, n);
        } else {
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            dw[SHARED ? 0 : j][i] += n[i];
            db[SHARED ? 0 : j][i] += cdy[j].get(i);
          }
        }
      }
    }
    if (!AHEAD && row + stride < a.T) load_row(row + stride);
  }
  if (!a.dw && !a.db) return;
  float* to = a.partial + (size_t)blockIdx.x * 2 * a.d;
  if (SHARED) {
    __syncthreads();
    for (int k = threadIdx.x; k < 2 * a.d; k += R) to[k] = sums[k];
  } else {
    float* at = R == 32 ? sums + group * 2 * a.d : to;
#pragma unroll
    for (int j = 0; j < (SHARED ? 1 : C); ++j) {
      const int c = (tid + j * R) * VEC;
      if (c < a.d) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          at[c + i] = dw[j][i];
          at[a.d + c + i] = db[j][i];
        }
      }
    }
    if (R == 32) {
      __syncthreads();
      for (int k = threadIdx.x; k < 2 * a.d; k += 128) {
        float v = sums[k];
        for (int g = 1; g < kRows; ++g) v += sums[g * 2 * a.d + k];
        to[k] = v;
      }
    }
  }
}

// dw and db from the partial sums: 32 columns of [dw | db] per block, 32 threads
// per column over every 32nd partial row, then the 32 in order.
__global__ void __launch_bounds__(1024) layer_norm_grad_sum_kernel(const float* partial, int rows, int d, void* dw,
                                                                   void* db, int w_dtype) {
  __shared__ float part[32][33];
  follow();
  const int c = blockIdx.x * 32 + threadIdx.x;
  float v = 0.f;
  if (c < 2 * d) {
#pragma unroll 4
    for (int r = threadIdx.y; r < rows; r += 32) v += partial[(size_t)r * 2 * d + c];
  }
  part[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  const float t = warp_sum(part[threadIdx.x][threadIdx.y]);  // column threadIdx.y of the block
  int k = blockIdx.x * 32 + threadIdx.y;
  void* to = k < d ? dw : db;
  if (threadIdx.x == 0 && k < 2 * d && to) {
    if (k >= d) k -= d;
    if (w_dtype == MOE_BF16)
      put(static_cast<__nv_bfloat16*>(to) + k, t);
    else
      put(static_cast<float*>(to) + k, t);
  }
}

template <typename ST, int R, int C, int VEC>
cudaError_t launch(const LayerNormGradArgs& a, cudaStream_t st) {
  constexpr int kBlock = R == 32 ? 128 : R, kRows = kBlock / R;
  constexpr int kWidest = R * C * VEC;
  constexpr size_t kMost = kAccShared<ST, R> ? (size_t)2 * kWidest * 4 : R == 32 ? (size_t)8 * kWidest * 4 : 0;
  const auto kernel = layer_norm_grad_kernel<ST, R, C, VEC>;
  const size_t smem = kAccShared<ST, R> ? (size_t)2 * a.d * 4 : R == 32 ? (size_t)8 * a.d * 4 : 0;
  const cudaError_t err = allow(kernel, smem, kMost);
  if (err != cudaSuccess) return err;
  int grid = (a.T + kRows - 1) / kRows;
  if (grid > 128) {
    static const int resident = resident_blocks(kernel, kBlock, kMost);
    if (grid > resident) grid = resident;
    if (grid > kLayerNormPartials) grid = kLayerNormPartials;
  }
  const cudaError_t e = launch_after(kernel, grid, dim3(kBlock), smem, st, a);
  if (e != cudaSuccess || (!a.dw && !a.db)) return e;
  return launch_after(layer_norm_grad_sum_kernel, (2 * a.d + 31) / 32, dim3(32, 32), 0, st, (const float*)a.partial,
                      grid, a.d, a.dw, a.db, a.w_dtype);
}
template <typename ST, int VEC>
cudaError_t by_width(const LayerNormGradArgs& a, cudaStream_t st) {
  if (a.d <= 512) return launch<ST, 32, 16 / VEC, VEC>(a, st);
  if (a.d <= 1024) return launch<ST, 128, 8 / VEC, VEC>(a, st);
  if (a.d <= 2048) return launch<ST, 128, 16 / VEC, VEC>(a, st);
  if (a.d <= 4096) return launch<ST, 256, 16 / VEC, VEC>(a, st);
  if (a.d <= 8192) return launch<ST, 512, 16 / VEC, VEC>(a, st);
  return launch<ST, 1024, 16 / VEC, VEC>(a, st);
}
template <typename ST>
cudaError_t typed(const LayerNormGradArgs& a, cudaStream_t st) {
  return a.d % 8 == 0 ? by_width<ST, 8>(a, st) : by_width<ST, 1>(a, st);
}

}  // namespace

cudaError_t launch_layer_norm_backward(const LayerNormGradArgs& a, cudaStream_t st) {
  return a.dtype == MOE_BF16 ? typed<__nv_bfloat16>(a, st) : typed<float>(a, st);
}

}  // namespace moe
