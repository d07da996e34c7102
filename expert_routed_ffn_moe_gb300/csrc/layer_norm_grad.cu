// Gradients of the layer norm.
//
//   c = s - mean(s), rstd = rsqrt(mean(c^2) + eps), n = c rstd, g = dy w
//   dx = rstd * (g - mean(g) - n * mean(g n)) + ds
//   dw = sum over the rows of dy n,  db = sum over the rows of dy
//
// Bound by memory: one pass over s, dy and ds.  mean(s) and mean(g) come from one
// sum over the row's threads, mean(c^2) and mean(g c) from a second.  The second sum
// of a row goes with the first of the next one, so that a row costs one barrier:
//   B(i)      c and g of row i; its squares and products
//   A(i + 1)  the sums of row i + 1, which is read again in its turn
//   barrier
//   C(i)      dx, and what row i adds to dw and db
// A thread has the same columns in every row and keeps their dw and db in registers.
// A block leaves the sums over its rows in `partial`, which a second kernel adds up in
// a fixed order: no atomics, the result does not depend on timing.
#include "layer_norm.cuh"

namespace moe {
namespace {

// Operands that come through the ring (s and dy, and ds where that leaves room for a row more than the two in work), and
// its rows; two blocks of 256 threads share an SM.
template <typename T, int R>
constexpr int kOperands = R < 1024 ? 3 : 2;
template <typename T, int R>
constexpr int kStagesOf = [] {
  const int row = ln_rows(R) * 16 * R * (int)sizeof(T) * kOperands<T, R>, most = (R <= 512 ? 220 / (512 / ln_block(R)) - 2 : 220) * 1024 / row;
  return most < 4 ? most : 4;
}();

template <typename ST, int R, bool ODD>
__global__ void __launch_bounds__(ln_block(R), R <= 512 ? 512 / ln_block(R) : 1) layer_norm_grad_kernel(LayerNormGradArgs a) {
  constexpr int kRows = ln_rows(R), S = kStagesOf<ST, R>, kOps = kOperands<ST, R>;
  constexpr int kSlot = 16 * R * (int)sizeof(ST);  // bytes of a row
  constexpr bool AHEAD = S >= 3;    // the next row's sums go with this one's
  constexpr bool CACHE = R < 1024;  // weight, c and g in registers (else read again)
  __shared__ RowRed<R, 4> red[2];
  extern __shared__ float4 ring4[];  // [kRows][S][kOps] rows; at the end [kRows][2][16 R] sums
  uint8_t* ring = reinterpret_cast<uint8_t*>(ring4);
  follow();
  const int tid = threadIdx.x % R, group = threadIdx.x / R;
  const int stride = gridDim.x * kRows, first = blockIdx.x * kRows + group;
  const Windows<R, ODD> win(tid, first, a.d);
  const size_t n = (size_t)a.T * a.d;
  const bool with_ds = a.ds && a.dx;
  const float inv_d = 1.0f / (float)a.d;
  uint8_t* here = ring + group * S * kOps * kSlot + tid * 16;
  auto from = [&](int k) { return static_cast<const ST*>(k == 0 ? a.s : k == 1 ? a.dy : a.ds); };

  auto issue = [&](int it, int slot) {  // the copies of the group's it-th row
    const long long row = first + (long long)it * stride;
    if (row < a.T) {
      const size_t lo = (size_t)row * a.d;
      const uint32_t to = smem_u32(here) + slot * kOps * kSlot;
#pragma unroll
      for (int k = 0; k < kOps; ++k) {
        if (k == 2 && !with_ds) break;
#pragma unroll
        for (int o = 0; o < 2; ++o)
          if (win.in[o]) win.copy(to + k * kSlot, from(k), lo, o, n);
      }
    }
    copies_end();
  };
  auto value = [&](int slot, int k, int o) {
    F8 f = win.template take<ST>(here + (slot * kOps + k) * kSlot, o);
    win.mask(o, f);
    return f;
  };

#pragma unroll
  for (int i = 0; i < S; ++i) issue(i, i);
  F8 dw[2], db[2], w[2];
#pragma unroll
  for (int o = 0; o < 2; ++o) {
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[o].v[i] = db[o].v[i] = 0.f;
    if (CACHE) w[o] = param_of(win, a.w, a.w_dtype, o, 1.f);
  }
  auto grad = [&](int slot, int o) {  // g = dy w
    F8 y = value(slot, 1, o);
    const F8 wo = CACHE ? w[o] : param_of(win, a.w, a.w_dtype, o, 1.f);
#pragma unroll
    for (int i = 0; i < 8; ++i) y.v[i] *= wo.v[i];
    return y;
  };
  // A: the sums of s and g
  auto first_sums = [&](int row, int slot, float& s, float& g) {
    s = g = 0.f;
#pragma unroll
    for (int o = 0; o < 2; ++o)
      if (win.in[o] && row < a.T) {
        const F8 x = value(slot, 0, o), y = grad(slot, o);
#pragma unroll
        for (int i = 0; i < 8; ++i) s += x.v[i], g += y.v[i];
      }
  };

  float sum[4] = {0.f, 0.f, 0.f, 0.f};  // c^2 and g c of this row, s and g of the next
  int base = blockIdx.x * kRows, slot = 0, parity = 0;
  copies_wait<S - 1>();
  first_sums(base + group, 0, sum[2], sum[3]);
  ln_row_sums<R>(sum, red[1]);
  for (int it = 0; base < a.T; base += stride, ++it) {
    const int row = base + group;
    const bool live = kRows == 1 || row < a.T;
    const size_t lo = (size_t)row * a.d;
    const int next = slot + 1 == S ? 0 : slot + 1;
    const float mean = sum[2] * inv_d, g_mean = sum[3] * inv_d;
    F8 c[2], g[2];
    Raw<ST> late[2];  // ds where the ring does not hold it
    sum[0] = sum[1] = 0.f;
    auto centred = [&](int o) {
      c[o] = value(slot, 0, o);
      g[o] = grad(slot, o);
#pragma unroll
      for (int i = 0; i < 8; ++i) c[o].v[i] -= mean;
      win.mask(o, c[o]);
    };
#pragma unroll
    for (int o = 0; o < 2; ++o)
      if (win.in[o] && live) {
        if (kOps == 2 && with_ds) win.load(late[o], from(2), lo, o, n);
        centred(o);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          sum[0] += c[o].v[i] * c[o].v[i];
          sum[1] += g[o].v[i] * c[o].v[i];
        }
      }
    if (AHEAD) {
      copies_wait<AHEAD ? S - 2 : 0>();
      first_sums(row + stride, next, sum[2], sum[3]);
    }
    ln_row_sums<R>(sum, red[parity]);
    parity ^= 1;
    const float rstd = rsqrtf(sum[0] * inv_d + a.eps);
    // dx = rstd g - rstd mean(g) - c rstd^2 mean(g n) + ds
    const float shift = -rstd * g_mean, slope = -rstd * rstd * (sum[1] * rstd * inv_d);
#pragma unroll
    for (int o = 0; o < 2; ++o)
      if (win.in[o] && live) {
        if (!CACHE) centred(o);
        const F8 y = value(slot, 1, o);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          dw[o].v[i] = fmaf(y.v[i], c[o].v[i] * rstd, dw[o].v[i]);
          db[o].v[i] += y.v[i];
        }
        if (a.dx) {
#pragma unroll
          for (int i = 0; i < 8; ++i) g[o].v[i] = fmaf(rstd, g[o].v[i], fmaf(slope, c[o].v[i], shift));
          if (with_ds) {
            const F8 e = kOps == 2 ? late[o].get() : value(slot, 2, o);
#pragma unroll
            for (int i = 0; i < 8; ++i) g[o].v[i] += e.v[i];
          }
          win.store(static_cast<ST*>(a.dx), lo, o, g[o]);
        }
      }
    issue(it + S, slot);
    slot = next;
    if (!AHEAD) {
      copies_wait<S - 1>();
      sum[0] = sum[1] = 0.f;
      first_sums(row + stride, slot, sum[2], sum[3]);
      ln_row_sums<R>(sum, red[parity]);
      parity ^= 1;
    }
  }
  copies_wait<0>();
  if (!a.dw && !a.db) return;
  // The groups' sums side by side, by window, then added up and written by column.
  float* sums = reinterpret_cast<float*>(ring4);
  __syncthreads();  // (the ring is done with)
#pragma unroll
  for (int o = 0; o < 2; ++o) {
    float* at = sums + group * 32 * R + (tid + o * R) * 8;
    store8(at, dw[o]);
    store8(at + 16 * R, db[o]);
  }
  __syncthreads();
  float* to = a.partial + (size_t)blockIdx.x * 2 * a.d;
  for (int k = threadIdx.x; k < 2 * a.d; k += ln_block(R)) {
    const int half = k >= a.d, c = k - half * a.d;
    float v = 0.f;
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int head = ODD ? (int)((long long)(blockIdx.x * kRows + r) * a.d & 7) : 0;
      v += sums[r * 32 * R + half * 16 * R + c + head];
    }
    if (gridDim.x > 1) {
      to[k] = v;
    } else if (void* out = half ? a.db : a.dw) {  // the only block's sums: no second kernel
      if (a.w_dtype == MOE_BF16)
        put(static_cast<__nv_bfloat16*>(out) + c, v);
      else
        put(static_cast<float*>(out) + c, v);
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
    constexpr int kBatch = 10;  // in flight at once: 304 partial rows
    for (int r0 = threadIdx.y; r0 < rows; r0 += 32 * kBatch) {
      float x[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) x[i] = r0 + 32 * i < rows ? partial[(size_t)(r0 + 32 * i) * 2 * d + c] : 0.f;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) v += x[i];
    }
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

template <typename ST, bool ODD>
struct Backward {
  template <int R>
  struct Launch {
    static cudaError_t run(const LayerNormGradArgs& a, cudaStream_t st) {
      constexpr int kBlock = ln_block(R), kRows = ln_rows(R);
      constexpr size_t per = kStagesOf<ST, R> * kOperands<ST, R> * sizeof(ST), smem = (size_t)kRows * 16 * R * per;
      static_assert(kStagesOf<ST, R> >= 1 && smem <= 224 * 1024 && per >= 8, "the ring; the sums of two rows of fp32 in it");
      const auto kernel = layer_norm_grad_kernel<ST, R, ODD>;
      static std::atomic<uint64_t> allowed{0};
      const cudaError_t err = allow_once(kernel, smem, allowed);
      if (err != cudaSuccess) return err;
      int grid = (a.T + kRows - 1) / kRows;
      if (grid > 128) {
        static ByDevice known;
        const int resident = min(resident_blocks(kernel, kBlock, smem, known), kLayerNormPartials) / 8 * 8;
        if (grid > resident) grid = resident;
      }
      if (ODD && !steps_of_eight(a.T, grid * kRows)) return cudaErrorInvalidValue;
      const cudaError_t e = launch_after(kernel, grid, dim3(kBlock), smem, st, a);
      if (e != cudaSuccess || (!a.dw && !a.db) || grid == 1) return e;
      return launch_after(layer_norm_grad_sum_kernel, (2 * a.d + 31) / 32, dim3(32, 32), 0, st, (const float*)a.partial,
                          grid, a.d, a.dw, a.db, a.w_dtype);
    }
  };
};
template <typename ST>
cudaError_t typed(const LayerNormGradArgs& a, cudaStream_t st) {
  return a.d % 8 == 0 ? by_width<Backward<ST, false>::template Launch>(a, st)
                      : by_width<Backward<ST, true>::template Launch>(a, st);
}

}  // namespace

cudaError_t launch_layer_norm_backward(const LayerNormGradArgs& a, cudaStream_t st) {
  return a.dtype == MOE_BF16 ? typed<__nv_bfloat16>(a, st) : typed<float>(a, st);
}

}  // namespace moe
