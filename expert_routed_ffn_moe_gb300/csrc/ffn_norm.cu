// Root-mean-square norm with the residual's addition, its gradients, and the
// rounding of a matrix to mx8.
//
//   forward   s = x + residual;  y = s * rsqrt(mean(s^2) + eps) * w
//   backward  n = s * rstd, g = dy * w:  dx = rstd * (g - n * mean(g * n)) + ds,
//             dw = sum over rows of dy * n
//
// Both are bound by memory: one pass over the rows, which stay in registers
// between the reduction and the output (s is never read back; above 8192 columns,
// where 1024 threads have 64 registers each, some of it spills: 32-256 bytes a
// thread forward with an fp32 operand, 368-852 backward; odd widths 996 and 1940).
// T = 16384, d = 4096, bf16: 84 us forward, 91 backward, against 79 at the measured
// copy rate; T = 8192, d = 16384: 179 and 351 against 158.  A row belongs
// to R threads, each holding up to two chunks of 8 neighbouring columns
// (16-byte loads of bf16, two of fp32); R follows from the width alone.  Blocks
// walk over rows and ask for the next row before they reduce the present one:
// without that a block waits out the memory's latency once per row, and the
// rows in flight do not cover the bandwidth.  All sums are fp32: a thread's
// columns, then a shuffle tree, then the warps' sums in order.  y is computed
// from the unrounded s and rounded once.
//
// A width that is not a multiple of 8 leaves rows unaligned; the chunks are
// then the aligned 16-byte windows of the whole matrix that cover the row, with
// the neighbours' columns masked, so the loads stay wide (ODD).  The weight is
// not aligned with those windows; it lies in shared memory by (column mod 8),
// where neighbouring threads' columns are neighbours.
#include "ffn_internal.h"

namespace moe {
namespace {

struct F8 {
  float v[8];
};

// The norm's kernels are launched while the kernel before may still run
// (programmatic stream serialization): their blocks come up during its end, and
// read and write nothing before it has finished.
MOE_DEV void follow() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), int grid, dim3 block, size_t smem, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

// A chunk as it lies in memory.
template <typename T>
struct Raw;
template <>
struct Raw<float> {
  float4 a, b;
  MOE_DEV void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  MOE_DEV void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  MOE_DEV F8 get() const { return F8{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}}; }
};
template <>
struct Raw<__nv_bfloat16> {
  uint4 a;
  MOE_DEV void load(const __nv_bfloat16* p) { a = *reinterpret_cast<const uint4*>(p); }
  MOE_DEV void zero() { a = make_uint4(0u, 0u, 0u, 0u); }
  MOE_DEV F8 get() const {
    return F8{{bf16_lo(a.x), bf16_hi(a.x), bf16_lo(a.y), bf16_hi(a.y), bf16_lo(a.z), bf16_hi(a.z), bf16_lo(a.w),
               bf16_hi(a.w)}};
  }
};
template <typename T>
MOE_DEV F8 load8(const T* p) {
  Raw<T> r;
  r.load(p);
  return r.get();
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

// The chunk of 8 columns at e of a matrix of n values; what lies past its end reads 0.
template <bool ODD, typename T>
MOE_DEV void load_raw(Raw<T>& r, const T* p, size_t e, size_t n) {
  if (!ODD || e + 8 <= n) {
    r.load(p + e);
  } else {
    __align__(16) T t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) put(t + i, e + i < n ? to_f(p[e + i]) : 0.f);
    r.load(t);
  }
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

// The sums over the R threads of a row, in every one of them.  `red` is another
// half of its memory from one row to the next, so one barrier per row suffices.
template <int R, int N>
MOE_DEV void row_sums(float (&v)[N], float (*red)[N][32]) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
  if (R == 32) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) (*red)[i][warp] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum(lane < R / 32 ? (*red)[i][lane] : 0.f);
}

// Rows of odd width: where value i of window c of a row that begins r = (its
// first value) mod 8 into the first window has its column in an array [8][pitch]
// by (column mod 8, column / 8): at off(i) + c, off() the same in all threads.
// Only the first and the last window hold values of other rows (not in()); for
// those off(i) + c is some other place of the array, or the one past its end.
struct OddRow {
  int r, pitch, d, chunks;
  MOE_DEV int off(int i) const { return i >= r ? (i - r) * pitch : (i - r + 8) * pitch - 1; }
  MOE_DEV bool edge(int c) const { return c == 0 || c >= chunks - 1; }
  MOE_DEV bool in(int c, int i) const { return (unsigned)(8 * c + i - r) < (unsigned)d; }
};

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
  __shared__ float red[2][1][32];
  extern __shared__ float wsm[];  // ODD: the weight, [8][(d + 7) / 8]
  follow();
  constexpr int kRows = R == 32 ? 4 : 1;
  const int tid = R == 32 ? threadIdx.x & 31 : threadIdx.x;
  const size_t tile_cols = mx_tile_cols(a.d);
  const size_t n = (size_t)a.T * a.d;
  const XT* x_in = static_cast<const XT*>(a.x);
  const ST* r_in = static_cast<const ST*>(a.res);
  ST* s_out = static_cast<ST*>(a.s);
  const int wpitch = (a.d + 7) / 8;
  const int rows = a.y_dtype == MOE_MX8 ? (a.T + 127) / 128 * 128 : a.T;  // (the last scale tile's padding too)
  const int stride = gridDim.x * kRows;
  int row = blockIdx.x * kRows + (R == 32 ? threadIdx.x >> 5 : 0);

  auto load_row = [&](int r, Raw<XT>(&x)[C], Raw<ST>(&res)[C]) {
    const size_t lo = (size_t)r * a.d, c0 = lo / 8;
    const int chunks = (int)((lo + a.d + 7) / 8 - c0);
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const int c = tid + j * R;
      if (c < chunks) {
        load_raw<ODD>(x[j], x_in, (c0 + c) * 8, n);
        if (r_in) load_raw<ODD>(res[j], r_in, (c0 + c) * 8, n);
      } else {
        x[j].zero();
        res[j].zero();
      }
    }
  };
  Raw<XT> x[C];
  Raw<ST> res[C];
#pragma unroll
  for (int j = 0; j < C; ++j) res[j].zero();
  if (row < a.T) load_row(row, x, res);
  F8 w[C];
  auto weight = [&](int k) {
    return a.w_dtype == MOE_BF16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.w)[k])
                                 : static_cast<const float*>(a.w)[k];
  };
  if (ODD) {
    for (int k = threadIdx.x; k < a.d; k += blockDim.x) wsm[(k & 7) * wpitch + (k >> 3)] = weight(k);
    __syncthreads();
  } else {
#pragma unroll
    for (int j = 0; j < C; ++j)
      if ((tid + j * R) * 8 < a.d)
        w[j] = a.w_dtype == MOE_BF16 ? load8(static_cast<const __nv_bfloat16*>(a.w) + (tid + j * R) * 8)
                                     : load8(static_cast<const float*>(a.w) + (tid + j * R) * 8);
  }

  for (int it = 0; row < rows; row += stride, it ^= 1) {
    if (row >= a.T) {  // (a row of the padding: R threads leave together)
      for (size_t q = tid; q < tile_cols; q += R)
        *reinterpret_cast<uint32_t*>(a.scales + mx_scale_word(row, q, tile_cols)) = 0u;
      continue;
    }
    const size_t lo = (size_t)row * a.d, hi = lo + a.d, c0 = lo / 8;
    const int chunks = (int)((hi + 7) / 8 - c0);
    const OddRow odd{(int)(lo & 7), wpitch, a.d, chunks};
    F8 s[C];
    float sum[1] = {0.f};
#pragma unroll
    for (int j = 0; j < C; ++j) {
      s[j] = x[j].get();
      const F8 r = res[j].get();
#pragma unroll
      for (int i = 0; i < 8; ++i) s[j].v[i] += r.v[i];
      if (ODD && odd.edge(tid + j * R)) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (!odd.in(tid + j * R, i)) s[j].v[i] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[0] += s[j].v[i] * s[j].v[i];
    }
    if (row + stride < a.T) load_row(row + stride, x, res);  // in flight while this row is finished
    if (s_out) {
#pragma unroll
      for (int j = 0; j < C; ++j)
        if (tid + j * R < chunks) store_chunk<ST, ODD>(s_out, (c0 + tid + j * R) * 8, lo, hi, s[j]);
    }
    row_sums<R>(sum, &red[it]);
    const float rstd = rsqrtf(sum[0] / (float)a.d + a.eps);
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const int c = tid + j * R;
      const bool in = c < chunks;
      const size_t e = (c0 + c) * 8;
      F8 y;
      if (ODD) {
#pragma unroll
        for (int i = 0; i < 8; ++i) y.v[i] = in ? s[j].v[i] * rstd * wsm[odd.off(i) + c] : 0.f;
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) y.v[i] = in ? s[j].v[i] * rstd * w[j].v[i] : 0.f;
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
}

// Gradients.  A block walks rows as above and leaves the
// weight gradient of all of them in a row of `partial`; norm_grad_sum_kernel
// adds those up in a fixed order (no atomics: the result does not depend on
// timing).  A thread has the same columns in every row and keeps their gradient
// in registers; where the width is not a multiple of 8 (ODD) the windows move
// from row to row, and the gradient lies in shared memory like the weight: a
// column has one thread per row, and the barrier of the row's sums stands
// between one row's additions and the next's.
template <typename ST, int R, int C, bool ODD>
__global__ void __launch_bounds__(R == 32 ? 128 : R) norm_grad_kernel(NormGradArgs a) {
  __shared__ float red[2][2][32];
  // ODD: the weight, [8][(d + 7) / 8], then the gradient likewise (R == 32: of each warp); else R == 32: the warps'
  // gradients at the end, [4][d]
  extern __shared__ float wsm[];
  follow();
  constexpr int kRows = R == 32 ? 4 : 1;
  const int tid = R == 32 ? threadIdx.x & 31 : threadIdx.x, group = R == 32 ? threadIdx.x >> 5 : 0;
  const int first = blockIdx.x * kRows + group, stride = gridDim.x * kRows;
  const ST* s_in = static_cast<const ST*>(a.s);
  const ST* dy_in = static_cast<const ST*>(a.dy);
  const ST* ds_in = static_cast<const ST*>(a.ds);
  ST* dx = static_cast<ST*>(a.dx);
  const size_t n = (size_t)a.T * a.d;
  const int wpitch = (a.d + 7) / 8;
  float* acc_sm = wsm + 8 * wpitch * (1 + group);
  auto place = [&](int k) { return (k & 7) * wpitch + (k >> 3); };
  auto weight = [&](int k) {
    return a.w_dtype == MOE_BF16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.w)[k])
                                 : static_cast<const float*>(a.w)[k];
  };

  Raw<ST> rs[C], rdy[C], rds[C];
#pragma unroll
  for (int j = 0; j < C; ++j) rds[j].zero();
  auto load_all = [&](int row) {
    const size_t lo = (size_t)row * a.d, c0 = lo / 8;
    const int chunks = (int)((lo + a.d + 7) / 8 - c0);
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const int c = tid + j * R;
      if (c < chunks) {
        load_raw<ODD>(rs[j], s_in, (c0 + c) * 8, n);
        load_raw<ODD>(rdy[j], dy_in, (c0 + c) * 8, n);
        if (ds_in) load_raw<ODD>(rds[j], ds_in, (c0 + c) * 8, n);
      } else {
        rs[j].zero();
        rdy[j].zero();
      }
    }
  };
  if (first < a.T) load_all(first);
  F8 acc[C], w[C];
  if (ODD) {
    for (int k = threadIdx.x; k < a.d; k += blockDim.x) wsm[place(k)] = weight(k);
    for (int k = tid; k < 8 * wpitch; k += R) acc_sm[k] = 0.f;
    __syncthreads();
  } else {
#pragma unroll
    for (int j = 0; j < C; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int k = (tid + j * R) * 8 + i;
        acc[j].v[i] = 0.f;
        w[j].v[i] = k < a.d ? weight(k) : 0.f;
      }
  }
  for (int row = first, it = 0; row < a.T; row += stride, it ^= 1) {
    const size_t lo = (size_t)row * a.d, hi = lo + a.d, c0 = lo / 8;
    const int chunks = (int)((hi + 7) / 8 - c0);
    const OddRow odd{(int)(lo & 7), wpitch, a.d, chunks};
    Raw<ST> cs[C], cdy[C], cds[C];
    float sum[2] = {0.f, 0.f};  // s^2 and s dy w
#pragma unroll
    for (int j = 0; j < C; ++j) {
      cs[j] = rs[j];
      cdy[j] = rdy[j];
      cds[j] = rds[j];
      F8 s = cs[j].get(), dy = cdy[j].get();
      const int c = tid + j * R;
      if (ODD) {
        if (c < chunks) {
#pragma unroll
          for (int i = 0; i < 8; ++i) w[j].v[i] = wsm[odd.off(i) + c];
        }
        if (odd.edge(c)) {  // (a neighbour's value may be anything)
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (!odd.in(c, i)) s.v[i] = dy.v[i] = w[j].v[i] = 0.f;
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        sum[0] += s.v[i] * s.v[i];
        sum[1] += s.v[i] * dy.v[i] * w[j].v[i];
      }
    }
    if (row + stride < a.T) load_all(row + stride);  // in flight while this row is finished
    row_sums<R>(sum, &red[it]);
    const float rstd = rsqrtf(sum[0] / (float)a.d + a.eps);
    const float k_mean = sum[1] * rstd / (float)a.d;  // mean(g n)
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const F8 s = cs[j].get(), dy = cdy[j].get();
      const int c = tid + j * R;
      F8 o = cds[j].get();
      if (ODD) {  // all loads before the stores: they lie in the same memory
        if (!odd.edge(c)) {
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[j].v[i] = acc_sm[odd.off(i) + c];
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[j].v[i] = odd.in(c, i) ? acc_sm[odd.off(i) + c] : 0.f;
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float nrm = s.v[i] * rstd;
        o.v[i] += rstd * (dy.v[i] * w[j].v[i] - nrm * k_mean);
        acc[j].v[i] += dy.v[i] * nrm;
      }
      if (ODD) {
        if (!odd.edge(c)) {
#pragma unroll
          for (int i = 0; i < 8; ++i) acc_sm[odd.off(i) + c] = acc[j].v[i];
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (odd.in(c, i)) acc_sm[odd.off(i) + c] = acc[j].v[i];
        }
      }
      if (dx && c < chunks) store_chunk<ST, ODD>(dx, (c0 + c) * 8, lo, hi, o);
    }
    if (ODD && R == 32) __syncwarp();
  }
  if (!a.dw) return;
  float* to = a.partial + (size_t)blockIdx.x * a.d;
  if (ODD || R == 32) {
    if (!ODD) {
#pragma unroll
      for (int j = 0; j < C; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if ((tid + j * R) * 8 < a.d) wsm[group * a.d + (tid + j * R) * 8 + i] = acc[j].v[i];
    }
    __syncthreads();
    for (int k = threadIdx.x; k < a.d; k += blockDim.x) {
      const float* from = ODD ? wsm + 8 * wpitch + place(k) : wsm + k;
      float v = from[0];
      for (int g = 1; g < kRows; ++g) v += from[g * (ODD ? 8 * wpitch : a.d)];
      to[k] = v;
    }
  } else {
#pragma unroll
    for (int j = 0; j < C; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int k = (tid + j * R) * 8 + i;
        if (k < a.d) to[k] = acc[j].v[i];
      }
  }
}

// dw[c] = the sum of the partial gradients: 32 columns per block, 32 threads
// per column over every 32nd partial row, then the 32 in order.
__global__ void __launch_bounds__(1024) norm_grad_sum_kernel(const float* partial, int rows, int d, void* dw,
                                                             int w_dtype) {
  __shared__ float part[32][33];
  follow();
  const int c = blockIdx.x * 32 + threadIdx.x;
  float v = 0.f;
  if (c < d) {
#pragma unroll 4
    for (int r = threadIdx.y; r < rows; r += 32) v += partial[(size_t)r * d + c];
  }
  part[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  const float t = warp_sum(part[threadIdx.x][threadIdx.y]);  // column threadIdx.y of the block
  const int k = blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x == 0 && k < d) {
    if (w_dtype == MOE_BF16)
      static_cast<__nv_bfloat16*>(dw)[k] = __float2bfloat16_rn(t);
    else
      static_cast<float*>(dw)[k] = t;
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

// Blocks that walk the rows: as many as are resident on the device's SMs.
template <typename K>
int resident_blocks(K kernel, int block, size_t smem) {
  int dev = 0, sms = 1, per = 1;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, block, smem) != cudaSuccess || per < 1) per = 1;
  return sms * per;
}

// Shared memory of the kernels for rows of width d (the weight, and the gradient's `copies`; see OddRow), and of the
// widest rows that R threads of C chunks take.
constexpr size_t odd_bytes(int d, int copies) { return (size_t)(d + 7) / 8 * 8 * 4 * copies + 4; }
constexpr int widest(int R, int C) { return R * C * 8 < kMaxNormWidth ? R * C * 8 : kMaxNormWidth; }
// A kernel's limit on shared memory belongs to all its launches, which threads of the host may issue side by side: it
// is set for the widest rows, never lower for narrower ones.
template <typename K>
cudaError_t allow(K kernel, size_t smem, size_t most) {
  return smem <= 48 * 1024
             ? cudaSuccess
             : cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
}

template <typename XT, typename ST, int R, int C, bool ODD>
cudaError_t norm_launch(const NormArgs& a, cudaStream_t st) {
  constexpr int kBlock = R == 32 ? 128 : R, kRows = kBlock / R;
  const auto kernel = norm_kernel<XT, ST, R, C, ODD>;
  const size_t smem = ODD ? odd_bytes(a.d, 1) : 0;
  const cudaError_t err = allow(kernel, smem, odd_bytes(widest(R, C), 1));
  if (err != cudaSuccess) return err;
  const int rows = a.y_dtype == MOE_MX8 ? (a.T + 127) / 128 * 128 : a.T;
  int grid = (rows + kRows - 1) / kRows;
  // (a grid of fewer blocks than SMs needs no look at what is resident; without the weight in shared memory the answer
  // is one number per kernel)
  if (grid > 128) {
    int most;
    if constexpr (ODD) {
      most = resident_blocks(kernel, kBlock, smem);
    } else {
      static const int resident = resident_blocks(kernel, kBlock, 0);
      most = resident;
    }
    if (grid > most) grid = most;
  }
  return launch_after(kernel, grid, dim3(kBlock), smem, st, a);
}
// Threads per row: one or two chunks of 8 columns each.
template <typename XT, typename ST, bool ODD>
cudaError_t norm_width(const NormArgs& a, cudaStream_t st) {
  const int chunks = ODD ? (a.d + 7) / 8 + 1 : a.d / 8;  // an unaligned row may touch one window more
  if (chunks <= 32) return norm_launch<XT, ST, 32, 1, ODD>(a, st);
  if (chunks <= 64) return norm_launch<XT, ST, 32, 2, ODD>(a, st);
  if (chunks <= 128) return norm_launch<XT, ST, 128, 1, ODD>(a, st);
  if (chunks <= 256) return norm_launch<XT, ST, 128, 2, ODD>(a, st);
  if (chunks <= 512) return norm_launch<XT, ST, 256, 2, ODD>(a, st);
  if (chunks <= 1024) return norm_launch<XT, ST, 512, 2, ODD>(a, st);
  if (chunks <= 2048) return norm_launch<XT, ST, 1024, 2, ODD>(a, st);
  if constexpr (ODD) return norm_launch<XT, ST, 1024, 3, true>(a, st);  // the widest odd rows
  return cudaErrorInvalidValue;
}
template <typename XT, typename ST>
cudaError_t norm_typed(const NormArgs& a, cudaStream_t st) {
  return a.d % 8 == 0 ? norm_width<XT, ST, false>(a, st) : norm_width<XT, ST, true>(a, st);
}

template <typename ST, int R, int C, bool ODD>
cudaError_t grad_launch(const NormGradArgs& a, cudaStream_t st) {
  constexpr int kBlock = R == 32 ? 128 : R, kRows = kBlock / R;
  const auto kernel = norm_grad_kernel<ST, R, C, ODD>;
  const size_t smem = ODD ? odd_bytes(a.d, 1 + kRows) : R == 32 ? (size_t)a.d * 4 * kRows : 0;
  const cudaError_t err = allow(kernel, smem, odd_bytes(widest(R, C), 1 + kRows));
  if (err != cudaSuccess) return err;
  int grid = (a.T + kRows - 1) / kRows;
  if (grid > 128) {
    int most;
    if constexpr (ODD) {
      most = resident_blocks(kernel, kBlock, smem);
    } else {
      static const int resident = resident_blocks(kernel, kBlock, R == 32 ? 512 * 4 * kRows : 0);  // (the widest)
      most = resident;
    }
    if (most > kNormPartials) most = kNormPartials;
    if (grid > most) grid = most;
  }
  const cudaError_t e = launch_after(kernel, grid, dim3(kBlock), smem, st, a);
  if (e != cudaSuccess || !a.dw) return e;
  return launch_after(norm_grad_sum_kernel, (a.d + 31) / 32, dim3(32, 32), 0, st, (const float*)a.partial, grid, a.d,
                      a.dw, a.w_dtype);
}
template <typename ST, bool ODD>
cudaError_t grad_width(const NormGradArgs& a, cudaStream_t st) {
  const int chunks = ODD ? (a.d + 7) / 8 + 1 : a.d / 8;
  if (chunks <= 32) return grad_launch<ST, 32, 1, ODD>(a, st);
  if (chunks <= 64) return grad_launch<ST, 32, 2, ODD>(a, st);
  if (chunks <= 128) return grad_launch<ST, 128, 1, ODD>(a, st);
  if (chunks <= 256) return grad_launch<ST, 128, 2, ODD>(a, st);
  if (chunks <= 512) return grad_launch<ST, 256, 2, ODD>(a, st);
  if (chunks <= 1024) return grad_launch<ST, 512, 2, ODD>(a, st);
  if (chunks <= 2048) return grad_launch<ST, 1024, 2, ODD>(a, st);
  if constexpr (ODD) return grad_launch<ST, 1024, 3, true>(a, st);  // the widest odd rows
  return cudaErrorInvalidValue;
}
template <typename ST>
cudaError_t grad_typed(const NormGradArgs& a, cudaStream_t st) {
  return a.d % 8 == 0 ? grad_width<ST, false>(a, st) : grad_width<ST, true>(a, st);
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
