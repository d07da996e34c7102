// What the layer norm's kernels share.
//
// A row belongs to R threads of one or two windows of 8 neighbouring columns each,
// moved in 16-byte accesses.  Where the width is not a multiple of 8 (ODD) rows are
// not aligned; the windows are then the aligned ones of the whole matrix that cover
// the row, the first and the last with values of the neighbouring rows in them,
// which count as 0 and are not written.  Where a row's first window begins depends
// on the row's number modulo 8 only, and the rows that a thread walks over are a
// multiple of 8 apart: its columns are the same in every row, so that weight and
// gradients stay with the thread.
#pragma once

#include "ops_internal.h"
#include "rows_common.cuh"

namespace moe {

// Blocks of up to 256 threads, several rows each where a row has fewer.
constexpr int ln_rows(int R) { return R < 256 ? 256 / R : 1; }
constexpr int ln_block(int R) { return ln_rows(R) * R; }

// Rows come through a ring in shared memory, filled by asynchronous copies some rows
// ahead; a thread copies the windows that it reads itself, and so waits for its own
// copies alone.

// A thread's windows; the same in every row that it walks over.
template <int R, bool ODD>
struct Windows {
  int head;     // values of the row before in the first window
  int c[2];     // first column (below 0: that many values of the row before)
  bool in[2];   // there is such a window
  bool edge[2];  // with values of other rows
  int d;
  MOE_DEV Windows(int tid, int first_row, int width) {
    d = width;
    head = ODD ? (int)((long long)first_row * width & 7) : 0;
#pragma unroll
    for (int o = 0; o < 2; ++o) {
      c[o] = (tid + o * R) * 8 - head;
      in[o] = c[o] < d;
      edge[o] = ODD && (c[o] < 0 || c[o] + 8 > d);
    }
  }
  MOE_DEV bool has(int o, int i) const { return (unsigned)(c[o] + i) < (unsigned)d; }
  MOE_DEV void mask(int o, F8& f) const {
    if (ODD && edge[o]) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (!has(o, i)) f.v[i] = 0.f;
    }
  }
  // Asynchronous copy of one of the row's windows, where in[o]; `lo` is the row's first value, n the matrix's number of
  // values (past which nothing is read).
  // In shared memory a row lies in planes of 16 bytes per thread, one for each 16-byte piece of a window, so that
  // neighbouring threads' accesses are neighbours; `to` and `from` are this thread's places in a row's first plane.
  template <typename T>
  MOE_DEV void copy(uint32_t to, const T* p, size_t lo, int o, size_t n) const {
    const size_t at = lo + c[o];
    const int left = ODD ? (int)min((size_t)8, n - at) * (int)sizeof(T) : 8 * (int)sizeof(T);
    to += o * R * 8 * (int)sizeof(T);
    copy16(to, p + at, ODD ? min(left, 16) : 16);
    if (sizeof(T) == 4)
      copy16(to + R * 16, ODD && left <= 16 ? p + at : p + at + 4, ODD ? max(left - 16, 0) : 16);
  }
  template <typename T>
  MOE_DEV F8 take(const uint8_t* from, int o) const {
    const uint8_t* at = from + o * R * 8 * (int)sizeof(T);
    if constexpr (sizeof(T) == 2) {
      return load8(reinterpret_cast<const T*>(at));
    } else {
      const float4 a = *reinterpret_cast<const float4*>(at), b = *reinterpret_cast<const float4*>(at + R * 16);
      return F8{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
    }
  }
  template <typename T>
  MOE_DEV void load(Raw<T>& r, const T* p, size_t lo, int o, size_t n) const {
    const T* at = p + lo + c[o];
    if (!ODD || lo + c[o] + 8 <= n) {
      r.load(at);
    } else {
      __align__(16) T t[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) put(t + i, has(o, i) ? to_f(at[i]) : 0.f);
      r.load(t);
    }
  }
  template <typename T>
  MOE_DEV void store(T* p, size_t lo, int o, const F8& f) const {
    T* at = p + lo + c[o];
    if (!ODD || !edge[o]) {
      store8(at, f);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (has(o, i)) put(at + i, f.v[i]);
    }
  }
};

MOE_DEV float param_value(const void* p, int dtype, int c, float otherwise) {
  return !p ? otherwise
         : dtype == MOE_BF16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[c]) : static_cast<const float*>(p)[c];
}
// Weight or bias of a window; `otherwise` without one.
template <int R, bool ODD>
MOE_DEV F8 param_of(const Windows<R, ODD>& win, const void* p, int dtype, int o, float otherwise) {
  F8 f;
  if (!win.in[o] || !p) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f.v[i] = otherwise;
  } else if (ODD) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f.v[i] = win.has(o, i) ? param_value(p, dtype, win.c[o] + i, otherwise) : 0.f;
  } else {
    f = dtype == MOE_BF16 ? load8(static_cast<const __nv_bfloat16*>(p) + win.c[o])
                          : load8(static_cast<const float*>(p) + win.c[o]);
  }
  return f;
}

// Whether rows that are not aligned may be walked over in steps of `stride`: see Windows.
inline bool steps_of_eight(int T, int stride) { return stride >= T || stride % 8 == 0; }

// Sums of four values over a warp, each in every lane: two exchanges leave one value each to a quarter of the warp.
MOE_DEV void warp_sum4(float (&v)[4]) {
  const bool up = (threadIdx.x & 16) != 0, odd = (threadIdx.x & 8) != 0;
  float a = up ? v[2] : v[0], b = up ? v[3] : v[1];
  a += __shfl_xor_sync(0xffffffffu, up ? v[0] : v[2], 16);
  b += __shfl_xor_sync(0xffffffffu, up ? v[1] : v[3], 16);
  float mine = odd ? b : a;
  mine += __shfl_xor_sync(0xffffffffu, odd ? a : b, 8);
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = __shfl_sync(0xffffffffu, mine, i * 8);
}
// Sums over the R threads of a row, in every one of them: the warps' sums meet in
// `red`, another array from one call to the next, so that one barrier per call
// suffices.
template <int R, int N>
struct __align__(16) RowRed {
  float v[ln_rows(R)][N][(R / 32 + 3) / 4 * 4];
};
template <int R, int N>
MOE_DEV void ln_row_sums(float (&v)[N], RowRed<R, N>& red) {
  static_assert(N == 1 || N == 4, "see the sums over a warp");
  if constexpr (N == 4)
    warp_sum4(v);
  else
    v[0] = warp_sum(v[0]);
  if constexpr (R > 32) {
    const int group = threadIdx.x / R, warp = threadIdx.x % R >> 5;
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) red.v[group][i][warp] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < R / 32; w += 4) {
        static_assert(alignof(RowRed<R, N>) >= alignof(float4), "read four at a time");
        const float4 q = *reinterpret_cast<const float4*>(&red.v[group][i][w]);
        s += q.x;
        if (w + 1 < R / 32) s += q.y;
        if (w + 2 < R / 32) s += q.z;
        if (w + 3 < R / 32) s += q.w;
      }
      v[i] = s;
    }
  }
}

// Threads of a row: two windows each, in classes close enough that few are idle (rows that are not aligned may touch one
// window more).
template <template <int> class Launch, typename A>
cudaError_t by_width(const A& a, cudaStream_t st) {
  const int windows = a.d % 8 == 0 ? a.d / 8 : (a.d + 14) / 8;
  if (windows <= 64) return Launch<32>::run(a, st);
  if (windows <= 128) return Launch<64>::run(a, st);
  if (windows <= 192) return Launch<96>::run(a, st);
  if (windows <= 256) return Launch<128>::run(a, st);
  if (windows <= 320) return Launch<160>::run(a, st);
  if (windows <= 384) return Launch<192>::run(a, st);
  if (windows <= 512) return Launch<256>::run(a, st);
  if (windows <= 768) return Launch<384>::run(a, st);
  if (windows <= 1024) return Launch<512>::run(a, st);
  if (windows <= 1088) return Launch<544>::run(a, st);
  return Launch<1024>::run(a, st);
}

}  // namespace moe
