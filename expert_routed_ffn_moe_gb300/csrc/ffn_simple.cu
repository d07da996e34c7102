// The gated feed-forward block's products on the CUDA cores: one 64 x 64 output
// tile per block, fp32 multiply-adds from shared memory.
#include "ffn_internal.h"

namespace moe {
namespace {

enum { kEpiStore, kEpiGateUp };

// Element (row, k) of an operand: bf16 with strides, or mx8 rows.
struct Operand {
  const void* p;
  const uint8_t* scales;  // mx8; NULL for bf16
  long long row_stride, k_stride;
  int rows, K;
  MOE_DEV float at(int r, int k) const {
    if (r >= rows || k >= K) return 0.f;
    if (!scales) {
      const uint16_t v = static_cast<const uint16_t*>(p)[r * row_stride + k * k_stride];
      return __uint_as_float((uint32_t)v << 16);
    }
    uint16_t h;
    const uint16_t q = static_cast<const uint8_t*>(p)[r * row_stride + k];
    uint32_t h2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(q));
    h = (uint16_t)h2;
    float f;
    asm("cvt.f32.f16 %0, %1;" : "=f"(f) : "h"(h));
    const size_t tc = mx_tile_cols(K);
    return f * mx_scale(scales[mx_scale_word(r, k / 128, tc) + k / 32 % 4]);
  }
};

struct Epilogue {
  uint16_t* out;           // kEpiStore: [M, N]; kEpiGateUp: h [M, N]
  uint16_t* pre;           // kEpiGateUp: [M, 2N] or NULL
  uint8_t *codes, *scales; // kEpiGateUp on mx8: h in mx8
  int act;
};

MOE_DEV uint16_t to_bf16(float v) { return __bfloat16_as_ushort(__float2bfloat16_rn(v)); }

// C[m, n] = sum_k A(m, k) B(n, k); kEpiGateUp also with the rows N + n of B.
template <int EPI>
__global__ void __launch_bounds__(256) simple_gemm(Operand A, Operand B, int M, int N, int K, Epilogue ep) {
  __shared__ float as[16][65], bs[16][65], us[EPI == kEpiGateUp ? 16 : 1][65];
  __shared__ float hs[EPI == kEpiGateUp ? 64 : 1][65];
  const int m0 = blockIdx.y * 64, n0 = blockIdx.x * 64;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  float c[4][4] = {}, u[4][4] = {};
  for (int k0 = 0; k0 < K; k0 += 16) {
    for (int i = threadIdx.x; i < 1024; i += 256) {
      const int r = i / 16, k = i % 16;
      as[k][r] = A.at(m0 + r, k0 + k);
      bs[k][r] = n0 + r < N ? B.at(n0 + r, k0 + k) : 0.f;
      if (EPI == kEpiGateUp) us[k][r] = n0 + r < N ? B.at(N + n0 + r, k0 + k) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 16; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          c[i][j] += as[k][ty * 4 + i] * bs[k][tx + 16 * j];
          if (EPI == kEpiGateUp) u[i][j] += as[k][ty * 4 + i] * us[k][tx + 16 * j];
        }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int m = m0 + ty * 4 + i, n = n0 + tx + 16 * j;
      const bool in = m < M && n < N;
      const size_t at = (size_t)m * N + n, pg = (size_t)m * 2 * N + n;
      if (EPI == kEpiStore) {
        if (in) ep.out[at] = to_bf16(c[i][j]);
      } else if (EPI == kEpiGateUp) {
        const float h = act_value(c[i][j], ep.act) * u[i][j];
        hs[ty * 4 + i][tx + 16 * j] = in ? h : 0.f;
        if (in && ep.out) ep.out[at] = to_bf16(h);
        if (in && ep.pre) {
          ep.pre[pg] = to_bf16(c[i][j]);
          ep.pre[pg + N] = to_bf16(u[i][j]);
        }
      }
    }
  if (EPI == kEpiGateUp && ep.codes) {
    __syncthreads();
    const size_t tc = mx_tile_cols(N);
    for (int t = threadIdx.x; t < 128; t += 256) {  // 64 rows x 2 groups
      const int r = t / 2, g = t % 2, m = m0 + r, n = n0 + 32 * g;
      if (m >= M || n >= N) continue;
      uint32_t top = 0;
      for (int i = 0; i < 32; ++i) top = max(top, mag_bits(hs[r][32 * g + i]));
      const uint32_t byte = mx_scale_byte(__uint_as_float(top));
      const float k = mx_inverse_scale(byte);
      for (int i = 0; i < 32; i += 2)
        *reinterpret_cast<uint16_t*>(ep.codes + (size_t)m * N + n + i) =
            (uint16_t)e4m3x2(hs[r][32 * g + i] * k, hs[r][32 * g + i + 1] * k);
      ep.scales[mx_scale_word(m, n / 128, tc) + n / 32 % 4] = (uint8_t)byte;
    }
  }
}

template <int EPI>
cudaError_t gemm(const Operand& A, const Operand& B, int M, int N, int K, const Epilogue& ep, cudaStream_t st) {
  simple_gemm<EPI><<<dim3((N + 63) / 64, (M + 63) / 64), 256, 0, st>>>(A, B, M, N, K, ep);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_simple_forward(const FfnShape& s, bool mx, const FfnForwardArgs& a, const FfnScratch& sc,
                                  cudaStream_t st) {
  Epilogue e1{};
  e1.act = s.act;
  e1.pre = static_cast<uint16_t*>(a.pre);
  if (mx) {
    e1.codes = sc.hq;
    e1.scales = sc.hs;
  } else {
    e1.out = sc.h;
  }
  cudaError_t err = gemm<kEpiGateUp>(Operand{a.x, a.xs, s.d, 1, s.T, s.d}, Operand{a.gate_up, a.gate_up_s, s.d, 1, 2 * s.I, s.d},
                                     s.T, s.I, s.d, e1, st);
  if (err != cudaSuccess) return err;
  Epilogue e2{};
  e2.out = static_cast<uint16_t*>(a.y);
  return gemm<kEpiStore>(Operand{mx ? (const void*)sc.hq : sc.h, mx ? sc.hs : nullptr, s.I, 1, s.T, s.I},
                         Operand{a.down, a.down_s, s.I, 1, s.d, s.I}, s.T, s.d, s.I, e2, st);
}

}  // namespace moe
