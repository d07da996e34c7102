// Internal declarations of the layer norm, of tokens sorted by expert and of the
// matrix product with its epilogue: arguments and kernel launchers.
#pragma once

#include "ffn_internal.h"

namespace moe {

// layer_norm.cu
// Widths that the kernels take: 2048 windows of 8 columns, which rows that are not aligned may exceed by 7 columns.
inline bool layer_norm_takes(int d) { return d <= kMaxNormWidth - (d % 8 ? 7 : 0); }
struct LayerNormArgs {
  const void *x, *res, *w, *b;
  void *s, *y;
  int T, d;
  int x_dtype, s_dtype, w_dtype, y_dtype;
  float eps;
};
cudaError_t launch_layer_norm(const LayerNormArgs& a, cudaStream_t st);

// layer_norm_grad.cu
// Blocks of a backward call, each with its own partial gradients of weight and bias.
constexpr int kLayerNormPartials = 608;  // 4 for each of 152 SMs
struct LayerNormGradArgs {
  const void *s, *w, *dy, *ds;
  void *dx, *dw, *db;
  float* partial;  // [kLayerNormPartials][2][d]
  int T, d;
  int dtype, w_dtype;
  float eps;
};
cudaError_t launch_layer_norm_backward(const LayerNormGradArgs& a, cudaStream_t st);

// moe_dispatch.cu
constexpr int kMaxSortExperts = 1024;
struct SortArgs {
  const int32_t* idx;
  int32_t *counts, *offsets, *perm, *slot;
  int picks, k, E;
};
cudaError_t launch_sort_tokens(const SortArgs& a, cudaStream_t st);
struct RowsArgs {
  const void* tokens;      // x, dy or add [T, d]
  const void* rows_in;     // [n_rows, d]
  void* out;               // dispatch, combine's gradient: rows [n_rows, d]; combine: y [T, d]
  const int32_t* slot;     // [T, k]
  const float* w;          // [T, k]
  float* dw;               // [T, k]
  int T, k, d, n_rows;
  int t_dtype, r_dtype;    // of the tokens' side and of the rows
};
cudaError_t launch_dispatch(const RowsArgs& a, cudaStream_t st);
cudaError_t launch_combine_rows(const RowsArgs& a, cudaStream_t st);
cudaError_t launch_combine_backward(const RowsArgs& a, cudaStream_t st);

// linear_gemv.cu: the product with its epilogue for up to four tokens.  Against a stream of tensor-core tiles (us), one
// token: 8192 to 4096 14.5, 15.9; 16384 to 4096 24.5, 26.1; 2048 to 2048 3.4, 6.4.  With more tokens the multiply-adds
// take as long as large weights: T = 4, 2048 to 2048 4.1 against 6.3, 2048 to 4096 7.3 against 7.8, but 4096 to 4096 12.0
// against 10.3 and 8192 to 4096 20.0 against 15.9.
inline bool gemv_tokens(const LinearShape& s) {
  return s.T == 1 || (s.T <= 4 && (long long)s.n * s.k <= 1LL << 23);
}
cudaError_t launch_linear_gemv(const FfnEngine& e, const LinearShape& s, const LinearForwardArgs& a, cudaStream_t st);

// linear_grad.cu: dpre = dy act'(pre) (dpre NULL: not stored), dbias = the sum of its rows (NULL: not wanted)
struct LinearGradArgs {
  const void* dy;
  const uint16_t* pre;
  uint16_t* dpre;
  void* dbias;
  int T, n, dy_dtype, bias_dtype, act;
};
cudaError_t launch_linear_grad(const LinearGradArgs& a, cudaStream_t st);
// For up to kFewTokens tokens the same with dw [n, k] = dpre^T x.  A backward call with gelu, against dw as tensor-core
// tiles (us): 4096 to 4096 T = 1 18, 23, T = 8 22, 25, but T = 12 26, 25; 2048 to 2048 T = 16 12, 15.
constexpr int kFewTokens = 16;
inline bool few_grad_tokens(const LinearShape& s) {
  return s.T <= 8 || (s.T <= kFewTokens && (long long)s.n * s.k < 1LL << 23);
}
cudaError_t launch_linear_few_grad(const LinearGradArgs& a, const void* x, void* dw, int k, cudaStream_t st);

}  // namespace moe
