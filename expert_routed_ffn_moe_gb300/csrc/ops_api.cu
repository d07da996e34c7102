// C ABI of the layer norm, of tokens sorted by expert and back, and of the matrix
// product with its epilogue: argument checking, the product's context and the
// kernels of each call.  Declarations and the full contract are in include/moe.h.
#include <new>

#include <nvtx3/nvToolsExt.h>

#include "ops_internal.h"

using namespace moe;

struct moe_linear {
  moe_linear_config cfg;
  void* block = nullptr;  // the single device allocation holding the workspace
  uint16_t* dpre = nullptr;
  FfnEngine eng{};
  long long launches = 0;
};

namespace {

constexpr long long kDefaultSpinNs = 1000000000LL;  // 1 s
constexpr int kMaxRows = 1 << 30;  // a row's number plus a grid of rows stays an int

bool stream_dtype(int t) { return t == MOE_F32 || t == MOE_BF16; }
int cuda_code(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }
template <typename... P>
bool aligned16(P... p) {
  return ((reinterpret_cast<uintptr_t>(p) | ...) & 15u) == 0;
}

struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
};

// Sizes that dispatch, combine and its gradient share; MOE_OK where they can run.
int check_rows(int T, int top_k, int d, int n_rows, int t_dtype, int r_dtype) {
  if (T < 0 || top_k < 1 || d <= 0 || n_rows < 0 || !stream_dtype(t_dtype) || !stream_dtype(r_dtype)) return MOE_ERR_ARG;
  if (top_k > 32 || d > (1 << 24) || (long long)T * top_k > kMaxRows || (long long)T * ((d + 255) / 256) > kMaxRows)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

}  // namespace

extern "C" {

// ------------------------------------------------------------------ layer norm
int moe_layer_norm(const void* x, int x_dtype, const void* residual, int s_dtype, const void* weight, const void* bias,
                   int w_dtype, int T, int d, float eps, void* s_out, void* y, int y_dtype, void* stream) {
  if (T < 0 || d <= 0 || !stream_dtype(x_dtype) || !stream_dtype(s_dtype) || !stream_dtype(w_dtype) ||
      !stream_dtype(y_dtype) || !(eps >= 0.f))
    return MOE_ERR_ARG;
  if (!layer_norm_takes(d) || T > kMaxRows) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!x || !y) return MOE_ERR_ARG;
  if (!aligned16(x, residual, weight, bias, s_out, y)) return MOE_ERR_ALIGN;
  const NvtxRange range("moe_layer_norm");
  const LayerNormArgs a{x, residual, weight, bias, s_out, y, T, d, x_dtype, s_dtype, w_dtype, y_dtype, eps};
  return cuda_code(launch_layer_norm(a, static_cast<cudaStream_t>(stream)));
}

long long moe_layer_norm_workspace(int d) { return d <= 0 ? 0 : (long long)kLayerNormPartials * 2 * d * 4; }

int moe_layer_norm_backward(const void* s, const void* weight, const void* dy, const void* ds, int dtype, int w_dtype,
                            int T, int d, float eps, void* dx, void* dweight, void* dbias, void* workspace,
                            void* stream) {
  if (T < 0 || d <= 0 || !stream_dtype(dtype) || !stream_dtype(w_dtype) || !(eps >= 0.f)) return MOE_ERR_ARG;
  if (!layer_norm_takes(d) || T > kMaxRows) return MOE_ERR_UNSUPPORTED;
  const bool sums = dweight || dbias;
  // (without rows dx is a tensor of no values, which may have no address)
  if (T > 0 && ((!dx && !sums) || !s || !dy || (sums && !workspace))) return MOE_ERR_ARG;
  if (!aligned16(s, weight, dy, ds, dx, dweight, dbias, workspace)) return MOE_ERR_ALIGN;
  const NvtxRange range("moe_layer_norm_backward");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (T == 0) {  // no rows: the gradients of weight and bias are sums of nothing
    const size_t n = (size_t)d * (w_dtype == MOE_BF16 ? 2 : 4);
    cudaError_t e = cudaSuccess;
    if (dweight) e = cudaMemsetAsync(dweight, 0, n, st);
    if (e == cudaSuccess && dbias) e = cudaMemsetAsync(dbias, 0, n, st);
    return cuda_code(e);
  }
  const LayerNormGradArgs a{s, weight, dy, ds, dx, dweight, dbias, static_cast<float*>(workspace), T, d, dtype, w_dtype,
                            eps};
  return cuda_code(launch_layer_norm_backward(a, st));
}

// ------------------------------------------------------------------ tokens sorted by expert
int moe_sort_tokens(const int32_t* idx, int T, int top_k, int n_experts, int32_t* counts, int32_t* offsets,
                    int32_t* perm, int32_t* slot, void* stream) {
  if (T < 0 || top_k < 1 || n_experts < 1) return MOE_ERR_ARG;
  if (top_k > 32 || n_experts > kMaxSortExperts || (long long)T * top_k > kMaxRows) return MOE_ERR_UNSUPPORTED;
  if (T > 0 && !idx) return MOE_ERR_ARG;
  if (!aligned16(idx, counts, offsets, perm, slot)) return MOE_ERR_ALIGN;
  if (T == 0 && !counts && !offsets) return MOE_OK;
  const NvtxRange range("moe_sort_tokens");
  const SortArgs a{idx, counts, offsets, perm, slot, T * top_k, top_k, n_experts};
  return cuda_code(launch_sort_tokens(a, static_cast<cudaStream_t>(stream)));
}

int moe_dispatch(const void* x, int x_dtype, const int32_t* slot, int T, int top_k, int d, void* rows, int rows_dtype,
                 int n_rows, void* stream) {
  const int code = check_rows(T, top_k, d, n_rows, x_dtype, rows_dtype);
  if (code != MOE_OK || T == 0) return code;
  if (!x || !slot || (n_rows > 0 && !rows)) return MOE_ERR_ARG;
  if (!aligned16(x, slot, rows)) return MOE_ERR_ALIGN;
  if (n_rows == 0) return MOE_OK;
  const NvtxRange range("moe_dispatch");
  RowsArgs a{};
  a.tokens = x;
  a.out = rows;
  a.slot = slot;
  a.T = T, a.k = top_k, a.d = d, a.n_rows = n_rows;
  a.t_dtype = x_dtype, a.r_dtype = rows_dtype;
  return cuda_code(launch_dispatch(a, static_cast<cudaStream_t>(stream)));
}

int moe_combine(const void* rows, int rows_dtype, int n_rows, const int32_t* slot, const float* w, int T, int top_k,
                int d, const void* add, void* y, int y_dtype, void* stream) {
  const int code = check_rows(T, top_k, d, n_rows, y_dtype, rows_dtype);
  if (code != MOE_OK || T == 0) return code;
  if (!slot || !y || (n_rows > 0 && !rows)) return MOE_ERR_ARG;
  if (!aligned16(rows, slot, w, add, y)) return MOE_ERR_ALIGN;
  const NvtxRange range("moe_combine");
  RowsArgs a{};
  a.tokens = add;
  a.rows_in = rows;
  a.out = y;
  a.slot = slot;
  a.w = w;
  a.T = T, a.k = top_k, a.d = d, a.n_rows = n_rows;
  a.t_dtype = y_dtype, a.r_dtype = rows_dtype;
  return cuda_code(launch_combine_rows(a, static_cast<cudaStream_t>(stream)));
}

int moe_combine_backward(const void* dy, int y_dtype, const void* rows, int rows_dtype, int n_rows, const int32_t* slot,
                         const float* w, int T, int top_k, int d, void* drows, float* dw, void* stream) {
  const int code = check_rows(T, top_k, d, n_rows, y_dtype, rows_dtype);
  if (code != MOE_OK || T == 0) return code;
  if ((!drows && !dw && n_rows > 0) || !dy || !slot || !w || (dw && n_rows > 0 && !rows)) return MOE_ERR_ARG;
  if (!aligned16(dy, rows, slot, w, drows, dw)) return MOE_ERR_ALIGN;
  if (!drows && !dw) return MOE_OK;
  const NvtxRange range("moe_combine_backward");
  RowsArgs a{};
  a.tokens = dy;
  a.rows_in = rows;
  a.out = drows;
  a.slot = slot;
  a.w = w;
  a.dw = dw;
  a.T = T, a.k = top_k, a.d = d, a.n_rows = n_rows;
  a.t_dtype = y_dtype, a.r_dtype = rows_dtype;
  return cuda_code(launch_combine_backward(a, static_cast<cudaStream_t>(stream)));
}

// ------------------------------------------------------------------ matrix product with its epilogue
int moe_linear_init(const moe_linear_config* cfg, moe_linear** out) {
  if (!cfg || !out) return MOE_ERR_ARG;
  *out = nullptr;
  const moe_linear_config c = *cfg;
  if (c.in_features <= 0 || c.out_features <= 0 || c.max_tokens <= 0) return MOE_ERR_ARG;
  if (c.activation != MOE_ACT_NONE && c.activation != MOE_ACT_SILU && c.activation != MOE_ACT_GELU) return MOE_ERR_ARG;
  if (c.training != 0 && c.training != 1) return MOE_ERR_ARG;
  if (c.in_features % 8 != 0 || c.out_features % 8 != 0 || c.in_features > (1 << 24) || c.out_features > (1 << 24) ||
      c.max_tokens > (1 << 28))
    return MOE_ERR_UNSUPPORTED;
  int dev = 0;
  cudaDeviceProp prop;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaGetDeviceProperties(&prop, dev) != cudaSuccess) {
    cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  if (!(prop.major == 10 && prop.minor == 3)) return MOE_ERR_UNSUPPORTED;
  FfnEngine eng{};
  eng.sms = prop.multiProcessorCount;
  eng.ctl.spin_limit = kDefaultSpinNs;
  void* fn = nullptr;
  cudaDriverEntryPointQueryResult q;
  if (prepare_ffn_gemm(&eng) != cudaSuccess || prepare_ffn_skinny() != cudaSuccess ||
      cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) != cudaSuccess ||
      q != cudaDriverEntryPointSuccess || !fn) {
    cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  eng.encode = reinterpret_cast<EncodeTiledFn>(fn);
  moe_linear* ctx = new (std::nothrow) moe_linear();
  if (!ctx) return MOE_ERR_NOMEM;
  ctx->cfg = c;
  const size_t bytes = 256 + (c.training ? (size_t)c.max_tokens * c.out_features * 2 : 0);
  if (cudaMalloc(&ctx->block, bytes) != cudaSuccess) {
    cudaGetLastError();
    delete ctx;
    return MOE_ERR_NOMEM;
  }
  if (cudaMemset(ctx->block, 0, 256) != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess) {  // the status word
    cudaGetLastError();
    cudaFree(ctx->block);
    delete ctx;
    return MOE_ERR_CUDA;
  }
  eng.ctl.status = static_cast<unsigned*>(ctx->block);
  if (c.training) ctx->dpre = reinterpret_cast<uint16_t*>(static_cast<char*>(ctx->block) + 256);
  ctx->eng = eng;
  *out = ctx;
  return MOE_OK;
}

int moe_linear_set_spin_limit(moe_linear* ctx, long long limit) {
  if (!ctx || limit < 0) return MOE_ERR_ARG;
  ctx->eng.ctl.spin_limit = limit == 0 ? kDefaultSpinNs : limit;
  return MOE_OK;
}

int moe_linear_inject_stall(moe_linear* ctx, int on) {
  if (!ctx || (on != 0 && on != 1)) return MOE_ERR_ARG;
  ctx->eng.ctl.stall = on;
  return MOE_OK;
}

int moe_linear_forward(moe_linear* ctx, const void* x, int T, const void* weight, const void* bias, int bias_dtype,
                       const void* residual, void* y, int y_dtype, void* pre, void* stream) {
  if (!ctx || T < 0 || T > ctx->cfg.max_tokens || !stream_dtype(bias_dtype) || !stream_dtype(y_dtype))
    return MOE_ERR_ARG;
  if (T == 0) return MOE_OK;
  if (!x || !weight || !y) return MOE_ERR_ARG;
  if (!aligned16(x, weight, bias, residual, y, pre)) return MOE_ERR_ALIGN;
  const NvtxRange range("moe_linear_forward");
  const LinearShape s{T, ctx->cfg.in_features, ctx->cfg.out_features, ctx->cfg.activation};
  const LinearForwardArgs a{x, weight, bias, residual, y, static_cast<uint16_t*>(pre), bias_dtype, y_dtype};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  ++ctx->launches;
  return cuda_code(gemv_tokens(s) ? launch_linear_gemv(ctx->eng, s, a, st)
                   : few_tokens(s, s.n) ? launch_linear_stream(ctx->eng, s, a, st)
                                        : launch_linear_tiles(ctx->eng, s, a, st));
}

int moe_linear_backward(moe_linear* ctx, const void* x, const void* pre, int T, const void* weight, const void* dy,
                        int dy_dtype, void* dx, void* dweight, void* dbias, int bias_dtype, void* stream) {
  if (!ctx || T < 0 || T > ctx->cfg.max_tokens || !stream_dtype(bias_dtype) || !stream_dtype(dy_dtype))
    return MOE_ERR_ARG;
  const moe_linear_config& c = ctx->cfg;
  if (!c.training) return MOE_ERR_UNSUPPORTED;
  const bool linear = c.activation == MOE_ACT_NONE;
  if (T > 0 && ((!dx && !dweight && !dbias) || !dy || (!linear && !pre) || (dx && !weight) || (dweight && !x)))
    return MOE_ERR_ARG;
  if (!aligned16(x, pre, weight, dy, dx, dweight, dbias)) return MOE_ERR_ALIGN;
  const NvtxRange range("moe_linear_backward");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (T == 0) {  // no rows: the gradients of weight and bias are sums of nothing
    const size_t n = c.out_features;
    cudaError_t e = cudaSuccess;
    if (dweight) e = cudaMemsetAsync(dweight, 0, n * c.in_features * 2, st);
    if (e == cudaSuccess && dbias) e = cudaMemsetAsync(dbias, 0, n * (bias_dtype == MOE_BF16 ? 2 : 4), st);
    return cuda_code(e);
  }
  const LinearShape s{T, c.in_features, c.out_features, c.activation};
  const bool as_is = linear && dy_dtype == MOE_BF16;  // dpre is dy
  const uint16_t* dpre = as_is ? static_cast<const uint16_t*>(dy) : ctx->dpre;
  const bool products = dx || dweight, few = few_tokens(s, s.k), least = few_grad_tokens(s);
  LinearGradArgs g{dy, static_cast<const uint16_t*>(pre), nullptr, dbias, T, c.out_features, dy_dtype, bias_dtype,
                   c.activation};
  cudaError_t err = cudaSuccess;
  if (least && dweight) {
    g.dpre = dx && !as_is ? ctx->dpre : nullptr;
    err = launch_linear_few_grad(g, x, dweight, c.in_features, st);
    ++ctx->launches;
  } else if (dbias || (products && !as_is)) {
    g.dpre = products && !as_is ? ctx->dpre : nullptr;
    err = launch_linear_grad(g, st);
    ++ctx->launches;
  }
  if (err == cudaSuccess && few && dx) {
    err = launch_linear_dx_stream(ctx->eng, s, dpre, weight, dx, st);
    ++ctx->launches;
  }
  if (err == cudaSuccess && ((!few && dx) || (!least && dweight))) {
    int n = 0;
    err = launch_linear_grads(ctx->eng, s, dpre, x, weight, dx, dweight, &n, st);
    ctx->launches += n;
  }
  return cuda_code(err);
}

long long moe_linear_launch_count(moe_linear* ctx) { return ctx ? ctx->launches : 0; }

int moe_linear_status(moe_linear* ctx) {
  if (!ctx) return MOE_ERR_ARG;
  if (cudaDeviceSynchronize() != cudaSuccess) return MOE_ERR_CUDA;
  unsigned v = 0;
  if (cudaMemcpy(&v, ctx->eng.ctl.status, 4, cudaMemcpyDeviceToHost) != cudaSuccess) return MOE_ERR_CUDA;
  if (v && cudaMemset(ctx->eng.ctl.status, 0, 4) != cudaSuccess) return MOE_ERR_CUDA;
  return v & kStatusTimeout ? MOE_ERR_TIMEOUT : (v & kStatusBounds ? MOE_ERR_BOUNDS : MOE_OK);
}

void moe_linear_destroy(moe_linear* ctx) {
  if (!ctx) return;
  cudaDeviceSynchronize();
  if (ctx->block) cudaFree(ctx->block);
  delete ctx;
}

}  // extern "C"
