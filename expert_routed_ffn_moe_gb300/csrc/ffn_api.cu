// C ABI of the dense gated feed-forward block and of the norm in front of it:
// argument checking, the context and its workspace, and the kernel sequence of
// each call.  Declarations and the full contract are in include/moe.h.
#include <new>

#include <nvtx3/nvToolsExt.h>

#include "ffn_internal.h"

using namespace moe;

struct moe_ffn {
  moe_ffn_config cfg;
  void* block = nullptr;  // the single device allocation holding the workspace
  FfnScratch sc{};
  FfnEngine eng{};
  long long launches = 0;
};

namespace {

constexpr long long kDefaultSpinNs = 1000000000LL;  // 1 s
constexpr int kMaxRows = 1 << 30;  // norm, rounding to mx8: a row's number plus a grid of rows stays an int

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool stream_dtype(int t) { return t == MOE_F32 || t == MOE_BF16; }
int cuda_code(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
};

}  // namespace

extern "C" {

long long moe_mx_scale_bytes(int rows, int cols) {
  if (rows < 0 || cols < 0) return 0;
  return (long long)mx_scale_bytes(rows, cols);
}

int moe_quantize_mx(const void* v, int dtype, int rows, int cols, void* codes, void* scales, void* stream) {
  if (rows < 0 || cols < 0 || !stream_dtype(dtype)) return MOE_ERR_ARG;
  if (cols % 32 != 0 || rows > kMaxRows) return MOE_ERR_UNSUPPORTED;
  if (rows == 0 || cols == 0) return MOE_OK;
  if (!v || !codes || !scales) return MOE_ERR_ARG;
  if (!aligned16(v) || !aligned16(codes) || !aligned16(scales)) return MOE_ERR_ALIGN;
  const NvtxRange range("moe_quantize_mx");
  return cuda_code(launch_mx_quantize(v, dtype, rows, cols, static_cast<uint8_t*>(codes), static_cast<uint8_t*>(scales),
                                      static_cast<cudaStream_t>(stream)));
}

int moe_add_norm(const void* x, int x_dtype, const void* residual, int s_dtype, const void* weight, int w_dtype, int T,
                 int d, float eps, void* s_out, void* y, int y_dtype, void* y_scales, void* stream) {
  if (T < 0 || d <= 0 || !stream_dtype(x_dtype) || !stream_dtype(s_dtype) || !stream_dtype(w_dtype)) return MOE_ERR_ARG;
  if ((!stream_dtype(y_dtype) && y_dtype != MOE_MX8) || !(eps >= 0.f)) return MOE_ERR_ARG;
  if (d > kMaxNormWidth || T > kMaxRows || (y_dtype == MOE_MX8 && d % 32 != 0)) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!x || !weight || !y || (y_dtype == MOE_MX8) != (y_scales != nullptr)) return MOE_ERR_ARG;
  if (!aligned16(x) || !aligned16(residual) || !aligned16(weight) || !aligned16(s_out) || !aligned16(y) ||
      !aligned16(y_scales))
    return MOE_ERR_ALIGN;
  const NvtxRange range("moe_add_norm");
  NormArgs a{x, residual, weight, s_out, y, static_cast<uint8_t*>(y_scales), T, d, x_dtype, s_dtype, w_dtype, y_dtype,
             eps};
  return cuda_code(launch_norm(a, static_cast<cudaStream_t>(stream)));
}

long long moe_add_norm_workspace(int d) { return d <= 0 ? 0 : (long long)kNormPartials * d * 4; }

int moe_add_norm_backward(const void* s, const void* weight, const void* dy, const void* ds, int dtype, int w_dtype,
                          int T, int d, float eps, void* dx, void* dweight, void* workspace, void* stream) {
  if (T < 0 || d <= 0 || !stream_dtype(dtype) || !stream_dtype(w_dtype) || !(eps >= 0.f)) return MOE_ERR_ARG;
  if (d > kMaxNormWidth || T > kMaxRows) return MOE_ERR_UNSUPPORTED;
  // (without rows dx is a tensor of no values, which may have no address)
  if (T > 0 && ((!dx && !dweight) || !s || !weight || !dy || (dweight && !workspace))) return MOE_ERR_ARG;
  if (!aligned16(s) || !aligned16(weight) || !aligned16(dy) || !aligned16(ds) || !aligned16(dx) ||
      !aligned16(dweight) || !aligned16(workspace))
    return MOE_ERR_ALIGN;
  const NvtxRange range("moe_add_norm_backward");
  cudaStream_t stm = static_cast<cudaStream_t>(stream);
  if (T == 0)  // no rows: the weight's gradient is a sum of nothing
    return dweight ? cuda_code(cudaMemsetAsync(dweight, 0, (size_t)d * (w_dtype == MOE_BF16 ? 2 : 4), stm)) : MOE_OK;
  NormGradArgs a{s, weight, dy, ds, dx, dweight, static_cast<float*>(workspace), T, d, dtype, w_dtype, eps};
  return cuda_code(launch_norm_backward(a, stm));
}

int moe_ffn_init(const moe_ffn_config* cfg, moe_ffn** out) {
  if (!cfg || !out) return MOE_ERR_ARG;
  *out = nullptr;
  const moe_ffn_config c = *cfg;
  if (c.d <= 0 || c.inter <= 0 || c.max_tokens <= 0) return MOE_ERR_ARG;
  if (c.activation != MOE_ACT_SILU && c.activation != MOE_ACT_GELU) return MOE_ERR_ARG;
  if (c.weight_format != MOE_W_BF16 && c.weight_format != MOE_W_MX8) return MOE_ERR_ARG;
  if (c.training != 0 && c.training != 1) return MOE_ERR_ARG;
  const bool mx = c.weight_format == MOE_W_MX8;
  const int unit = mx ? 32 : 8;
  if (c.d % unit != 0 || c.inter % unit != 0 || (mx && c.training)) return MOE_ERR_UNSUPPORTED;
  if (c.d > (1 << 24) || c.inter > (1 << 24) || c.max_tokens > (1 << 28)) return MOE_ERR_UNSUPPORTED;
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

  const size_t T = c.max_tokens, I = c.inter;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = (off + bytes + 255) / 256 * 256;
    return o;
  };
  const size_t o_status = take(16);
  const size_t o_h = take(mx ? 0 : T * I * 2);
  const size_t o_hq = take(mx ? T * I : 0);
  const size_t o_hs = take(mx ? mx_scale_bytes(T, I) : 0);
  const size_t o_up_s = take(mx && I % 128 != 0 ? mx_scale_bytes(I, c.d) : 0);
  const size_t o_dpre = take(c.training ? T * 2 * I * 2 : 0);
  moe_ffn* ctx = new (std::nothrow) moe_ffn();
  if (!ctx) return MOE_ERR_NOMEM;
  ctx->cfg = c;
  if (cudaMalloc(&ctx->block, off) != cudaSuccess) {
    cudaGetLastError();
    delete ctx;
    return MOE_ERR_NOMEM;
  }
  char* b = static_cast<char*>(ctx->block);
  // the status word, and the scale bytes past the last row and group, which no kernel writes
  if (cudaMemset(b + o_status, 0, 16) != cudaSuccess ||
      (mx && cudaMemset(b + o_hs, 0, mx_scale_bytes(T, I)) != cudaSuccess) || cudaDeviceSynchronize() != cudaSuccess) {
    cudaGetLastError();
    cudaFree(ctx->block);
    delete ctx;
    return MOE_ERR_CUDA;
  }
  ctx->sc.status = reinterpret_cast<unsigned*>(b + o_status);
  ctx->sc.h = reinterpret_cast<uint16_t*>(b + o_h);
  ctx->sc.hq = reinterpret_cast<uint8_t*>(b + o_hq);
  ctx->sc.hs = reinterpret_cast<uint8_t*>(b + o_hs);
  ctx->sc.up_s = reinterpret_cast<uint8_t*>(b + o_up_s);
  ctx->sc.dpre = reinterpret_cast<uint16_t*>(b + o_dpre);
  eng.ctl.status = ctx->sc.status;
  ctx->eng = eng;
  *out = ctx;
  return MOE_OK;
}

int moe_ffn_set_spin_limit(moe_ffn* ctx, long long limit) {
  if (!ctx || limit < 0) return MOE_ERR_ARG;
  ctx->eng.ctl.spin_limit = limit == 0 ? kDefaultSpinNs : limit;
  return MOE_OK;
}

int moe_ffn_inject_stall(moe_ffn* ctx, int on) {
  if (!ctx || (on != 0 && on != 1)) return MOE_ERR_ARG;
  ctx->eng.ctl.stall = on;
  return MOE_OK;
}

int moe_ffn_forward(moe_ffn* ctx, const void* x, const void* x_scales, int T, const void* gate_up,
                    const void* gate_up_scales, const void* down, const void* down_scales, void* y, void* pre,
                    void* stream) {
  if (!ctx || T < 0 || T > ctx->cfg.max_tokens) return MOE_ERR_ARG;
  if (T == 0) return MOE_OK;
  const moe_ffn_config& c = ctx->cfg;
  const bool mx = c.weight_format == MOE_W_MX8;
  if (!x || !gate_up || !down || !y) return MOE_ERR_ARG;
  if (mx != (x_scales != nullptr) || mx != (gate_up_scales != nullptr) || mx != (down_scales != nullptr))
    return MOE_ERR_ARG;
  if (mx && pre) return MOE_ERR_UNSUPPORTED;
  for (const void* p : {x, x_scales, gate_up, gate_up_scales, down, down_scales, (const void*)y, (const void*)pre})
    if (!aligned16(p)) return MOE_ERR_ALIGN;
  const NvtxRange range("moe_ffn_forward");
  const FfnShape s{T, c.d, c.inter, c.activation};
  const FfnForwardArgs a{x,   gate_up, down, static_cast<const uint8_t*>(x_scales),
                         static_cast<const uint8_t*>(gate_up_scales), static_cast<const uint8_t*>(down_scales), y, pre};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const FfnScratch& sc = ctx->sc;
  cudaError_t err = cudaSuccess;
  const uint8_t* up_s = nullptr;
  if (mx) {
    up_s = a.gate_up_s + mx_scale_bytes(s.I, s.d);  // row tile I / 128 on
    if (s.I % 128 != 0) {
      err = launch_mx_up_scales(s, a.gate_up_s, sc.up_s, st);
      ++ctx->launches;
      up_s = sc.up_s;
    }
  }
  if (err != cudaSuccess) return cuda_code(err);
  ctx->launches += 2;
  if (few_tokens(s)) {
    err = launch_skinny_forward(ctx->eng, s, mx, a, up_s, sc, st);
  } else if (mx) {
    err = launch_ffn_gate_up_mx(ctx->eng, s, a, up_s, sc.hq, sc.hs, st);
    if (err == cudaSuccess) err = launch_ffn_down_mx(ctx->eng, s, sc.hq, sc.hs, a, st);
  } else {
    err = launch_ffn_gate_up(ctx->eng, s, x, gate_up, sc.h, static_cast<uint16_t*>(pre), st);
    if (err == cudaSuccess) err = launch_ffn_down(ctx->eng, s, sc.h, down, y, st);
  }
  return cuda_code(err);
}

int moe_ffn_backward(moe_ffn* ctx, const void* x, const void* pre, int T, const void* gate_up, const void* down,
                     const void* dy, void* dx, void* dgate_up, void* ddown, void* stream) {
  if (!ctx || T < 0 || T > ctx->cfg.max_tokens) return MOE_ERR_ARG;
  const moe_ffn_config& c = ctx->cfg;
  if (!c.training) return MOE_ERR_UNSUPPORTED;
  if (T > 0 && ((!dx && !dgate_up && !ddown) || !pre || !down || !dy || (dx && !gate_up) || (dgate_up && !x)))
    return MOE_ERR_ARG;
  for (const void* p : {x, pre, gate_up, down, dy, (const void*)dx, (const void*)dgate_up, (const void*)ddown})
    if (!aligned16(p)) return MOE_ERR_ALIGN;
  const NvtxRange range("moe_ffn_backward");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (T == 0) {  // no rows: the weights' gradients are sums of nothing
    const size_t n = (size_t)c.d * c.inter * 2;
    cudaError_t e = cudaSuccess;
    if (dgate_up) e = cudaMemsetAsync(dgate_up, 0, 2 * n, st);
    if (e == cudaSuccess && ddown) e = cudaMemsetAsync(ddown, 0, n, st);
    return cuda_code(e);
  }
  const FfnShape s{T, c.d, c.inter, c.activation};
  auto in = [](const void* p) { return static_cast<const uint16_t*>(p); };
  auto out = [](void* p) { return static_cast<uint16_t*>(p); };
  const FfnBackwardArgs a{in(x), in(pre), in(gate_up), in(down), in(dy), out(dx), out(dgate_up), out(ddown)};
  const bool skinny = few_tokens(s);
  cudaError_t err = skinny ? launch_skinny_backward(ctx->eng, s, a, ctx->sc, st)
                           : launch_ffn_grad_h(ctx->eng, s, a, ctx->sc, st);
  ctx->launches += skinny && dx ? 2 : 1;
  if (err == cudaSuccess) {
    int n = 0;
    err = launch_ffn_grads(ctx->eng, s, a, ctx->sc, &n, st);
    ctx->launches += n;
  }
  return cuda_code(err);
}

long long moe_ffn_launch_count(moe_ffn* ctx) { return ctx ? ctx->launches : 0; }

int moe_ffn_status(moe_ffn* ctx) {
  if (!ctx) return MOE_ERR_ARG;
  if (cudaDeviceSynchronize() != cudaSuccess) return MOE_ERR_CUDA;
  unsigned v = 0;
  if (cudaMemcpy(&v, ctx->sc.status, 4, cudaMemcpyDeviceToHost) != cudaSuccess) return MOE_ERR_CUDA;
  if (v && cudaMemset(ctx->sc.status, 0, 4) != cudaSuccess) return MOE_ERR_CUDA;
  return v & kStatusTimeout ? MOE_ERR_TIMEOUT : (v & kStatusBounds ? MOE_ERR_BOUNDS : MOE_OK);
}

void moe_ffn_destroy(moe_ffn* ctx) {
  if (!ctx) return;
  cudaDeviceSynchronize();
  if (ctx->block) cudaFree(ctx->block);
  delete ctx;
}

}  // extern "C"
