// Entry points of the decoder block's products: the base projection with its
// epilogue, the gated feed-forward block and its gradients.  Every argument is
// checked before the first HIP call; the plan of a product (tile shape, K
// split) depends on sizes and types alone, so the workspace query and the call
// agree.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdlib>

#include "lora_block.h"

namespace lora {

int32_t check_launch(const char* what) {
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(LORA_E_HIP, "%s launch: %s", what, hipGetErrorString(e));
  return LORA_OK;
}

namespace {

constexpr int64_t kMaxFeatures = 1 << 20;   // K, O and I
constexpr int64_t kMaxRows = 1 << 21;       // T

int64_t esize(int32_t dtype) { return dtype == LORA_F32 ? 4 : dtype == LORA_BF16 ? 2 : 1; }

// ---------------------------------------------------------------- products

// Sums the K splits' partials in their order and applies the epilogue, eight
// columns a thread.
template <bool kGated>
__global__ __launch_bounds__(256) void join_kernel(GemmArgs p) {
  const int per = (p.N + 7) / 8;
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (id >= (int64_t)p.M * per) return;
  const int m = (int)(id / per), n = (int)(id % per) * 8;
  float z[8], u[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) z[j] = 0.f, u[j] = 0.f;
  for (int s = 0; s < p.splits; ++s) {
    const float* d = p.part + ((int64_t)s * p.M + m) * p.ldp + n;
    float t[8];
    load8(d, 0, 8, LORA_F32, t);
#pragma unroll
    for (int j = 0; j < 8; ++j) z[j] += t[j];
    if constexpr (kGated) {
      load8(d, p.N, 8, LORA_F32, t);
#pragma unroll
      for (int j = 0; j < 8; ++j) u[j] += t[j];
    }
  }
  epilogue8<kGated>(p, m, n, z, u);
}

}  // namespace

GemmPlan gemm_plan(int32_t dtype, bool gated, int64_t M, int64_t N, int64_t kb) {
  GemmPlan g{0, 1, 0};
  const int64_t width = gated ? 2 * N : N;  // rows of B
  auto tiles = [&](int s) {
    return ((M + kShapes[s].bm - 1) / kShapes[s].bm) *
           ((width + kShapes[s].bn - 1) / kShapes[s].bn);
  };
  // the large tile where it gives every compute unit one
  g.shape = tiles(2) >= kComputeUnits ? 2 : tiles(1) >= kComputeUnits ? 1 : 0;
  const int64_t steps = (kb + kStepBytes - 1) / kStepBytes;
  const int64_t t = tiles(g.shape);
  // a K split where the tiles leave compute units idle: up to two workgroups a
  // unit, at least eight steps a part
  int64_t s = std::max<int64_t>(1, std::min<int64_t>(2 * kComputeUnits / t, steps / 8));
  s = std::min<int64_t>(s, 16);
  if (const char* e = std::getenv("LORA_GEMM_PLAN")) {  // tuning override: shape,splits
    char* end = nullptr;
    const long shape = std::strtol(e, &end, 10);
    const long parts = *end == ',' ? std::strtol(end + 1, nullptr, 10) : 0;
    if (shape >= 0 && shape < (long)(sizeof(kShapes) / sizeof(kShapes[0])))
      g.shape = (int32_t)shape;
    if (parts >= 1 && parts <= 64) s = std::min<int64_t>(parts, steps);
  }
  if (s > 1) {
    const int64_t per = (steps + s - 1) / s;
    s = (steps + per - 1) / per;  // no part is empty
  }
  g.splits = (int32_t)s;
  if (s > 1) g.ws_bytes = s * M * ((width + 7) / 8 * 8) * 4;
  return g;
}

int32_t gemm_run(int32_t dtype, bool gated, const GemmPlan& plan, GemmArgs a, void* ws,
                 hipStream_t st) {
  const TileShape sh = kShapes[plan.shape];
  const int width = gated ? 2 * a.N : a.N;
  a.tiles_m = (a.M + sh.bm - 1) / sh.bm;
  a.tiles_n = (width + sh.bn - 1) / sh.bn;
  a.splits = plan.splits;
  a.part = plan.splits > 1 ? (float*)ws : nullptr;
  a.ldp = (width + 7) / 8 * 8;
  int32_t e = dtype == LORA_BF16   ? gemm_launch_bf16(gated, plan.shape, a, st)
              : dtype == LORA_E4M3 ? gemm_launch_e4m3(gated, plan.shape, a, st)
                                   : gemm_launch_f32(gated, plan.shape, a, st);
  if (e || plan.splits == 1) return e;
  const int64_t threads = (int64_t)a.M * ((a.N + 7) / 8);
  const dim3 grid((unsigned)((threads + 255) / 256));
  if (gated)
    hipLaunchKernelGGL(join_kernel<true>, grid, dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL(join_kernel<false>, grid, dim3(256), 0, st, a);
  return check_launch("join of the K splits");
}

namespace {

// ---------------------------------------------------------------- backward

// dpre from dout and what the forward pass saved: with value a(g) and slope
// a'(g) of the activation at the gate g,
//   d gate = dout * up * a'(g),   d up = dout * a(g).
// Eight columns a thread, five reads and writes of one [T][I] array each.
template <int DT>
__global__ __launch_bounds__(256) void gate_grad_kernel(const void* dout, const void* pre,
                                                        void* dpre, int64_t T, int I, int act) {
  const int per = I / 8;
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (id >= T * per) return;
  const int64_t m = id / per;
  const int n = (int)(id % per) * 8;
  float d[8], g[8], u[8];
  load8(dout, m * I + n, 8, DT, d);
  load8(pre, m * 2 * I + n, 8, DT, g);
  load8(pre, m * 2 * I + I + n, 8, DT, u);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float value, slope;
    act_curve(act, g[j], value, slope);
    g[j] = d[j] * u[j] * slope;
    u[j] = d[j] * value;
  }
  store8(dpre, m * 2 * I + n, 8, DT, g);
  store8(dpre, m * 2 * I + I + n, 8, DT, u);
}

// dst[c][r] = src[r][c] for r < R, zero for R <= r < ldd; a 64 x 64 tile a
// workgroup through LDS.
template <typename E>
__global__ __launch_bounds__(256) void transpose_kernel(const E* src, E* dst, int R, int C,
                                                        int ldd) {
  __shared__ E tile[64][65];
  const int r0 = blockIdx.y * 64, c0 = blockIdx.x * 64;
  for (int i = threadIdx.x; i < 64 * 64; i += 256) {
    const int r = i >> 6, c = i & 63;
    tile[r][c] = r0 + r < R && c0 + c < C ? src[(int64_t)(r0 + r) * C + c0 + c] : E(0);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 64 * 64; i += 256) {
    const int c = i >> 6, r = i & 63;
    if (c0 + c < C && r0 + r < ldd) dst[(int64_t)(c0 + c) * ldd + r0 + r] = tile[r][c];
  }
}

void transpose(int32_t dtype, const void* src, void* dst, int R, int C, int ldd, hipStream_t st) {
  const dim3 grid((C + 63) / 64, (ldd + 63) / 64);
  if (dtype == LORA_BF16)
    hipLaunchKernelGGL(transpose_kernel<uint16_t>, grid, dim3(256), 0, st, (const uint16_t*)src,
                       (uint16_t*)dst, R, C, ldd);
  else
    hipLaunchKernelGGL(transpose_kernel<uint32_t>, grid, dim3(256), 0, st, (const uint32_t*)src,
                       (uint32_t*)dst, R, C, ldd);
}

__global__ __launch_bounds__(256) void clear_kernel(bk_u32x4* p, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
    p[i] = bk_u32x4{0, 0, 0, 0};
}

struct BackwardLayout {
  int64_t wt, dt, xt, part, total;
  GemmPlan dx, dw;
  int32_t ldt;  // elements a row of the arrays transposed over the tokens
};

BackwardLayout backward_layout(const lora_gated_desc& d, int64_t T, bool dx, bool dw) {
  BackwardLayout b{};
  const int64_t e = esize(d.dtype), K = d.in_features, I2 = 2 * (int64_t)d.inter_features;
  b.ldt = (int32_t)align_up(T, 16 / e);
  int64_t at = 0, part = 0;
  b.wt = at;
  if (dx) {
    at = align_up(at + e * K * I2, 256);
    b.dx = gemm_plan(d.dtype, false, T, K, e * I2);
    part = std::max(part, b.dx.ws_bytes);
  }
  b.dt = at;
  if (dw) {
    at = align_up(at + e * I2 * b.ldt, 256);
    b.xt = at;
    at = align_up(at + e * K * b.ldt, 256);
    b.dw = gemm_plan(d.dtype, false, I2, K, e * b.ldt);
    part = std::max(part, b.dw.ws_bytes);
  }
  b.part = at;
  b.total = at + part;
  return b;
}

// ------------------------------------------------------------------ checks

int32_t check_types(int32_t dtype, int32_t out_dtype, const char* what) {
  if (dtype != LORA_F32 && dtype != LORA_BF16 && dtype != LORA_E4M3)
    return fail(LORA_E_DTYPE, "unknown %s dtype %d (0 = fp32, 1 = bf16, 2 = e4m3)", what, dtype);
  if (out_dtype != LORA_F32 && out_dtype != LORA_BF16)
    return fail(LORA_E_DTYPE, "%s output dtype must be fp32 or bf16, got %d", what, out_dtype);
  if (dtype == LORA_F32 && out_dtype != LORA_F32)
    return fail(LORA_E_DTYPE, "%s of fp32 operands has fp32 outputs", what);
  return LORA_OK;
}

int32_t check_size(int32_t v, int32_t multiple, const char* name) {
  if (v < multiple || v > kMaxFeatures)
    return fail(LORA_E_SHAPE, "%s must be in [%d, %lld], got %d", name, multiple,
                (long long)kMaxFeatures, v);
  if (v % multiple)
    return fail(LORA_E_ALIGN, "%s must be a multiple of %d, got %d", name, multiple, v);
  return LORA_OK;
}

int32_t check_act(int32_t act) {
  if (act < LORA_ACT_NONE || act > LORA_ACT_RELU)
    return fail(LORA_E_ARG, "unknown activation %d", act);
  return LORA_OK;
}

int32_t check_linear(const lora_linear_desc* d) {
  if (!d) return fail(LORA_E_ARG, "descriptor is NULL");
  if (int32_t e = check_types(d->dtype, d->out_dtype, "linear")) return e;
  // a row of an operand is a whole number of 16-byte pieces
  if (int32_t e = check_size(d->in_features, (int32_t)(d->dtype == LORA_E4M3 ? 16 : 8),
                             "in_features"))
    return e;
  if (int32_t e = check_size(d->out_features, 1, "out_features")) return e;
  return check_act(d->act);
}

int32_t check_gated(const lora_gated_desc* d) {
  if (!d) return fail(LORA_E_ARG, "descriptor is NULL");
  if (int32_t e = check_types(d->dtype, d->out_dtype, "gated")) return e;
  const int32_t unit = d->dtype == LORA_E4M3 ? 16 : 8;
  if (int32_t e = check_size(d->in_features, unit, "in_features")) return e;
  if (int32_t e = check_size(d->inter_features, unit, "inter_features")) return e;
  return check_act(d->act);
}

int32_t check_rows(int32_t T) {
  if (T < 0) return fail(LORA_E_ARG, "T must be >= 0, got %d", T);
  if (T > kMaxRows)
    return fail(LORA_E_SHAPE, "T must be at most %lld, got %d", (long long)kMaxRows, T);
  return LORA_OK;
}

int32_t need(const void* p, const char* name) {
  if (!p) return fail(LORA_E_ARG, "%s is NULL", name);
  if (!aligned16(p)) return fail(LORA_E_ALIGN, "%s is not 16-byte aligned", name);
  return LORA_OK;
}
int32_t may(const void* p, const char* name) { return p ? need(p, name) : LORA_OK; }

int32_t check_scales(int32_t dtype, const float* xs, const float* ws) {
  if (dtype == LORA_E4M3) {
    if (int32_t e = need(xs, "x_scale")) return e;
    return need(ws, "w_scale");
  }
  if (xs || ws) return fail(LORA_E_ARG, "x_scale and w_scale are for e4m3 operands only");
  return LORA_OK;
}

int32_t check_ws(const void* ws, int64_t have, int64_t want) {
  if (want == 0) return LORA_OK;
  if (have < want)
    return fail(LORA_E_WORKSPACE, "workspace has %lld bytes, needs %lld", (long long)have,
                (long long)want);
  return need(ws, "ws");
}

}  // namespace

}  // namespace lora

using namespace lora;

extern "C" {

int64_t lora_linear_workspace_bytes(const lora_linear_desc* desc, int32_t T) {
  clear_error();
  if (int32_t e = check_linear(desc)) return e;
  if (int32_t e = check_rows(T)) return e;
  if (T == 0) return 0;
  return gemm_plan(desc->dtype, false, T, desc->out_features,
                   desc->in_features * esize(desc->dtype))
      .ws_bytes;
}

int32_t lora_linear(const lora_linear_desc* desc, const void* x, const void* w,
                    const float* x_scale, const float* w_scale, const void* bias,
                    const void* delta, const void* residual, void* out, int32_t T, void* ws,
                    int64_t ws_bytes, void* stream) {
  clear_error();
  if (int32_t e = check_linear(desc)) return e;
  if (int32_t e = check_rows(T)) return e;
  if (T == 0) return LORA_OK;
  if (int32_t e = need(x, "x")) return e;
  if (int32_t e = need(w, "w")) return e;
  if (int32_t e = check_scales(desc->dtype, x_scale, w_scale)) return e;
  if (int32_t e = may(bias, "bias")) return e;
  if (int32_t e = may(delta, "delta")) return e;
  if (int32_t e = may(residual, "residual")) return e;
  if (int32_t e = need(out, "out")) return e;
  const int64_t kb = desc->in_features * esize(desc->dtype);
  const GemmPlan plan = gemm_plan(desc->dtype, false, T, desc->out_features, kb);
  if (int32_t e = check_ws(ws, ws_bytes, plan.ws_bytes)) return e;
  GemmArgs a{};
  a.A = (const char*)x;
  a.B = (const char*)w;
  a.sa = x_scale;
  a.sb = w_scale;
  a.bias = bias;
  a.delta = delta;
  a.residual = residual;
  a.out = out;
  a.kb = kb;
  a.M = T;
  a.N = desc->out_features;
  a.out_dtype = desc->out_dtype;
  a.act = desc->act;
  return gemm_run(desc->dtype, false, plan, a, ws, (hipStream_t)stream);
}

int64_t lora_gated_ffn_workspace_bytes(const lora_gated_desc* desc, int32_t T) {
  clear_error();
  if (int32_t e = check_gated(desc)) return e;
  if (int32_t e = check_rows(T)) return e;
  if (T == 0) return 0;
  return gemm_plan(desc->dtype, true, T, desc->inter_features,
                   desc->in_features * esize(desc->dtype))
      .ws_bytes;
}

int32_t lora_gated_ffn(const lora_gated_desc* desc, const void* x, const void* w,
                       const float* x_scale, const float* w_scale, const void* delta, void* pre,
                       void* out, int32_t T, void* ws, int64_t ws_bytes, void* stream) {
  clear_error();
  if (int32_t e = check_gated(desc)) return e;
  if (int32_t e = check_rows(T)) return e;
  if (T == 0) return LORA_OK;
  if (int32_t e = need(x, "x")) return e;
  if (int32_t e = need(w, "w")) return e;
  if (int32_t e = check_scales(desc->dtype, x_scale, w_scale)) return e;
  if (int32_t e = may(delta, "delta")) return e;
  if (int32_t e = may(pre, "pre")) return e;
  if (int32_t e = need(out, "out")) return e;
  const int64_t kb = desc->in_features * esize(desc->dtype);
  const GemmPlan plan = gemm_plan(desc->dtype, true, T, desc->inter_features, kb);
  if (int32_t e = check_ws(ws, ws_bytes, plan.ws_bytes)) return e;
  GemmArgs a{};
  a.A = (const char*)x;
  a.B = (const char*)w;
  a.sa = x_scale;
  a.sb = w_scale;
  a.delta = delta;
  a.pre = pre;
  a.out = out;
  a.kb = kb;
  a.M = T;
  a.N = desc->inter_features;
  a.out_dtype = desc->out_dtype;
  a.act = desc->act;
  return gemm_run(desc->dtype, true, plan, a, ws, (hipStream_t)stream);
}

static int32_t check_backward(const lora_gated_desc* desc) {
  if (int32_t e = check_gated(desc)) return e;
  if (desc->dtype == LORA_E4M3)
    return fail(LORA_E_DTYPE, "the gradients take fp32 or bf16 operands");
  if (desc->out_dtype != desc->dtype)
    return fail(LORA_E_DTYPE, "the gradients have the operands' dtype");
  return LORA_OK;
}

int64_t lora_gated_ffn_backward_workspace_bytes(const lora_gated_desc* desc, int32_t T,
                                                int32_t need_dx, int32_t need_dw) {
  clear_error();
  if (int32_t e = check_backward(desc)) return e;
  if (int32_t e = check_rows(T)) return e;
  if (T == 0) return 0;
  return backward_layout(*desc, T, need_dx != 0, need_dw != 0).total;
}

int32_t lora_gated_ffn_backward(const lora_gated_desc* desc, const void* dout, const void* pre,
                                const void* x, const void* w, void* dpre, void* dx, void* dw,
                                int32_t T, void* ws, int64_t ws_bytes, void* stream) {
  clear_error();
  if (int32_t e = check_backward(desc)) return e;
  if (int32_t e = check_rows(T)) return e;
  const hipStream_t st = (hipStream_t)stream;
  const int64_t es = esize(desc->dtype);
  const int K = desc->in_features, I = desc->inter_features;
  if (int32_t e = may(dw, "dw")) return e;
  if (T == 0) {  // a sum over no tokens
    if (!dw) return LORA_OK;
    const int64_t n = 2 * (int64_t)I * K * es / 16;
    hipLaunchKernelGGL(clear_kernel, dim3((unsigned)std::min<int64_t>((n + 255) / 256, 4096)),
                       dim3(256), 0, st, (bk_u32x4*)dw, n);
    return check_launch("clear");
  }
  if (int32_t e = need(dout, "dout")) return e;
  if (int32_t e = need(pre, "pre")) return e;
  if (int32_t e = need(dpre, "dpre")) return e;
  if (int32_t e = may(dx, "dx")) return e;
  if (dw) {
    if (int32_t e = need(x, "x")) return e;
  }
  if (dx) {
    if (int32_t e = need(w, "w")) return e;
  }
  const BackwardLayout b = backward_layout(*desc, T, dx != nullptr, dw != nullptr);
  if (int32_t e = check_ws(ws, ws_bytes, b.total)) return e;

  const dim3 grid((unsigned)(((int64_t)T * (I / 8) + 255) / 256));
  if (desc->dtype == LORA_BF16)
    hipLaunchKernelGGL(gate_grad_kernel<LORA_BF16>, grid, dim3(256), 0, st, dout, pre, dpre,
                       (int64_t)T, I, desc->act);
  else
    hipLaunchKernelGGL(gate_grad_kernel<LORA_F32>, grid, dim3(256), 0, st, dout, pre, dpre,
                       (int64_t)T, I, desc->act);
  if (int32_t e = check_launch("gate gradient")) return e;

  char* base = (char*)ws;
  GemmArgs a{};
  a.out_dtype = desc->dtype;
  a.act = LORA_ACT_NONE;
  if (dx) {
    transpose(desc->dtype, w, base + b.wt, 2 * I, K, 2 * I, st);
    if (int32_t e = check_launch("transpose")) return e;
    a.A = (const char*)dpre;
    a.B = base + b.wt;
    a.out = dx;
    a.kb = 2 * I * es;
    a.M = T;
    a.N = K;
    if (int32_t e = gemm_run(desc->dtype, false, b.dx, a, base + b.part, st)) return e;
  }
  if (dw) {
    transpose(desc->dtype, dpre, base + b.dt, T, 2 * I, b.ldt, st);
    transpose(desc->dtype, x, base + b.xt, T, K, b.ldt, st);
    if (int32_t e = check_launch("transpose")) return e;
    a.A = base + b.dt;
    a.B = base + b.xt;
    a.out = dw;
    a.kb = b.ldt * es;
    a.M = 2 * I;
    a.N = K;
    if (int32_t e = gemm_run(desc->dtype, false, b.dw, a, base + b.part, st)) return e;
  }
  return LORA_OK;
}

}  // extern "C"
