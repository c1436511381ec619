// Entry points of the decoder block's products: the base projection with its
// epilogue, the gated feed-forward block and its gradients.  Every argument is
// checked before the first HIP call; the plan of a product (tile shape, K
// split) and the workspace asked for depend on sizes and types alone (and on the
// tuning overrides), so the workspace query and the call agree.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdlib>
#include <cstring>

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

// Sums the partials of the split tiles in the order of K and applies the
// epilogue, eight columns a thread.
template <bool kGated>
__global__ __launch_bounds__(256) void join_kernel(GemmArgs p, int bm, int bn) {
  const int cols = kGated ? bn / 2 : bn, per = cols / 8;
  const int id = blockIdx.x * 256 + threadIdx.x;
  const int tile = id / (bm * per), in = id - tile * (bm * per);
  if (tile >= p.tiles_m * p.tiles_n - p.whole) return;
  const int r = in / per, c = (in - r * per) * 8;
  int tm, tn;
  tile_place(p, p.whole + tile, tm, tn);
  const int m = tm * bm + r, n = tn * cols + c;
  if (m >= p.M || n >= p.N) return;
  float z[8], u[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) z[j] = 0.f, u[j] = 0.f;
  const float* d = p.part + (int64_t)tile * p.splits * (bm * bn) + r * bn + c;
#pragma unroll 4
  for (int s = 0; s < p.splits; ++s, d += bm * bn) {
    float t[8];
    load8(d, 0, 8, LORA_F32, t);
#pragma unroll
    for (int j = 0; j < 8; ++j) z[j] += t[j];
    if constexpr (kGated) {
      load8(d, bn / 2, 8, LORA_F32, t);
#pragma unroll
      for (int j = 0; j < 8; ++j) u[j] += t[j];
    }
  }
  epilogue8<kGated, false>(p, m, n, z, u, Extra<kGated>{});
}

}  // namespace

namespace {

// What a workgroup of a tile shape takes, in microseconds: a start and an end,
// and a step of kStepBytes.  A compute unit holds up to three workgroups of the
// smallest shape and two of the next: their step with one, two and three on the
// busiest unit.  It holds one of the others: their step where few units run and
// where all do.  Fitted to times of products of 1 to 8960 rows, rows of whole
// cache lines and not, under every shape and split.  Over 600 random products
// with their weights in memory the plan that the model picks is 0.6 to 4.6%
// slower than the best shape and split (means by type and rows), and at worst
// 38% (978 x 256 x 4160 bf16: four steps a tile).  The largest shape that fills
// the units, else a split that does, takes 178 us instead of 86 for 700 x 14336
// x 4096 bf16.
// Where memory and caches want different plans, memory's is taken: a layer's
// weights are read from there, the other layers' having passed through the
// caches since.  A step of 0.42 for two 64 x 64 bf16 tiles a unit, as measured
// from the caches, changes 47 of 360 plans of 33 to 2048 rows; they are 10%
// slower from memory on average and 5% faster from the caches (256 x 4096 x 6144:
// one round of 64 x 64 tiles 35.5 and 25.1 us, 128 x 128 tiles in two parts 31.8
// and 29.9; gated 300 x 4096 x 6144 69.5 and 55.2, 57.2 and 52.3).
struct ShapeCost {
  float start, step[3];
};
constexpr ShapeCost kCosts[4][kNumShapes] = {
    // fp32
    {{1.6f, {0.27f, 0.41f, 0.54f}}, {1.5f, {0.64f, 1.18f}}, {2.3f, {1.95f, 2.22f}}, {5.0f, {7.4f, 8.0f}}},
    // bf16
    {{1.2f, {0.19f, 0.27f, 0.36f}}, {1.6f, {0.32f, 0.50f}}, {2.6f, {0.56f, 0.68f}}, {4.7f, {0.86f, 1.42f}}},
    // e4m3 with bf16 outputs, with fp32 outputs
    {{1.4f, {0.18f, 0.27f, 0.35f}}, {1.9f, {0.33f, 0.48f}}, {2.8f, {0.57f, 0.69f}}, {4.0f, {0.79f, 1.50f}}},
    {{1.8f, {0.29f, 0.36f, 0.39f}}, {2.2f, {0.35f, 0.60f}}, {2.3f, {1.05f, 1.14f}}, {4.3f, {3.4f, 3.7f}}}};
// Where B is read once and does not fit a cache, a compute unit loads no more
// than this a microsecond (a probe that only loads: 46 KB from memory).
constexpr float kColdRate = 55e3f;
constexpr float kColdBytes = 50e6f;
// The smallest gated tile has two waves to load with, not four.
constexpr float kGatedSmall = 1.4f;
constexpr float kJoinStart = 2.6f;       // a second launch
constexpr float kJoinPart = 0.1f;        // a part of a tile
constexpr float kJoinPerByte = 0.2e-6f;  // partials written and read again

// gemm_rows_kernel: its start, a step of each of its waves for 16 rows of B and
// for a row of A (fp32: more products a byte), and what it reads of B a
// microsecond at most.  Fitted to times of 1 to 32 rows beside the other shapes':
// over 260 random products of such rows the pick is 0.6 to 2.3% slower than the
// best (means by type), and at worst 27% (3 x 11776 x 14976 e4m3 to fp32).
constexpr float kRowsStart = 0.5f, kRowsStepB = 0.6f, kRowsStepA = 0.028f, kRowsF32 = 1.5f;
constexpr float kRowsRate = 4.4e6f;

// Reduction-major bf16 tiles against row-major ones, by shape: a row of the
// smallest is 64 bytes, half a cache line; the middle one's workgroups, two a
// unit, share most of what they load (gradients of 300 x 2048 x 2048 in one
// launch: 57, 32 and 41 us in the three shapes).
constexpr float kColumnsCost[kNumShapes] = {1.7f, 0.85f, 1.2f, 1.05f};

// workgroups of a shape that a compute unit holds
constexpr int units_hold(int shape) { return shape < 2 ? 3 - shape : 1; }
// a step where all units hold what they can
constexpr float full_step(const ShapeCost& c, int shape) { return c.step[shape == 0 ? 2 : 1]; }

// Operands from which on whole cache lines are worth loading.
constexpr float kLineBytes = 30e6f;

constexpr int64_t kMaxPartials = 64 << 20;  // bytes
constexpr int64_t kMostParts = 16;          // of a tile
constexpr int kPairParts = 4;               // choices of them in one launch: 1, 2, 4, 8

// `n` workgroups of `steps` steps.
float round_time(const ShapeCost& c, int shape, int64_t n, int64_t steps) {
  const int64_t cap = (int64_t)units_hold(shape) * kComputeUnits;
  const int64_t full = n / cap, rest = n % cap;
  float us = full * (c.start + steps * full_step(c, shape));
  if (rest) {
    const float step = units_hold(shape) > 1
                           ? c.step[(rest - 1) / kComputeUnits]
                           : c.step[0] + (c.step[1] - c.step[0]) * rest / kComputeUnits;
    us += c.start + steps * step;
  }
  return us;
}

// A tile of 128 or 256 rows for at most 64 of them is never the fastest (none of
// 400000 random products' plans had one), and its partials are the largest.
bool shape_allowed(int shape, int64_t M) { return shape < 2 || M > 64; }

// few rows
float rows_time(Form form, int type, int64_t M, int64_t N, int64_t kb) {
  const int64_t rounds = ((N + 15) / 16 + kComputeUnits - 1) / kComputeUnits;
  const int64_t turns = (kb + kRowsWaves * kStepBytes - 1) / (kRowsWaves * kStepBytes);
  const int each = form == kGatedForm ? 2 : 1;
  const float a = M * kRowsStepA * (type == LORA_F32 ? kRowsF32 : 1.f);
  return std::max(rounds * (kRowsStart + turns * (each * kRowsStepB + a)),
                  (float)(each * N) * (float)kb / kRowsRate);
}

}  // namespace

GemmPlan gemm_plan(int32_t dtype, int32_t out_dtype, Form form, int64_t M, int64_t N,
                   int64_t kb) {
  const int64_t width = form == kGatedForm ? 2 * N : N;  // rows of B
  const int64_t steps = (kb + kStepBytes - 1) / kStepBytes;
  const int type = dtype == LORA_E4M3 && out_dtype == LORA_F32 ? 3 : dtype;
  const bool few = M <= kMostRows && (form == kLinearForm || form == kGatedForm);
  int only_shape = -1, only_parts = 0;
  if (const char* e = std::getenv("LORA_GEMM_PLAN")) {  // tuning override: shape,parts
    char* end = nullptr;
    const long shape = std::strtol(e, &end, 10);
    const long parts = *end == ',' ? std::strtol(end + 1, nullptr, 10) : 0;
    if (shape >= 0 && shape < kNumShapes + few) only_shape = (int)shape;
    if (parts >= 1 && parts <= 64) only_parts = (int)parts;
  }
  GemmPlan best{};
  if (few && (only_shape < 0 || only_shape == kRowsShape))
    best = {kRowsShape, 1, 1, 0, rows_time(form, type, M, N, kb)};
  if (only_shape == kRowsShape) return best;
  for (int shape = 0; shape < kNumShapes; ++shape) {
    if (only_shape >= 0 ? shape != only_shape : !shape_allowed(shape, M)) continue;
    const TileShape& sh = kShapes[shape];
    ShapeCost c = kCosts[type][shape];
    if (M <= sh.bm && (float)(M + width) * (float)kb > kColdBytes)
      for (int k = 0; k < units_hold(shape); ++k)
        c.step[k] = std::max(c.step[k], (k + 1) * (sh.bm + sh.bn) * kStepBytes / kColdRate);
    if (form == kGatedForm && shape == 0)
      for (float& step : c.step) step *= kGatedSmall;
    if ((form == kGradX || form == kGradW) && dtype == LORA_BF16)
      for (float& step : c.step) step *= kColumnsCost[shape];
    const int64_t t = ((M + sh.bm - 1) / sh.bm) * ((width + sh.bn - 1) / sh.bn);
    // Whole rounds of tiles, one a compute unit, are not split; the tiles of the
    // last round may be, where they leave compute units idle.
    const int64_t rest = t % kComputeUnits;
    for (int64_t s = 1; s <= kMostParts; ++s) {
      const int64_t want = only_parts ? only_parts : s;
      const int64_t per = (steps + want - 1) / want, parts = (steps + per - 1) / per;
      GemmPlan g{shape, (int32_t)t, 1, 0, 0.f};
      float us = 0.f, join = 0.f;
      if (parts > 1 && rest) {
        const int64_t bytes = rest * parts * sh.bm * sh.bn * 4;
        if (bytes > kMaxPartials && !only_parts) break;
        g = {shape, (int32_t)(t - rest), (int32_t)parts, bytes, 0.f};
        us = round_time(c, shape, t - rest, steps) + round_time(c, shape, rest * parts, per);
        join = kJoinStart + parts * kJoinPart + bytes * kJoinPerByte;
      } else {
        us = round_time(c, shape, t, steps);
      }
      if (join > 0.f) us += join + 0.3f;  // (a tie goes to one launch)
      g.us = us;
      if (best.us == 0.f || us < best.us) best = g;
      if (only_parts || rest == 0 || rest * s > 4 * kComputeUnits) break;
    }
  }
  return best;
}

// What the partials of a product take at most, over the plans of all M up to this
// one and all reductions up to kb bytes: of one launched by itself (a split is
// not refined once it makes more than four workgroups a unit), or of one that
// shares its launch.
static int64_t partials_bound(Form form, int64_t M, int64_t N, int64_t kb, bool pair) {
  const int64_t width = form == kGatedForm ? 2 * N : N;
  const int64_t steps = (kb + kStepBytes - 1) / kStepBytes;
  const int64_t parts = std::min<int64_t>(pair ? 1 << (kPairParts - 1) : kMostParts, steps);
  int64_t bytes = 0;
  if (parts < 2) return 0;
  for (int shape = 0; shape < (pair ? kPairShapes : kNumShapes); ++shape) {
    if (!pair && !shape_allowed(shape, M)) continue;
    const TileShape& sh = kShapes[shape];
    const int64_t t = ((M + sh.bm - 1) / sh.bm) * ((width + sh.bn - 1) / sh.bn);
    const int64_t rest = std::min<int64_t>(t, kComputeUnits - 1);
    const int64_t n = pair ? rest * parts : std::min(rest * parts, 4 * kComputeUnits + rest);
    bytes = std::max(bytes, n * sh.bm * sh.bn * 4);
  }
  return std::min(bytes, kMaxPartials);
}

// The workspace that a product asks for: enough for every M up to this one, so
// that a buffer for the largest batch serves the smaller ones, whose plans may
// split more.
static int64_t gemm_workspace(const GemmPlan& plan, Form form, int64_t M, int64_t N, int64_t kb) {
  return std::max(plan.ws_bytes,  // (a forced plan may take more)
                  partials_bound(form, M, N, kb, false));
}

namespace {

void fill_plan(GemmArgs& a, const GemmPlan& plan, Form form, void* ws) {
  if (plan.shape == kRowsShape) return;
  const TileShape sh = kShapes[plan.shape];
  const int width = form == kGatedForm ? 2 * a.N : a.N;
  a.tiles_m = (a.M + sh.bm - 1) / sh.bm;
  a.tiles_n = (width + sh.bn - 1) / sh.bn;
  a.whole = plan.whole;
  a.splits = plan.splits;
  a.part = (float*)ws;
  const char* force = std::getenv("LORA_GEMM_LINES");  // tuning override: 0 or 1
  a.lines = force ? *force == '1' : (float)(a.M + width) * (float)a.kb > kLineBytes;
}

int32_t join_parts(const GemmArgs& a, const GemmPlan& plan, Form form, hipStream_t st) {
  if (plan.splits == 1) return LORA_OK;
  const TileShape sh = kShapes[plan.shape];
  const bool gated = form == kGatedForm;
  const int rest = a.tiles_m * a.tiles_n - a.whole;
  const dim3 grid((unsigned)((rest * (sh.bm * (gated ? sh.bn / 2 : sh.bn) / 8) + 255) / 256));
  if (gated)
    hipLaunchKernelGGL(join_kernel<true>, grid, dim3(256), 0, st, a, sh.bm, sh.bn);
  else
    hipLaunchKernelGGL(join_kernel<false>, grid, dim3(256), 0, st, a, sh.bm, sh.bn);
  return check_launch("join of the K splits");
}

}  // namespace

int32_t gemm_run(int32_t dtype, Form form, const GemmPlan& plan, GemmArgs a, void* ws,
                 hipStream_t st) {
  fill_plan(a, plan, form, ws);
  int32_t e = dtype == LORA_BF16   ? gemm_launch_bf16(form, plan.shape, a, st)
              : dtype == LORA_E4M3 ? gemm_launch_e4m3(form, plan.shape, a, st)
                                   : gemm_launch_f32(form, plan.shape, a, st);
  return e ? e : join_parts(a, plan, form, st);
}

namespace {

// ---------------------------------------------------------------- backward

// dpre from dout and what the forward pass saved: with value a(g) and slope
// a'(g) of the activation at the gate g,
//   d gate = dout * up * a'(g),   d up = dout * a(g).
// Eight columns a thread, five reads and writes of one [T][I] array each: 590 MB
// in 95 us at 4096 x 14336 bf16 (6.2 TB/s).
template <int DT>
__global__ __launch_bounds__(256) void gate_grad_kernel(const void* dout, const void* pre,
                                                        void* dpre, int64_t T, int I, int act) {
  const int per = I / 8;
  for (int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x; id < T * per;
       id += (int64_t)gridDim.x * 256) {
    const int64_t m = id / per;
    const int n = (int)(id % per) * 8;
    float d[8], g[8], u[8];
    load8(dout, m * I + n, 8, DT, d);
    load8(pre, m * 2 * I + n, 8, DT, g);
    load8(pre, m * 2 * I + I + n, 8, DT, u);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float value, slope;
      act_curve<DT == LORA_BF16>(act, g[j], value, slope);
      g[j] = d[j] * u[j] * slope;
      u[j] = d[j] * value;
    }
    store8(dpre, m * 2 * I + n, 8, DT, g);
    store8(dpre, m * 2 * I + I + n, 8, DT, u);
  }
}

__global__ __launch_bounds__(256) void clear_kernel(bk_u32x4* p, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
    p[i] = bk_u32x4{0, 0, 0, 0};
}

// The two products: one after the other (they share the workspace), or in one
// launch (each has its own part).
struct BackwardPlan {
  bool pair;
  GemmPlan dx, dw;
  int64_t dw_at, total;
};

// What separate launches cost beside the estimates of their products: the gap
// between them, in which the compute units drain and fill (measured 3 to 18 us
// at 300 to 2567 rows).
constexpr float kLaunchGap = 10.f;

// Both products in tiles of one shape, each split into up to eight parts: the
// time of the longest workgroup, or of all of them dealt over the units.
// `only`: a forced choice, "shape,i,j" with 2^i and 2^j parts.
BackwardPlan pair_plan(int32_t dtype, const int64_t (&M)[2], int64_t N, const int64_t (&kb)[2],
                       const char* only) {
  BackwardPlan best{};
  float best_us = 0.f;
  for (int shape = 0; shape < kPairShapes; ++shape) {
    if (only && only[0] != '0' + shape) continue;
    const TileShape& sh = kShapes[shape];
    ShapeCost c = kCosts[dtype][shape];
    if (dtype == LORA_BF16)
      for (float& s : c.step) s *= kColumnsCost[shape];
    const float cap = (float)(units_hold(shape) * kComputeUnits), step = full_step(c, shape);
    GemmPlan g[2][kPairParts];
    float longest[2][kPairParts], work[2][kPairParts], join[2][kPairParts];
    for (int p = 0; p < 2; ++p) {
      const int64_t t = ((M[p] + sh.bm - 1) / sh.bm) * ((N + sh.bn - 1) / sh.bn);
      const int64_t steps = (kb[p] + kStepBytes - 1) / kStepBytes, rest = t % kComputeUnits;
      for (int i = 0; i < kPairParts; ++i) {
        const int64_t per = (steps + (1 << i) - 1) >> i, parts = (steps + per - 1) / per;
        const bool split = parts > 1 && rest;
        const int64_t bytes = split ? rest * parts * sh.bm * sh.bn * 4 : 0;
        g[p][i] = {shape, (int32_t)(split ? t - rest : t), (int32_t)(split ? parts : 1), bytes, 0.f};
        const float whole = c.start + steps * step, part = c.start + per * step;
        longest[p][i] = c.start + (t >= kComputeUnits || !split ? steps : per) * c.step[0];
        work[p][i] = split ? (t - rest) * whole + rest * parts * part : t * whole;
        join[p][i] = split ? kJoinStart + parts * kJoinPart + bytes * kJoinPerByte : 0.f;
      }
    }
    for (int i = 0; i < kPairParts; ++i)
      for (int j = 0; j < kPairParts; ++j) {
        if (only ? only[2] != '0' + i || only[4] != '0' + j
                 : g[0][i].ws_bytes + g[1][j].ws_bytes > kMaxPartials)
          continue;
        const float us = std::max(std::max(longest[0][i], longest[1][j]),
                                  (work[0][i] + work[1][j]) / cap) +
                         join[0][i] + join[1][j];
        if (best_us == 0.f || us < best_us * 0.97f) {
          best = {true, g[0][i], g[1][j], align_up(g[0][i].ws_bytes, 256), 0};
          best.dx.us = best_us = us;
        }
      }
  }
  best.total = best.dw_at + best.dw.ws_bytes;
  return best;
}

BackwardPlan backward_plan(const lora_gated_desc& d, int64_t T, bool dx, bool dw) {
  BackwardPlan b{};
  const int64_t e = esize(d.dtype), K = d.in_features, I2 = 2 * (int64_t)d.inter_features;
  if (dx) b.dx = gemm_plan(d.dtype, d.dtype, kGradX, T, K, e * I2);
  if (dw) b.dw = gemm_plan(d.dtype, d.dtype, kGradW, I2, K, e * T);
  b.total = std::max(b.dx.ws_bytes, b.dw.ws_bytes);
  if (dx && dw) {
    // tuning overrides: "shape,i,j", or anything else for separate launches
    const char* f = std::getenv("LORA_GRAD_PAIR");
    const bool forced = f && std::strlen(f) == 5 && f[0] >= '0' && f[0] < '0' + kPairShapes &&
                        f[2] >= '0' && f[2] < '0' + kPairParts && f[4] >= '0' && f[4] < '0' + kPairParts;
    if (!forced && (f || std::getenv("LORA_GEMM_PLAN"))) return b;
    BackwardPlan p = pair_plan(d.dtype, {T, I2}, K, {e * I2, e * T}, forced ? f : nullptr);
    p.total = std::max(p.total, b.total);  // (either gradient alone fits as well)
    if (forced || p.dx.us < b.dx.us + b.dw.us + kLaunchGap) return p;
  }
  return b;
}

// What the gradients ask for: enough for every T up to this one, and for either
// gradient alone.
int64_t backward_workspace(const BackwardPlan& plan, const lora_gated_desc& d, int64_t T, bool dx,
                           bool dw) {
  const int64_t e = esize(d.dtype), K = d.in_features, I2 = 2 * (int64_t)d.inter_features;
  int64_t n = plan.total;  // (a forced plan may take more)
  if (dx) n = std::max(n, partials_bound(kGradX, T, K, e * I2, false));
  if (dw) n = std::max(n, partials_bound(kGradW, I2, K, e * T, false));
  if (dx && dw) {
    const int64_t both = align_up(partials_bound(kGradX, T, K, e * I2, true), 256) +
                         partials_bound(kGradW, I2, K, e * T, true);
    n = std::max(n, std::min(both, kMaxPartials + 256));
  }
  return n;
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

int32_t check_rows(int32_t T) {
  if (T < 0) return fail(LORA_E_ARG, "T must be >= 0, got %d", T);
  if (T > kMaxRows)
    return fail(LORA_E_SHAPE, "T must be at most %lld, got %d", (long long)kMaxRows, T);
  return LORA_OK;
}

}  // namespace lora

using namespace lora;

extern "C" {

int64_t lora_linear_workspace_bytes(const lora_linear_desc* desc, int32_t T) {
  clear_error();
  if (int32_t e = check_linear(desc)) return e;
  if (int32_t e = check_rows(T)) return e;
  if (T == 0) return 0;
  const int64_t kb = desc->in_features * esize(desc->dtype);
  return gemm_workspace(
      gemm_plan(desc->dtype, desc->out_dtype, kLinearForm, T, desc->out_features, kb), kLinearForm,
      T, desc->out_features, kb);
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
  const GemmPlan plan = gemm_plan(desc->dtype, desc->out_dtype, kLinearForm, T, desc->out_features, kb);
  if (int32_t e = check_ws(ws, ws_bytes,
                           gemm_workspace(plan, kLinearForm, T, desc->out_features, kb)))
    return e;
  GemmArgs a{};
  a.A = (const char*)x;
  a.B = (const char*)w;
  a.sa = x_scale;
  a.sb = w_scale;
  a.bias = bias;
  a.delta = delta;
  a.residual = residual;
  a.out = out;
  a.kb = a.lda = a.ldb = kb;
  a.M = T;
  a.N = desc->out_features;
  a.out_dtype = desc->out_dtype;
  a.act = desc->act;
  return gemm_run(desc->dtype, kLinearForm, plan, a, ws, (hipStream_t)stream);
}

int64_t lora_gated_ffn_workspace_bytes(const lora_gated_desc* desc, int32_t T) {
  clear_error();
  if (int32_t e = check_gated(desc)) return e;
  if (int32_t e = check_rows(T)) return e;
  if (T == 0) return 0;
  const int64_t kb = desc->in_features * esize(desc->dtype);
  return gemm_workspace(
      gemm_plan(desc->dtype, desc->out_dtype, kGatedForm, T, desc->inter_features, kb), kGatedForm,
      T, desc->inter_features, kb);
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
  const GemmPlan plan = gemm_plan(desc->dtype, desc->out_dtype, kGatedForm, T, desc->inter_features, kb);
  if (int32_t e = check_ws(ws, ws_bytes,
                           gemm_workspace(plan, kGatedForm, T, desc->inter_features, kb)))
    return e;
  GemmArgs a{};
  a.A = (const char*)x;
  a.B = (const char*)w;
  a.sa = x_scale;
  a.sb = w_scale;
  a.delta = delta;
  a.pre = pre;
  a.out = out;
  a.kb = a.lda = a.ldb = kb;
  a.M = T;
  a.N = desc->inter_features;
  a.out_dtype = desc->out_dtype;
  a.act = desc->act;
  return gemm_run(desc->dtype, kGatedForm, plan, a, ws, (hipStream_t)stream);
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
  const bool dx = need_dx != 0, dw = need_dw != 0;
  return backward_workspace(backward_plan(*desc, T, dx, dw), *desc, T, dx, dw);
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
  const BackwardPlan b = backward_plan(*desc, T, dx != nullptr, dw != nullptr);
  if (int32_t e = check_ws(ws, ws_bytes,
                           backward_workspace(b, *desc, T, dx != nullptr, dw != nullptr)))
    return e;

  // (a grid holds less than 2^32 threads)
  const dim3 grid((unsigned)std::min<int64_t>(((int64_t)T * (I / 8) + 255) / 256, 1 << 23));
  if (desc->dtype == LORA_BF16)
    hipLaunchKernelGGL(gate_grad_kernel<LORA_BF16>, grid, dim3(256), 0, st, dout, pre, dpre,
                       (int64_t)T, I, desc->act);
  else
    hipLaunchKernelGGL(gate_grad_kernel<LORA_F32>, grid, dim3(256), 0, st, dout, pre, dpre,
                       (int64_t)T, I, desc->act);
  if (int32_t e = check_launch("gate gradient")) return e;

  GemmArgs a{};
  a.A = (const char*)dpre;
  a.lda = 2 * I * es;
  a.N = K;
  a.ldb = K * es;
  a.out_dtype = desc->dtype;
  a.act = LORA_ACT_NONE;
  GemmArgs ax = a, aw = a;
  ax.B = (const char*)w;
  ax.out = dx;
  ax.M = T;
  ax.kb = 2 * I * es;
  aw.B = (const char*)x;
  aw.out = dw;
  aw.M = 2 * I;
  aw.kb = T * es;
  if (b.pair) {
    fill_plan(ax, b.dx, kGradX, ws);
    fill_plan(aw, b.dw, kGradW, (char*)ws + b.dw_at);
    if (int32_t e = desc->dtype == LORA_BF16 ? gemm_launch_pair_bf16(b.dx.shape, ax, aw, st)
                                             : gemm_launch_pair_f32(b.dx.shape, ax, aw, st))
      return e;
    if (int32_t e = join_parts(ax, b.dx, kGradX, st)) return e;
    return join_parts(aw, b.dw, kGradW, st);
  }
  if (dx) {
    if (int32_t e = gemm_run(desc->dtype, kGradX, b.dx, ax, ws, st)) return e;
  }
  if (dw) {
    if (int32_t e = gemm_run(desc->dtype, kGradW, b.dw, aw, ws, st)) return e;
  }
  return LORA_OK;
}

}  // extern "C"
