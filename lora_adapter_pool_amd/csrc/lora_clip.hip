// Gradient norms and clipping over many tensors.
//
//   norm_g = sqrt(sum of x^2 over group g's tensors)
//   out = round(x min(1, max_norm / norm_g))
//
// The tensors are cut into chunks on the host (once for a list of tensors), a
// workgroup takes a chunk, and chunks of a group follow each other, so that a
// group's norm is a sum of neighbouring partials in a fixed order.  Squares are
// summed in 64 bits: a square of fp32 or bf16 may be past fp32's range, and a sum
// of 10^9 of them would lose the last bits of fp32.
//
// Few chunks: two launches, and every workgroup of the second adds its group's
// partials again.  Many: a launch between the two adds them once.  The second
// pass goes through the chunks backwards: what the first pass read last is still
// in the last-level cache.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <vector>

#include "lora_block.h"

namespace lora {

namespace {

constexpr int kThreads = 256;
constexpr int kStep = kThreads * 8;      // elements a pass of a workgroup
constexpr int64_t kMinChunk = kStep, kMaxChunk = 16 * kStep;
constexpr int64_t kAimChunks = 2048;     // eight a compute unit
constexpr int32_t kMaxGroups = 1 << 20;
constexpr int64_t kMaxChunks = (1 << 24) - 1;  // a grid holds under 2^32 threads
// most chunks of a group whose partials every workgroup adds by itself: 0.5 to 1.3 us in
// the second pass where a launch between the two takes 2 to 4.6 (128 tensors in 64
// groups); for 7869 chunks 210 us where the launch (5) leaves it at 179
constexpr int kOwnSums = 512;

struct Chunk {
  uint64_t in, out;
  int32_t count, dtype, group, reserved;
};
static_assert(sizeof(Chunk) == 32, "");

struct ClipArgs {
  const Chunk* chunks;
  const int32_t* starts;  // [groups + 1]: a group's chunks
  double* partials;       // [chunks]
  double* totals;         // [groups], or nullptr: each workgroup adds the partials
  float* norms;
  int32_t n;
  float max_norm;
};

__device__ __forceinline__ double sum_group(double v, double* room) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
  if ((threadIdx.x & 63) == 0) room[threadIdx.x >> 6] = v;
  __syncthreads();
  v = 0.0;
  for (int i = 0; i < (int)(blockDim.x >> 6); ++i) v += room[i];
  return v;
}

template <int DT>
__device__ __forceinline__ double squares(const Chunk& c) {
  double s[2] = {0.0, 0.0};
#pragma unroll 4
  for (int i = threadIdx.x * 8; i < c.count; i += kStep) {
    float v[8];
    load8((const void*)c.in, i, c.count - i, DT, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) s[j & 1] = __builtin_fma((double)v[j], (double)v[j], s[j & 1]);
  }
  return s[0] + s[1];
}

__global__ __launch_bounds__(kThreads) void norm_partials(ClipArgs a) {
  __shared__ double room[kThreads / 64];
  const Chunk c = a.chunks[blockIdx.x];
  const double s = sum_group(c.dtype == LORA_BF16 ? squares<LORA_BF16>(c) : squares<LORA_F32>(c),
                             room);
  if (threadIdx.x == 0) a.partials[blockIdx.x] = s;
}

// A group's sum of squares, in the order of threads and waves.
__device__ __forceinline__ double total_of(const ClipArgs& a, int group, double* room) {
  double s = 0.0;
  for (int i = a.starts[group] + threadIdx.x; i < a.starts[group + 1]; i += blockDim.x)
    s += a.partials[i];
  return sum_group(s, room);
}

__global__ __launch_bounds__(1024) void norm_totals(ClipArgs a) {
  __shared__ double room[16];
  const double s = total_of(a, blockIdx.x, room);
  if (threadIdx.x == 0) {
    a.totals[blockIdx.x] = s;
    a.norms[blockIdx.x] = (float)__builtin_sqrt(s);
  }
}

template <int DT>
__device__ __forceinline__ void scale_chunk(const Chunk& c, float f) {
#pragma unroll 4
  for (int i = threadIdx.x * 8; i < c.count; i += kStep) {
    float v[8];
    load8((const void*)c.in, i, c.count - i, DT, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= f;
    store8((void*)c.out, i, c.count - i, DT, v);
  }
}

__global__ __launch_bounds__(kThreads) void clip_chunks(ClipArgs a) {
  __shared__ double room[kThreads / 64];
  const int id = a.n - 1 - (int)blockIdx.x;
  const Chunk c = a.chunks[id];
  const double s = a.totals ? a.totals[c.group] : total_of(a, c.group, room);
  const double norm = __builtin_sqrt(s);
  if (!a.totals && threadIdx.x == 0 && id == a.starts[c.group]) a.norms[c.group] = (float)norm;
  // (a norm that is infinite or NaN in fp32 clips nothing: the caller reads it there)
  const float n = (float)norm;
  const float f = n < __builtin_inff() && norm > (double)a.max_norm
                      ? (float)((double)a.max_norm / norm) : 1.f;
  if (f == 1.f && c.in == c.out) return;
  if (c.dtype == LORA_BF16)
    scale_chunk<LORA_BF16>(c, f);
  else
    scale_chunk<LORA_F32>(c, f);
}

int64_t bytes_of(int32_t dtype) { return dtype == LORA_BF16 ? 2 : 4; }

// Elements a chunk holds, for lists of `total` elements.
int64_t chunk_size(int64_t total) {
  int64_t c = (total / kAimChunks + kStep - 1) / kStep * kStep;
  return c < kMinChunk ? kMinChunk : c > kMaxChunk ? kMaxChunk : c;
}

int32_t check_grads(const lora_grad* g, int32_t n, int32_t groups, int64_t* chunks,
                    int64_t* size) {
  if (n < 0) return fail(LORA_E_ARG, "the number of tensors must be >= 0, got %d", n);
  if (groups < 1 || groups > kMaxGroups)
    return fail(LORA_E_SHAPE, "groups must be in [1, %d], got %d", kMaxGroups, groups);
  if (n && !g) return fail(LORA_E_ARG, "the list of tensors is NULL");
  int64_t total = 0;
  for (int32_t i = 0; i < n; ++i) {
    if (g[i].dtype != LORA_F32 && g[i].dtype != LORA_BF16)
      return fail(LORA_E_DTYPE, "tensor %d: dtype must be fp32 or bf16, got %d", i, g[i].dtype);
    if (g[i].count < 0 || g[i].count > (int64_t)1 << 40)
      return fail(LORA_E_SHAPE, "tensor %d: %lld elements", i, (long long)g[i].count);
    if (g[i].group < 0 || g[i].group >= groups)
      return fail(LORA_E_ID, "tensor %d: group %d of %d", i, g[i].group, groups);
    if (g[i].count && !g[i].grad) return fail(LORA_E_ARG, "tensor %d is NULL", i);
    const uint64_t mask = bytes_of(g[i].dtype) - 1;
    if (((uintptr_t)g[i].grad | (uintptr_t)g[i].out) & mask)
      return fail(LORA_E_ALIGN, "tensor %d is not aligned to its elements", i);
    total += g[i].count;
    if (total > kMaxChunks * kMaxChunk)
      return fail(LORA_E_SHAPE, "the tensors hold more than %lld elements",
                  (long long)(kMaxChunks * kMaxChunk));
  }
  *size = chunk_size(total);
  *chunks = 0;
  for (int32_t i = 0; i < n; ++i) *chunks += (g[i].count + *size - 1) / *size;
  if (*chunks > kMaxChunks)
    return fail(LORA_E_SHAPE, "the tensors hold more than %lld chunks", (long long)kMaxChunks);
  return LORA_OK;
}

int64_t starts_bytes(int32_t groups) { return align_up((int64_t)(groups + 1) * 4, 32); }

int32_t check_list(const lora_grad_list* l) {
  if (!l) return fail(LORA_E_ARG, "the list is NULL");
  if (l->groups < 1 || l->groups > kMaxGroups || l->chunks < 0 || l->chunks > kMaxChunks ||
      l->most_chunks < 0 || l->most_chunks > l->chunks || l->empty < 0 ||
      l->empty > l->groups || (l->separate != 0 && l->separate != 1) ||
      l->bytes != starts_bytes(l->groups) + (int64_t)l->chunks * (int64_t)sizeof(Chunk))
    return fail(LORA_E_ARG, "the list was not filled in by lora_grad_list_build");
  return LORA_OK;
}

}  // namespace

}  // namespace lora

using namespace lora;

extern "C" int64_t lora_grad_list_bytes(const lora_grad* grads, int32_t n, int32_t groups) {
  clear_error();
  int64_t chunks, size;
  if (int32_t e = check_grads(grads, n, groups, &chunks, &size)) return e;
  return starts_bytes(groups) + chunks * (int64_t)sizeof(Chunk);
}

extern "C" int32_t lora_grad_list_build(const lora_grad* grads, int32_t n, int32_t groups,
                                        void* image, int64_t image_bytes, lora_grad_list* list) {
  clear_error();
  int64_t chunks, size;
  if (int32_t e = check_grads(grads, n, groups, &chunks, &size)) return e;
  const int64_t need = starts_bytes(groups) + chunks * (int64_t)sizeof(Chunk);
  if (!image || !list) return fail(LORA_E_ARG, "image and list must not be NULL");
  if (image_bytes < need)
    return fail(LORA_E_WORKSPACE, "image holds %lld bytes, the list needs %lld",
                (long long)image_bytes, (long long)need);
  // No byte may be read or written for two tensors: they would be scaled twice.
  struct Range {
    uint64_t from, to;
  };
  std::vector<Range> ranges;
  try {
    ranges.reserve(2 * (size_t)n);
  } catch (...) {
    return fail(LORA_E_WORKSPACE, "no host memory for %d tensors", n);
  }
  for (int32_t i = 0; i < n; ++i) {
    if (!grads[i].count) continue;
    const uint64_t b = (uint64_t)(grads[i].count * bytes_of(grads[i].dtype));
    const uint64_t in = (uint64_t)(uintptr_t)grads[i].grad;
    const uint64_t out = (uint64_t)(uintptr_t)grads[i].out;
    ranges.push_back({in, in + b});
    if (out && out != in) ranges.push_back({out, out + b});
  }
  std::sort(ranges.begin(), ranges.end(),
            [](const Range& a, const Range& b) { return a.from < b.from; });
  for (size_t i = 1; i < ranges.size(); ++i)
    if (ranges[i].from < ranges[i - 1].to)
      return fail(LORA_E_ARG, "two tensors of the list overlap");

  int32_t* starts = (int32_t*)image;
  Chunk* out = (Chunk*)((char*)image + starts_bytes(groups));
  for (int64_t i = 0; i < starts_bytes(groups) / 4; ++i) starts[i] = 0;
  for (int32_t i = 0; i < n; ++i)
    starts[grads[i].group + 1] += (int32_t)((grads[i].count + size - 1) / size);
  int32_t most = 0, empty = 0;
  for (int32_t g = 0; g < groups; ++g) {
    most = std::max(most, starts[g + 1]);
    empty += starts[g + 1] == 0;
    starts[g + 1] += starts[g];
  }
  // each group's next chunk: its start, which the loop after this one puts back
  bool separate = false;
  for (int32_t i = 0; i < n; ++i) {
    const int64_t e = bytes_of(grads[i].dtype);
    const uint64_t in = (uint64_t)(uintptr_t)grads[i].grad;
    const uint64_t to = grads[i].out ? (uint64_t)(uintptr_t)grads[i].out : in;
    separate |= grads[i].count && to != in;
    for (int64_t at = 0; at < grads[i].count; at += size)
      out[starts[grads[i].group]++] =
          Chunk{in + at * e, to + at * e, (int32_t)std::min(size, grads[i].count - at),
                grads[i].dtype, grads[i].group, 0};
  }
  for (int32_t g = groups; g > 0; --g) starts[g] = starts[g - 1];
  starts[0] = 0;
  *list = lora_grad_list{(int32_t)chunks, groups, most, empty, separate ? 1 : 0, 0, need};
  return LORA_OK;
}

extern "C" int64_t lora_clip_grads_workspace_bytes(const lora_grad_list* list) {
  clear_error();
  if (int32_t e = check_list(list)) return e;
  return 8 * ((int64_t)list->chunks + list->groups);
}

extern "C" int32_t lora_clip_grads(const lora_grad_list* list, const void* image, float max_norm,
                                   float* norms, void* ws, int64_t ws_bytes, void* stream) {
  clear_error();
  if (int32_t e = check_list(list)) return e;
  if (!(max_norm >= 0.f)) return fail(LORA_E_ARG, "max_norm must be >= 0, got %g", max_norm);
  if (!norms || !image) return fail(LORA_E_ARG, "norms and the list's image must not be NULL");
  const int64_t need = lora_clip_grads_workspace_bytes(list);
  if (!ws) return fail(LORA_E_ARG, "workspace is NULL");
  if (ws_bytes < need)
    return fail(LORA_E_WORKSPACE, "workspace holds %lld bytes, the call needs %lld",
                (long long)ws_bytes, (long long)need);
  if (!aligned16(image) || !aligned16(norms) || !aligned16(ws))
    return fail(LORA_E_ALIGN, "image, norms and workspace must be 16-byte aligned");
  const hipStream_t st = (hipStream_t)stream;
  const bool write = max_norm < __builtin_inff() || list->separate;
  // (groups without a chunk have no workgroup that writes their norm)
  const bool own = write && list->most_chunks <= kOwnSums && !list->empty;
  ClipArgs a{(const Chunk*)((const char*)image + starts_bytes(list->groups)),
             (const int32_t*)image,
             (double*)ws,
             own ? nullptr : (double*)ws + list->chunks,
             norms,
             list->chunks,
             max_norm};
  if (list->chunks)
    hipLaunchKernelGGL(norm_partials, dim3(list->chunks), dim3(kThreads), 0, st, a);
  if (!own) {
    const int nt = list->most_chunks > 256 ? 1024 : 256;
    hipLaunchKernelGGL(norm_totals, dim3(list->groups), dim3(nt), 0, st, a);
  }
  if (write && list->chunks)
    hipLaunchKernelGGL(clip_chunks, dim3(list->chunks), dim3(kThreads), 0, st, a);
  return check_launch("gradient norm");
}
