// Gradients of the adapters' delta: from dy, with u = B^T dy and v = A x in rank
// space, dx += A^T u, dA = u x^T and dB = dy v^T summed over each adapter's rows.
//
// Launches, all over the host plan's records:
//   1 ranks   u and v of 64-row tiles (reductions over out and in features, cut
//             into parts where tiles are few)
//   2 join    adds the parts, where there are any
//   3 spread  dx of 64-row tiles by 512 columns; dA and dB of a piece of an
//             adapter's rows by 256 bytes of columns
//   4 sums    adds the partials of adapters whose rows were cut
//
// Every product is MFMA (16x16x32 bf16, 16x16x4 fp32).  The ranks are at most a
// few hundred, so that every product is bound by memory: x and dy are read twice
// (once for the ranks, once for the gradients), dx once in and out.  A bf16
// pool's u and v are held as sums of three bf16 values (24 bits): one product with
// fp32 operands is three with bf16 ones, which the loads hide.
#include <hip/hip_runtime.h>

#include "lora_delta.h"
#include "lora_gemm.h"

namespace lora {

namespace {

using gemm::barrier;
using gemm::bk_half4;
using gemm::bk_u32x2;
using gemm::kZeros;
using gemm::read_columns;
using gemm::wait_all_lds;

constexpr int kPlanes = 3;  // bf16 pieces of an fp32 value

struct DeltaArgs {
  const char* A;
  const char* B;
  const char* x;
  const char* dy;
  const char* dx_in;
  char* dx;
  float* dA;
  float* dB;
  const int32_t* perm;
  const int32_t* tiles;
  const int32_t* parts;
  const int32_t* multi;
  char* ranks;      // bf16: [planes][2 S][rows][padded]; fp32: [2 S][rows][padded]
  float* partial;   // [splits][2 S][rows][padded]
  float* grads;     // [partials][values of a slot]
  int32_t num_tiles, none_tiles, num_parts, num_multi;
  int32_t rows;     // with an adapter
  int32_t partials;
  int32_t all;      // rows of x, dy, dx
  int32_t max_loras, K, S, O, R;
  int32_t padded, blocks;
  int32_t chunk;
  int32_t accumulate;
  int32_t dx_blocks, dx_groups;  // workgroups of dx, of them for one tile
  int32_t out[LORA_MAX_SLICES], off[LORA_MAX_SLICES];
};

constexpr int es(int dt) { return dt == LORA_BF16 ? 2 : 4; }

__device__ __forceinline__ int64_t plane_values(const DeltaArgs& a) {
  return (int64_t)2 * a.S * a.rows * a.padded;
}

// ---- operands in LDS: rows of RB bytes, 16-byte pieces in an order that keeps
// the reads below free of bank conflicts
//
// Reduction contiguous, 128 bytes a row: piece p of row r is at place p ^ (r & 7).
__device__ __forceinline__ int row_place(int p, int r) { return p ^ (r & 7); }
// Reduction-major, one row a reduction index k: byte c of row k is at this one (its
// own inverse).  bf16: four lanes of a read take 8 bytes of rows k .. k + 3 and the
// lanes' groups rows 8 apart; fp32: the groups take 64 bytes of rows 8 apart.
template <int DT, int RB>
__device__ __forceinline__ int column_place(int c, int k) {
  if constexpr (DT == LORA_F32) {
    if constexpr (RB == 256) return c ^ (((k >> 3) & 3) << 6);
    if constexpr (RB == 128) return c ^ (((k >> 3) & 1) << 6);
    return c;
  }
  if constexpr (RB == 256) return c ^ (((k & 3) | ((k >> 3) & 1) << 2) << 5);
  if constexpr (RB == 128) return c ^ ((((k >> 1) & 1) | ((k >> 3) & 1) << 1) << 5);
  if constexpr (RB == 64) return c ^ (((k >> 3) & 1) << 5);
  return c;
}

// Operand fragment of 32 reduction indexes: lane (l, g) holds index l of the
// output's dimension and reduction indexes 8 g .. 8 g + 7, in both types (the
// fp32 instruction takes four at a time, one a group).
template <int DT>
struct Frag {
  bk_u32x4 v[DT == LORA_BF16 ? 1 : 2];
};
template <int DT>
__device__ __forceinline__ bk_f32x4 product(const Frag<DT>& a, const Frag<DT>& b, bk_f32x4 c) {
  if constexpr (DT == LORA_BF16) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bk_bf16x8, a.v[0]),
                                                   __builtin_bit_cast(bk_bf16x8, b.v[0]), c, 0, 0,
                                                   0);
  } else {
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a.v[s][j]),
                                                 __uint_as_float(b.v[s][j]), c, 0, 0, 0);
    return c;
  }
}
// from rows of 128 bytes (reduction contiguous), the s-th 32 indexes of them
template <int DT>
__device__ __forceinline__ Frag<DT> read_rows(const char* tile, int row, int g, int s) {
  Frag<DT> f;
  const char* at = tile + row * 128;
  if constexpr (DT == LORA_BF16) {
    f.v[0] = *reinterpret_cast<const bk_u32x4*>(at + 16 * row_place(4 * s + g, row));
  } else {
    f.v[0] = *reinterpret_cast<const bk_u32x4*>(at + 16 * row_place(2 * g, row));
    f.v[1] = *reinterpret_cast<const bk_u32x4*>(at + 16 * row_place(2 * g + 1, row));
  }
  return f;
}
// from a reduction-major tile: index l of the output's dimension is column
// col + (l >> 2) stride + (l & 3), reduction rows k0 ..
template <int DT, int RB>
__device__ __forceinline__ Frag<DT> read_cols(const char* tile, int k0, int col, int stride,
                                              int l16, int g) {
  Frag<DT> f;
  if constexpr (DT == LORA_BF16) {
    // 16 lanes read four rows of four pieces of four values; lane l gets column l
    const int k = k0 + 8 * g + (l16 >> 2), c = 2 * (col + (l16 & 3) * stride);
    const char* at = tile + k * RB + column_place<DT, RB>(c, k);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // (rows k and k + 4 have the same place of a column)
      const bk_u32x2 v =
          read_columns((__attribute__((address_space(3))) bk_half4*)(at + 4 * h * RB));
      f.v[0][2 * h] = v[0];
      f.v[0][2 * h + 1] = v[1];
    }
  } else {
    const int k = k0 + 8 * g, c = 4 * (col + (l16 >> 2) * stride + (l16 & 3));
    const char* at = tile + k * RB + column_place<DT, RB>(c, k);
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        f.v[s][j] = *reinterpret_cast<const uint32_t*>(at + (4 * s + j) * RB);
  }
  return f;
}

__device__ __forceinline__ void to_lds(const char* from, char* to) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)from,
                                   (__attribute__((address_space(3))) void*)to, 16, 0, 0);
}
__device__ __forceinline__ const char* zeros() { return reinterpret_cast<const char*>(kZeros); }

// At most N loads outstanding, and this wave's reads of LDS done; after a barrier
// the stage is there for every wave, and the stage before has been read by all.
template <int N>
__device__ __forceinline__ void wait_loads() {
  __builtin_amdgcn_s_waitcnt(wait_all_lds(N));
}

// An fp32 value as bf16 pieces, the largest first (each the nearest to what is
// left, so that three hold 24 bits).  An infinity or a NaN is in the first alone.
__device__ __forceinline__ void pieces_of(const float (&v)[4], bk_u32x2 (&p)[kPlanes]) {
  float left[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
  for (int k = 0; k < kPlanes; ++k) {
    const uint32_t a = bk_pack(left[0], left[1]), b = bk_pack(left[2], left[3]);
    p[k] = bk_u32x2{a, b};
    if (k + 1 == kPlanes) break;
    const float h[4] = {bk_lo(a), bk_hi(a), bk_lo(b), bk_hi(b)};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      left[i] = __builtin_fabsf(h[i]) < __builtin_inff() ? left[i] - h[i] : 0.f;
  }
}

typedef const __attribute__((address_space(4))) int32_t* scalar_words;

// Four values of a row's ranks, `at` their place in [2 S][rows][padded].
template <int DT>
__device__ __forceinline__ void put_ranks(const DeltaArgs& a, int64_t at, const float (&v)[4]) {
  if constexpr (DT == LORA_F32) {
    *reinterpret_cast<bk_f32x4*>(a.ranks + at * 4) = bk_f32x4{v[0], v[1], v[2], v[3]};
  } else {
    bk_u32x2 p[kPlanes];
    pieces_of(v, p);
#pragma unroll
    for (int k = 0; k < kPlanes; ++k)
      *reinterpret_cast<bk_u32x2*>(a.ranks + (k * plane_values(a) + at) * 2) = p[k];
  }
}

// ------------------------------------------------------------- 1: rank space
//
// One workgroup: 64 rows of one adapter, one rank block, one part of one
// reduction.  A ring of four stages of 128 bytes of the reduction (x or dy rows,
// and A rows or B's rows as columns), filled by direct loads; a wave multiplies 16
// rows with all ranks of the block.
template <int DT, int NT, bool kOut>  // kOut: u, from dy and B; else v, from x and A
__device__ __forceinline__ void ranks_tile(const DeltaArgs& a, char* lds, int slot, int rows,
                                           int first, int s, int rank0, int part) {
  constexpr int ES = es(DT), KS = 128 / ES;   // reduction indexes a stage
  constexpr int WB = 16 * NT * ES;            // bytes of a column row of B
  constexpr int XB = 64 * 128, STAGE = XB + 16 * NT * 128, NST = 4;
  constexpr int WL = (NT + 1) / 2;            // loads of a wave for the weights
  constexpr int LOADS = 2 + WL;
  static_assert(KS * WB == 16 * NT * 128, "");
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const int len = kOut ? a.out[s] : a.K;
  const int lo = part * a.chunk, hi = lo + a.chunk < len ? lo + a.chunk : len;
  const int nk = (hi - lo + KS - 1) / KS;

  // what this lane loads: two pieces of rows, WL pieces of the weights
  const char* xp[2];
  int xk[2];  // reduction index of the piece in a stage
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int r = 8 * (2 * wave + j) + (lane >> 3), p = row_place(lane & 7, r);
    const int t = r < rows ? a.perm[first + r] : -1;
    xk[j] = p * (16 / ES);
    xp[j] = t < 0 || t >= a.all ? nullptr
            : kOut ? a.dy + ((int64_t)t * a.O + a.off[s] + lo + xk[j]) * ES
                   : a.x + ((int64_t)t * a.K + lo + xk[j]) * ES;
  }
  const char* wp[WL];
  int wk[WL];
  int64_t step;
#pragma unroll
  for (int j = 0; j < WL; ++j) {
    const int i = NT == 1 ? wave & 1 : WL * wave + j;  // (NT = 1: two waves load the same)
    if constexpr (kOut) {
      const int o = i * 1024 + lane * 16, k = o / WB, c = column_place<DT, WB>(o % WB, k);
      wk[j] = k;
      wp[j] = rank0 + c / ES < a.R
                  ? a.B + (((int64_t)slot * a.O + a.off[s] + lo + k) * a.R + rank0) * ES + c
                  : nullptr;
      step = (int64_t)KS * a.R * ES;
    } else {
      const int r = i * 8 + (lane >> 3), p = row_place(lane & 7, r);
      wk[j] = p * (16 / ES);
      wp[j] = rank0 + r < a.R
                  ? a.A + ((((int64_t)slot * a.S + s) * a.R + rank0 + r) * a.K + lo + wk[j]) * ES
                  : nullptr;
      step = 128;
    }
  }
  auto load = [&](int kt) {
    char* to = lds + (kt % NST) * STAGE;
    const int left = kt < nk ? hi - lo - kt * KS : 0;
#pragma unroll
    for (int j = 0; j < 2; ++j)
      to_lds(xp[j] && xk[j] < left ? xp[j] + kt * 128 : zeros(), to + (2 * wave + j) * 1024);
#pragma unroll
    for (int j = 0; j < WL; ++j) {
      const int i = NT == 1 ? wave & 1 : WL * wave + j;
      to_lds(wp[j] && wk[j] < left ? wp[j] + kt * step : zeros(), to + XB + i * 1024);
    }
  };
  bk_f32x4 acc[NT] = {};
#pragma unroll
  for (int i = 0; i < NST - 1; ++i) load(i);
  for (int kt = 0; kt < nk; ++kt) {
    wait_loads<(NST - 2) * LOADS>();
    barrier();
    load(kt + NST - 1);  // (past the end: zeros, so that the count of loads holds)
    const char* at = lds + (kt % NST) * STAGE;
#pragma unroll
    for (int q = 0; q < KS / 32; ++q) {
      const Frag<DT> x = read_rows<DT>(at, 16 * wave + l16, g, q);
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const Frag<DT> w = kOut
            ? read_cols<DT, WB>(at + XB, 32 * q, 16 * i, 4, l16, g)
            : read_rows<DT>(at + XB, 16 * i + l16, g, q);
        acc[i] = product<DT>(w, x, acc[i]);
      }
    }
  }
  wait_loads<0>();
  // a lane holds ranks 4 g .. 4 g + 3 of every tile, of row l16
  const int row = 16 * wave + l16;
  if (row >= rows) return;
  const int q = kOut ? s : a.S + s;
  const int64_t at = ((int64_t)q * a.rows + first + row) * a.padded + rank0 + 4 * g;
  const bool whole = a.chunk >= len;
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const float v[4] = {acc[i][0], acc[i][1], acc[i][2], acc[i][3]};
    if (whole)
      put_ranks<DT>(a, at + 16 * i, v);
    else
      *reinterpret_cast<bk_f32x4*>(a.partial + part * plane_values(a) + at + 16 * i) = acc[i];
  }
}

__device__ __forceinline__ int parts_of(int len, int chunk) { return (len + chunk - 1) / chunk; }

// A record's rows, if they and its slot are in range.
__device__ __forceinline__ bool take(const DeltaArgs& a, const int32_t* rec, int limit, int& slot,
                                     int& rows, int& first) {
  slot = rec[0];
  rows = rec[1];
  first = rec[2];
  return slot >= 0 && slot < a.max_loras && rows > 0 && rows <= limit && first >= 0 &&
         first <= a.rows - rows;
}

template <int DT, int NT>
__global__ __launch_bounds__(256) void ranks_kernel(DeltaArgs a) {
  __shared__ __attribute__((aligned(16))) char lds[4 * (64 + 16 * NT) * 128];
  // jobs of a tile together, neighbouring tiles on one XCD: they share x, dy and
  // the weights in its L2
  const int item = xcd_item(blockIdx.x, gridDim.x);
  const int jobs = gridDim.x / a.num_tiles, tile = item / jobs;
  int job = item - tile * jobs, slot, rows, first;
  if (!take(a, a.tiles + 4 * tile, kDeltaTileRows, slot, rows, first)) return;
  const int rank0 = job % a.blocks * 16 * NT;
  job /= a.blocks;
  for (int s = 0; s < a.S; ++s) {
    const int n = parts_of(a.out[s], a.chunk);
    if (job < n)
      return ranks_tile<DT, NT, true>(a, lds, slot, rows, first, s, rank0, job);
    job -= n;
  }
  const int n = parts_of(a.K, a.chunk);
  ranks_tile<DT, NT, false>(a, lds, slot, rows, first, job / n, rank0, job % n);
}

// ------------------------------------------------------- 2: parts of the sums
template <int DT>
__global__ __launch_bounds__(256) void join_kernel(DeltaArgs a) {
  const int q = blockIdx.y;
  const int n = parts_of(q < a.S ? a.out[q] : a.K, a.chunk);
  if (n == 1) return;
  const int64_t values = (int64_t)a.rows * a.padded;
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= values) return;
  const int64_t at = q * values + i;
  bk_f32x4 s = *reinterpret_cast<const bk_f32x4*>(a.partial + at);
  for (int p = 1; p < n; ++p)
    s += *reinterpret_cast<const bk_f32x4*>(a.partial + p * plane_values(a) + at);
  const float v[4] = {s[0], s[1], s[2], s[3]};
  put_ranks<DT>(a, at, v);
}

// ------------------------------------------------------------- 3a: the input's
//
// 64 rows of one adapter (or none: a copy), 512 columns in steps of 64.  A step
// holds up to 128 ranks of A for its columns; a wave multiplies its 16 rows' u,
// which stay in registers where one step holds all ranks, with all 64 columns.
// The columns are dealt to the output's index so that a lane's are neighbours.
template <int DT>
__device__ __forceinline__ void dx_tile(const DeltaArgs& a, char* lds, int block) {
  constexpr int ES = es(DT), RB = 64 * ES, P = DT == LORA_BF16 ? 2 : 1;
  constexpr int RANKS = 128, STAGE = RANKS * RB, PL = STAGE / 4096;  // loads of a wave
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const int tile = block / a.dx_groups;
  const int c_lo = (block - tile * a.dx_groups) * kDeltaColumns;
  const int c_hi = c_lo + kDeltaColumns < a.K ? c_lo + kDeltaColumns : a.K;
  int slot, rows, first;
  const int32_t* rec = a.tiles + 4 * tile;
  const bool none = tile >= a.num_tiles;
  if (none) {
    rows = rec[1];
    first = rec[2];
    if (rows < 1 || rows > kDeltaTileRows || first < a.rows || first > a.all - rows) return;
  } else if (!take(a, rec, kDeltaTileRows, slot, rows, first)) {
    return;
  }
  const int row = 16 * wave + l16;
  int t = row < rows ? a.perm[first + row] : -1;
  if (t >= a.all) t = -1;
  if (none) {
    if (t < 0 || a.dx_in == a.dx) return;
    for (int c = c_lo + g * (16 / ES); c < c_hi; c += 64 / ES) {
      const int64_t at = ((int64_t)t * a.K + c) * ES;
      bk_u32x4 v = {0, 0, 0, 0};
      if (a.dx_in) v = *reinterpret_cast<const bk_u32x4*>(a.dx_in + at);
      *reinterpret_cast<bk_u32x4*>(a.dx + at) = v;
    }
    return;
  }

  const int all_ranks = a.S * a.padded;               // of the reduction
  const int groups = (all_ranks + RANKS - 1) / RANKS; // steps of a column step
  const int steps = (c_hi - c_lo + 63) / 64 * groups;
  // rank index i of the reduction is rank i % padded of slice i / padded
  auto load = [&](int st) {
    if (st >= steps) return;
    const int cs = st / groups, r0 = (st - cs * groups) * RANKS;
    char* to = lds + (st & 1) * STAGE;
#pragma unroll
    for (int j = 0; j < PL; ++j) {
      const int o = (wave * PL + j) * 1024 + lane * 16, k = o / RB;
      const int c = c_lo + cs * 64 + column_place<DT, RB>(o % RB, k) / ES;
      const int i = r0 + k, s = i / a.padded, r = i - s * a.padded;
      const bool in = i < all_ranks && r < a.R && c < a.K;
      to_lds(in ? a.A + ((((int64_t)slot * a.S + s) * a.R + r) * a.K + c) * ES : zeros(),
             to + (wave * PL + j) * 1024);
    }
  };
  Frag<DT> u[P][RANKS / 32];
  auto fetch = [&](int r0) {
#pragma unroll
    for (int q = 0; q < RANKS / 32; ++q) {
      const int i = r0 + 32 * q + 8 * g, s = i / a.padded, r = i - s * a.padded;
      const int64_t at = ((int64_t)s * a.rows + first + (row < rows ? row : 0)) * a.padded + r;
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const char* from = a.ranks + (p * plane_values(a) + at) * ES;
#pragma unroll
        for (int h = 0; h < (int)(sizeof(Frag<DT>) / 16); ++h)
          u[p][q].v[h] = i < all_ranks ? reinterpret_cast<const bk_u32x4*>(from)[h]
                                       : bk_u32x4{0, 0, 0, 0};
      }
    }
  };
  bk_f32x4 acc[4] = {};
  load(0);
  fetch(0);
  for (int st = 0; st < steps; ++st) {
    const int cs = st / groups, rg = st - cs * groups;
    if (groups > 1 && st) fetch(rg * RANKS);
    wait_loads<0>();
    barrier();
    load(st + 1);
    const char* at = lds + (st & 1) * STAGE;
    const int left = all_ranks - rg * RANKS;
#pragma unroll
    for (int q = 0; q < RANKS / 32; ++q) {
      if (32 * q >= left) break;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const Frag<DT> w = read_cols<DT, RB>(at, 32 * q, 4 * i, 16, l16, g);
#pragma unroll
        for (int p = 0; p < P; ++p) acc[i] = product<DT>(w, u[p][q], acc[i]);
      }
    }
    if (rg + 1 < groups) continue;
    // a lane holds columns 16 g .. 16 g + 15 of its row
    const int c = c_lo + cs * 64 + 16 * g;
    if (t >= 0) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (c + 8 * h >= c_hi) continue;
        float z[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) z[i] = acc[2 * h + (i >> 2)][i & 3];
        const int64_t to = (int64_t)t * a.K + c + 8 * h;
        if (a.dx_in) add8(z, a.dx_in, to, 8, DT);
        store8(a.dx, to, 8, DT, z);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = bk_f32x4{0.f, 0.f, 0.f, 0.f};
  }
}

// ------------------------------------------------------ 3b: the adapters' own
//
// One workgroup: a piece of an adapter's rows, 256 bytes of columns of x or dy,
// one rank block.  A ring of four stages of 32 rows; both operands are
// reduction-major (a row of memory is a reduction index).
template <int DT, int NT>
constexpr int grads_stage() {
  return 32 * 256 + (DT == LORA_BF16 ? kPlanes : 1) * 32 * 16 * NT * es(DT);
}
template <int DT, int NT, bool kOut>  // kOut: dB, from dy and v; else dA, from x and u
__device__ __forceinline__ void grads_tile(const DeltaArgs& a, char* lds, int slot, int rows,
                                           int first, int partial, int s, int rank0, int c0) {
  constexpr int ES = es(DT), P = DT == LORA_BF16 ? kPlanes : 1;
  constexpr int UB = 16 * NT * ES, UP = 32 * UB;         // a row of ranks, a plane's stage
  constexpr int XB = 32 * 256, STAGE = XB + P * UP, NST = 4;
  constexpr int RUNS = P * UP / 1024, UL = (RUNS + 3) / 4;  // 1 KB runs of ranks, a wave's
  constexpr int LOADS = 2 + UL;
  // waves: over the ranks where there are two tiles of them, and over the columns
  constexpr int WR = NT >= 2 ? 2 : 1, WC = 4 / WR;
  constexpr int CT = 256 / ES / 16 / WC, RT = NT / WR;   // a wave's tiles
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const int len = kOut ? a.out[s] : a.K;
  const int col = wave / WR * CT * 16, rank = wave % WR * RT * 16;
  const int nk = (rows + 31) / 32;

  const char* base = kOut ? a.dy : a.x;
  const int64_t stride = (int64_t)(kOut ? a.O : a.K) * ES;
  int xr[2], xc[2];  // row of a stage, and column of the row in memory or -1
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int o = (2 * wave + j) * 1024 + lane * 16;
    xr[j] = o / 256;
    const int c = column_place<DT, 256>(o % 256, xr[j]) / ES;
    xc[j] = c0 + c < len ? (kOut ? a.off[s] : 0) + c0 + c : -1;
  }
  const int q = kOut ? a.S + s : s;
  const char* up[UL];
  int ur[UL];
#pragma unroll
  for (int j = 0; j < UL; ++j) {
    const int i = UL * wave + j < RUNS ? UL * wave + j : RUNS - 1;  // (the last one again)
    const int o = i * 1024 + lane * 16, p = o / UP, k = o % UP / UB;
    const int c = column_place<DT, UB>(o % UB, k);
    ur[j] = k;
    up[j] = a.ranks + (p * plane_values(a) + ((int64_t)q * a.rows + first + k) * a.padded + rank0) *
                          ES + c;
  }
  // Tokens of the wave's eight rows of a stage, by scalar loads: these are not
  // counted with the direct loads, which stay in flight.  (Past the piece's last row
  // the words behind it are read, at most seven: records follow perm in the image.)
  struct Tokens {
    int t[8];
  };
  auto fetch = [&](int kt) {
    const int i = kt * 32 + 8 * wave, at = first + (i < rows ? i : rows - 1);
    const scalar_words p = (scalar_words)(uintptr_t)(a.perm + at);
    Tokens k;
#pragma unroll
    for (int j = 0; j < 8; ++j) k.t[j] = p[j];
    return k;
  };
  auto load = [&](int kt, const Tokens& tok) {
    char* to = lds + (kt % NST) * STAGE;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int t = g == 0   ? tok.t[4 * j]
                    : g == 1 ? tok.t[4 * j + 1]
                    : g == 2 ? tok.t[4 * j + 2]
                             : tok.t[4 * j + 3];
      const bool in = kt * 32 + xr[j] < rows && t >= 0 && t < a.all && xc[j] >= 0;
      to_lds(in ? base + t * stride + (int64_t)xc[j] * ES : zeros(), to + (2 * wave + j) * 1024);
    }
#pragma unroll
    for (int j = 0; j < UL; ++j) {
      const int i = UL * wave + j < RUNS ? UL * wave + j : RUNS - 1;
      to_lds(kt * 32 + ur[j] < rows ? up[j] + (int64_t)kt * 32 * a.padded * ES : zeros(),
             to + XB + i * 1024);
    }
  };
  bk_f32x4 acc[CT][RT] = {};
  Tokens tok = fetch(0);
#pragma unroll
  for (int i = 0; i < NST - 1; ++i) {
    const Tokens next = fetch(i + 1);
    load(i, tok);
    tok = next;
  }
  for (int kt = 0; kt < nk; ++kt) {
    wait_loads<(NST - 2) * LOADS>();
    barrier();
    const Tokens next = fetch(kt + NST);
    load(kt + NST - 1, tok);
    tok = next;
    const char* at = lds + (kt % NST) * STAGE;
    Frag<DT> xf[CT], uf[P][RT];
#pragma unroll
    for (int i = 0; i < CT; ++i)
      xf[i] = kOut ? read_cols<DT, 256>(at, 0, col + 16 * i, 4, l16, g)
                   : read_cols<DT, 256>(at, 0, col + 4 * i, 4 * CT, l16, g);
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int i = 0; i < RT; ++i)
        uf[p][i] = kOut ? read_cols<DT, UB>(at + XB + p * UP, 0, rank + 4 * i, 4 * RT, l16, g)
                        : read_cols<DT, UB>(at + XB + p * UP, 0, rank + 16 * i, 4, l16, g);
#pragma unroll
    for (int p = P - 1; p >= 0; --p)  // the smallest first
#pragma unroll
      for (int i = 0; i < CT; ++i)
#pragma unroll
        for (int j = 0; j < RT; ++j)
          acc[i][j] = kOut ? product<DT>(uf[p][j], xf[i], acc[i][j])
                           : product<DT>(xf[i], uf[p][j], acc[i][j]);
  }
  wait_loads<0>();

  const int64_t values = (int64_t)a.R * ((int64_t)a.S * a.K + a.O);
  const bool add = partial < 0 && a.accumulate;
  auto put = [&](float* to, const bk_f32x4& v) {
    bk_f32x4* p = reinterpret_cast<bk_f32x4*>(to);
    *p = add ? *p + v : v;
  };
  if constexpr (!kOut) {
    // a lane holds columns 4 CT g + 4 i .. + 3 of rank l16 of every rank tile
    float* to = partial < 0 ? a.dA + (int64_t)slot * a.S * a.R * a.K : a.grads + partial * values;
#pragma unroll
    for (int j = 0; j < RT; ++j) {
      const int r = rank0 + rank + 16 * j + l16;
      if (r >= a.R) continue;
#pragma unroll
      for (int i = 0; i < CT; ++i) {
        const int c = c0 + col + 4 * CT * g + 4 * i;
        if (c < a.K) put(to + ((int64_t)s * a.R + r) * a.K + c, acc[i][j]);
      }
    }
  } else {
    // ranks 4 RT g + 4 j .. + 3 of column l16 of every column tile
    float* to = partial < 0 ? a.dB + (int64_t)slot * a.O * a.R
                            : a.grads + partial * values + (int64_t)a.S * a.R * a.K;
#pragma unroll
    for (int i = 0; i < CT; ++i) {
      const int c = c0 + col + 16 * i + l16;
      if (c >= len) continue;
#pragma unroll
      for (int j = 0; j < RT; ++j) {
        const int r = rank0 + rank + 4 * RT * g + 4 * j;
        if (r < a.R) put(to + (int64_t)(a.off[s] + c) * a.R + r, acc[i][j]);
      }
    }
  }
}

template <int DT, int NT>
constexpr int spread_lds() {
  const int dx = 2 * 128 * 64 * es(DT), grads = 4 * grads_stage<DT, NT>();
  return dx > grads ? dx : grads;
}
template <int DT, int NT>
__global__ __launch_bounds__(256) void spread_kernel(DeltaArgs a) {
  __shared__ __attribute__((aligned(16))) char lds[spread_lds<DT, NT>()];
  constexpr int CB = 256 / es(DT);
  const int nb = gridDim.x - a.dx_blocks;  // the gradients' workgroups, the long ones, first
  if ((int)blockIdx.x >= nb) {
    dx_tile<DT>(a, lds, xcd_item(blockIdx.x - nb, a.dx_blocks));
    return;
  }
  const int item = xcd_item(blockIdx.x, nb);
  const int jobs = nb / a.num_parts, part = item / jobs;
  int job = item - part * jobs, slot, rows, first;
  const int32_t* rec = a.parts + 4 * part;
  if (!take(a, rec, a.rows, slot, rows, first) || rec[3] < -1 || rec[3] >= a.partials) return;
  const int rank0 = job % a.blocks * 16 * NT;
  job /= a.blocks;
  for (int s = 0; s < a.S; ++s) {
    const int n = parts_of(a.out[s], CB);
    if (job < n)
      return grads_tile<DT, NT, true>(a, lds, slot, rows, first, rec[3], s, rank0, job * CB);
    job -= n;
  }
  const int n = parts_of(a.K, CB);
  grads_tile<DT, NT, false>(a, lds, slot, rows, first, rec[3], job / n, rank0, job % n * CB);
}

// ----------------------------------------------------- 4: cut adapters' sums
__global__ __launch_bounds__(256) void sums_kernel(DeltaArgs a) {
  const int32_t* rec = a.multi + 4 * blockIdx.y;
  const int slot = rec[0], from = rec[1], n = rec[2];
  if (slot < 0 || slot >= a.max_loras || from < 0 || n < 1 || from > a.partials - n) return;
  const int64_t of_a = (int64_t)a.S * a.R * a.K, of_b = (int64_t)a.O * a.R;
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= of_a + of_b) return;
  const float* p = a.grads + from * (of_a + of_b) + i;
  bk_f32x4 s = *reinterpret_cast<const bk_f32x4*>(p);
  for (int k = 1; k < n; ++k) s += *reinterpret_cast<const bk_f32x4*>(p + k * (of_a + of_b));
  float* to = i < of_a ? a.dA + slot * of_a + i : a.dB + slot * of_b + (i - of_a);
  bk_f32x4* d = reinterpret_cast<bk_f32x4*>(to);
  *d = a.accumulate ? *d + s : s;
}

template <int DT, int NT>
int32_t run(const DeltaArgs& a, hipStream_t st) {
  auto count = [&](int32_t width) {
    int64_t n = (int64_t)a.S * ((a.K + width - 1) / width);
    for (int s = 0; s < a.S; ++s) n += (a.out[s] + width - 1) / width;
    return n * a.blocks;
  };
  if (a.rows) {
    const int64_t blocks = a.num_tiles * count(a.chunk);
    if (blocks > INT32_MAX) return fail(LORA_E_SHAPE, "too many workgroups");
    hipLaunchKernelGGL((ranks_kernel<DT, NT>), dim3((uint32_t)blocks), dim3(256), 0, st, a);
    bool cut = a.K > a.chunk;
    for (int s = 0; s < a.S; ++s) cut |= a.out[s] > a.chunk;
    if (cut) {
      const int64_t values = (int64_t)a.rows * a.padded;
      hipLaunchKernelGGL(join_kernel<DT>, dim3((uint32_t)((values + 1023) / 1024), 2 * a.S),
                         dim3(256), 0, st, a);
    }
  }
  const int64_t grads = a.dA ? a.num_parts * count(256 / es(DT)) : 0;
  if (grads + a.dx_blocks > INT32_MAX) return fail(LORA_E_SHAPE, "too many workgroups");
  if (grads + a.dx_blocks)
    hipLaunchKernelGGL((spread_kernel<DT, NT>), dim3((uint32_t)(grads + a.dx_blocks)), dim3(256),
                       0, st, a);
  if (a.dA && a.num_multi) {
    const int64_t values = (int64_t)a.R * ((int64_t)a.S * a.K + a.O);
    hipLaunchKernelGGL(sums_kernel, dim3((uint32_t)((values + 1023) / 1024), a.num_multi),
                       dim3(256), 0, st, a);
  }
  return check_launch("gradients of the delta");
}

}  // namespace

}  // namespace lora

using namespace lora;

extern "C" int32_t lora_delta_backward(const lora_pool_desc* desc, const void* A_pool,
                                       const void* B_pool, const void* x, const void* dy,
                                       const void* dx_in, void* dx, float* dA, float* dB,
                                       int32_t T, const lora_delta_plan* plan, const void* image,
                                       int32_t accumulate, void* ws, int64_t ws_bytes,
                                       void* stream) {
  clear_error();
  Geo g;
  if (int32_t e = check_desc(desc, &g)) return e;
  if (int32_t e = check_rows(T)) return e;
  if (accumulate != 0 && accumulate != 1)
    return fail(LORA_E_ARG, "accumulate must be 0 or 1, got %d", accumulate);
  if (T == 0) return LORA_OK;
  if (int32_t e = delta_check_plan(g, T, plan)) return e;
  if (!A_pool || !B_pool || !x || !dy || !image)
    return fail(LORA_E_ARG, "A_pool, B_pool, x, dy and image must not be NULL");
  if ((dA != nullptr) != (dB != nullptr))
    return fail(LORA_E_ARG, "dA and dB go together: one of them is NULL");
  if (dx_in && !dx) return fail(LORA_E_ARG, "dx_in without dx");
  if (!dx && !dA) return fail(LORA_E_ARG, "dx, dA and dB are all NULL");
  const DeltaLayout l = delta_layout(g, T);
  if (!ws) return fail(LORA_E_ARG, "workspace is NULL");
  if (ws_bytes < l.total)
    return fail(LORA_E_WORKSPACE, "workspace holds %lld bytes, the call needs %lld",
                (long long)ws_bytes, (long long)l.total);
  const void* ptrs[] = {A_pool, B_pool, x, dy, dx_in, dx, dA, dB, image, ws};
  for (const void* p : ptrs)
    if (!aligned16(p)) return fail(LORA_E_ALIGN, "every buffer must be 16-byte aligned");

  const DeltaRanks r = delta_ranks(g.R);
  const int32_t* im = (const int32_t*)image;
  DeltaArgs a{};
  a.A = (const char*)A_pool;
  a.B = (const char*)B_pool;
  a.x = (const char*)x;
  a.dy = (const char*)dy;
  a.dx_in = (const char*)dx_in;
  a.dx = (char*)dx;
  a.dA = dA;
  a.dB = dB;
  a.perm = im + plan->off_perm;
  a.tiles = im + plan->off_tiles;
  a.parts = im + plan->off_parts;
  a.multi = im + plan->off_multi;
  a.ranks = (char*)ws + l.ranks;
  a.partial = (float*)((char*)ws + l.partial);
  a.grads = (float*)((char*)ws + l.grads);
  a.num_tiles = plan->tiles;
  a.none_tiles = plan->none_tiles;
  a.num_parts = plan->parts;
  a.num_multi = plan->multi;
  a.rows = plan->rows;
  a.partials = plan->partials;
  a.all = T;
  a.max_loras = g.max_loras;
  a.K = g.K;
  a.S = g.S;
  a.O = g.O;
  a.R = g.R;
  a.padded = r.padded;
  a.blocks = r.blocks;
  a.chunk = plan->chunk;
  a.accumulate = accumulate;
  for (int s = 0; s < g.S; ++s) a.out[s] = g.out[s], a.off[s] = g.off[s];
  a.dx_groups = (g.K + kDeltaColumns - 1) / kDeltaColumns;
  const int64_t tiles = (int64_t)plan->tiles + plan->none_tiles;
  if (dx && tiles * a.dx_groups > INT32_MAX / 2) return fail(LORA_E_SHAPE, "too many workgroups");
  a.dx_blocks = dx ? (int32_t)(tiles * a.dx_groups) : 0;
  const hipStream_t st = (hipStream_t)stream;
  if (g.dtype == LORA_BF16)
    return r.tiles == 1   ? run<LORA_BF16, 1>(a, st)
           : r.tiles == 2 ? run<LORA_BF16, 2>(a, st)
                          : run<LORA_BF16, 4>(a, st);
  return r.tiles == 1   ? run<LORA_F32, 1>(a, st)
         : r.tiles == 2 ? run<LORA_F32, 2>(a, st)
                        : run<LORA_F32, 4>(a, st);
}
