// Gradients of the adapters' delta: from dy, with u = B^T dy and v = A x in rank
// space, dx += A^T u, dA = u x^T and dB = dy v^T summed over each adapter's rows.
//
// Launches, all over the host plan's records:
//   1 ranks  u and v of 64-row tiles (reductions over out and in features, cut
//            into parts where tiles are few)
//   2 join   adds the parts, where there are any
//   3 dx     of 64-row tiles by 256 bytes of columns, and
//   4 grads  dA and dB of a piece of an adapter's rows by 512 bytes of columns, in
//            one launch where both are wanted: they read the same rank space, and
//            the end of one fills with the other (8704 x 4096 x 4096 168 -> 152 us,
//            32 rows 13.3 -> 9.9)
//   5 sums   adds the partials of adapters whose rows were cut
//
// Every product is MFMA (16x16x32 bf16, 16x16x4 fp32).  The ranks are at most a
// few hundred, so that every product is bound by memory: x and dy are read twice
// (once for the ranks, once for the gradients), dx once in and out.  A bf16
// pool's u and v enter every product as sums of three bf16 values (24 bits): one
// product with fp32 operands is three with bf16 ones, which the loads hide (matrix units
// are busy 20 to 26% of the gradients' cycles; a third piece for dx, which had two, left 8704 x 4096
// x 4096 at 142 us and took gate/up of 8960 rows from 459 to 461).
//
// Measured (us, bf16, 64 ranks): 8704 x 4096 x 4096 of 16 adapters 142 to 146 (floor of
// its 335 MB at a copy's rate 65), 8960 x 4096 x 2 x 14336 of 28 adapters 442 to 478 by
// the card (230); 256 x 4096 x 6144 of 43 adapters of 16 ranks 47 (17); 32 rows fp32 8.8.
#include <hip/hip_runtime.h>

#include "lora_delta.h"
#include "lora_gemm.h"

namespace lora {

namespace {

using gemm::barrier;
using gemm::bk_half4;
using gemm::bk_u32x2;
using gemm::kZeros;
using gemm::load_lds;
using gemm::read_columns;
using gemm::wait_all_lds;

constexpr int kMaxFeatures = 1 << 22;
constexpr int kMaxRank = 1 << 16;             // (rank tiles are a grid's z)
constexpr int64_t kMaxGroups = (1 << 24) - 1;  // of 256 threads: a grid holds under 2^32
constexpr int kPlanes = 3;       // bf16 pieces of an fp32 value

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
  char* turned;     // rank space, ranks outside
  float* straight;  // u, rows outside
  float* partial;   // [splits][2 S][slots][padded]
  float* grads;     // [partials][values of a slot]
  int32_t num_tiles, none_tiles, num_parts, num_multi;
  int32_t rows;     // with an adapter
  int64_t slots;    // 64 a tile
  int32_t partials;
  int32_t longest;  // piece, in rows
  int32_t all;      // rows of x, dy, dx
  int32_t max_loras, K, S, O, R;
  int32_t padded, blocks;
  int32_t chunk;
  int32_t accumulate;
  int32_t dx_groups;  // of dx for one tile
  int32_t dx_blocks;  // of dx in the gradients' launch
  int32_t out[LORA_MAX_SLICES], off[LORA_MAX_SLICES];
};

constexpr int es(int dt) { return dt == LORA_BF16 ? 2 : 4; }

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
    if constexpr (RB >= 256) return c ^ (((k >> 3) & 3) << 6);
    if constexpr (RB == 128) return c ^ (((k >> 3) & 1) << 6);
    return c;
  }
  if constexpr (RB >= 256) return c ^ (((k & 3) | ((k >> 3) & 1) << 2) << 5);
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

// a fragment's values, as the matrix instruction takes them
__device__ __forceinline__ void pieces_of(const Frag<LORA_F32>& v, Frag<LORA_BF16> (&f)[kPlanes]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float x[4] = {__uint_as_float(v.v[h][0]), __uint_as_float(v.v[h][1]),
                        __uint_as_float(v.v[h][2]), __uint_as_float(v.v[h][3])};
    bk_u32x2 p[kPlanes];
    pieces_of(x, p);
#pragma unroll
    for (int k = 0; k < kPlanes; ++k) {
      f[k].v[0][2 * h] = p[k][0];
      f[k].v[0][2 * h + 1] = p[k][1];
    }
  }
}
__device__ __forceinline__ void pieces_of(const Frag<LORA_F32>& v, Frag<LORA_F32> (&f)[1]) {
  f[0] = v;
}

typedef const __attribute__((address_space(4))) int32_t* scalar_words;

// Where a value of rank space is kept: `turned` [planes][2 S][padded][slots], ranks
// outside (a gradient's operand, whose reduction is over the rows), and for u also
// `straight` [S][slots][padded] in fp32 (dx's operand, read for every 256 bytes of
// columns and cut into its pieces there: 8704 x 4096 x 4096 142 us in all, and 150 with
// three planes of pieces in memory, which are half as many bytes again).  slots: 64 for
// every tile; those past a tile's rows are zero.
__device__ __forceinline__ int64_t turned_values(const DeltaArgs& a) {
  return (int64_t)2 * a.S * a.padded * a.slots;
}

// Stores four values as they are kept, pieces `apart` values from each other.
template <int DT>
__device__ __forceinline__ void keep(char* base, int64_t at, int64_t apart,
                                     const float (&v)[4]) {
  if constexpr (DT == LORA_F32) {
    *reinterpret_cast<bk_f32x4*>(base + at * 4) = bk_f32x4{v[0], v[1], v[2], v[3]};
  } else {
    bk_u32x2 p[kPlanes];
    pieces_of(v, p);
#pragma unroll
    for (int k = 0; k < kPlanes; ++k)
      *reinterpret_cast<bk_u32x2*>(base + (k * apart + at) * 2) = p[k];
  }
}

// A tile's values of RB ranks, from LDS (64 rows of LD, the sums already in it).  16 lanes
// take the 64 rows of a rank: whole cache lines of `turned`.
template <int DT, int RB>
__device__ __forceinline__ void finish_ranks(const DeltaArgs& a, const float* sums, int q, int tile,
                                             int rank0) {
  constexpr int LD = RB + 4;
  const int tid = threadIdx.x, row = tid % 16 * 4;
  if (a.dA)
#pragma unroll
    for (int i = 0; i < RB / 16; ++i) {
      const int r = 16 * i + tid / 16;
      float v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = sums[(row + j) * LD + r];
      keep<DT>(a.turned, ((int64_t)q * a.padded + rank0 + r) * a.slots + tile * 64 + row,
               turned_values(a), v);
    }
  if (q >= a.S || !a.dx) return;
#pragma unroll
  for (int i = 0; i < RB / 16; ++i) {
    const int o = (i * 256 + tid) * 4, r = rank0 + o % RB;
    // (an infinite dy times the zeros past the last rank is NaN, and so would dx be)
    *reinterpret_cast<bk_f32x4*>(a.straight +
                                 ((int64_t)q * a.slots + tile * 64 + o / RB) * a.padded + r) =
        r < a.R ? *reinterpret_cast<const bk_f32x4*>(sums + o / RB * LD + o % RB)
                : bk_f32x4{0.f, 0.f, 0.f, 0.f};
  }
}

// ------------------------------------------------------------- 1: rank space
//
// One workgroup: 64 rows of one adapter, one rank block, one part of one
// reduction, which its four waves share: wave w takes every fourth 128 bytes of it,
// multiplies all rows with all ranks of the block, and the waves' sums meet in LDS at
// the end.  So nothing waits for another wave on the way: x or dy comes straight to
// registers, two steps ahead, and A or B through the wave's own part of LDS (B is
// read as columns there).  8704 x 4096 x 4096: 53 us, 3.4 TB/s; 2 x 14336 out features:
// 193 us, 3.9 TB/s.  Bound by what a compute unit pulls: the weights' block of each
// 64 rows is as many bytes as the rows.  (Rings that the waves share, three and eight
// steps deep, with their barriers: the same.)
template <int DT, int NT>
constexpr int ranks_lds() {
  const int ring = 4 * 2 * 16 * NT * 128, sums = 4 * 64 * (16 * NT + 4) * 4;
  return ring > sums ? ring : sums;
}
// kOut: u, from dy and B; else v, from x and A.  NR: row tiles that are multiplied.
template <int DT, int NT, bool kOut, int NR>
__device__ __forceinline__ void ranks_tile(const DeltaArgs& a, char* lds, int tile, int slot,
                                           int rows, int first, int s, int rank0, int part) {
  constexpr int ES = es(DT), KS = 128 / ES;   // reduction indexes a step
  constexpr int QS = KS / 32, XV = sizeof(Frag<DT>) / 16;
  constexpr int WB = 16 * NT * ES;            // bytes of a column row of B
  constexpr int WL = 2 * NT, SLOT = WL * 1024;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const int len = kOut ? a.out[s] : a.K;
  const int lo = part * a.chunk, hi = lo + a.chunk < len ? lo + a.chunk : len;
  const int whole_steps = (hi - lo) / KS;           // of the workgroup
  const int nk = (whole_steps - wave + 3) / 4;      // of this wave (it may be 0)
  char* const ring = lds + wave * 2 * SLOT;

  // Rows past the last one read row 0 of the batch: their sums are not kept.
  const char* xp[NR];
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const int r = 16 * i + l16;
    int t = r < rows ? a.perm[first + r] : 0;
    if (t < 0 || t >= a.all) t = 0;
    const int64_t k = lo + wave * KS + 8 * g;
    xp[i] = kOut ? a.dy + ((int64_t)t * a.O + a.off[s] + k) * ES : a.x + ((int64_t)t * a.K + k) * ES;
  }
  // the weights' block of the step, and a lane's place in each 1 KB of it
  const char* wbase =
      kOut ? a.B + (((int64_t)slot * a.O + a.off[s] + lo + wave * KS) * a.R + rank0) * ES
           : a.A + ((((int64_t)slot * a.S + s) * a.R + rank0) * a.K + lo + wave * KS) * ES;
  const int64_t wstep = kOut ? (int64_t)4 * KS * a.R * ES : 512;
  // reduction index and rank of a lane's piece of the j-th KB of a step
  auto place = [&](int ln, int j, int& k, int& r) {
    if constexpr (kOut) {
      const int o = j * 1024 + ln * 16;
      k = o / WB;
      r = column_place<DT, WB>(o % WB, k) / ES;
    } else {
      r = j * 8 + (ln >> 3);
      k = row_place(ln & 7, r) * (16 / ES);
    }
  };
  auto offset = [&](int k, int r) {
    return (uint32_t)(kOut ? k * a.R + r : r * a.K + k) * (uint32_t)ES;
  };
  uint32_t off[kOut ? WL : 1];
#pragma unroll
  for (int j = 0; j < (kOut ? WL : 1); ++j) {
    int k, r;
    place(lane, j, k, r);
    off[j] = offset(k, r);
  }
  struct Rows {
    Frag<DT> f[NR][QS];
  };
  bk_f32x4 acc[NR][NT] = {};
  // Step i of this wave into ring slot i & 1; left: reduction indexes it holds.
  auto load_w = [&](int i, int slot, int left) {
    char* to = ring + slot * SLOT;
    const char* from = wbase + i * wstep;
    const int ranks = a.R - rank0;
    if (left >= KS && ranks >= 16 * NT) {
#pragma unroll
      for (int j = 0; j < WL; ++j)
        load_lds(from, kOut ? off[kOut ? j : 0] : off[0] + (uint32_t)(j * 8 * ES) * (uint32_t)a.K,
                 to + j * 1024);
    } else {
      int ln = lane;
      asm volatile("" : "+v"(ln));  // (so that the places are not kept in registers)
#pragma unroll
      for (int j = 0; j < WL; ++j) {
        int k, r;
        place(ln, j, k, r);
        to_lds(k < left && r < ranks ? from + offset(k, r) : zeros(), to + j * 1024);
      }
    }
  };
  auto multiply = [&](int slot, const Rows& x) {
    const char* at = ring + slot * SLOT;
#pragma unroll
    for (int q = 0; q < QS; ++q) {
      Frag<DT> w[NT];
#pragma unroll
      for (int j = 0; j < NT; ++j)
        w[j] = kOut ? read_cols<DT, WB>(at, 32 * q, 16 * j, 4, l16, g)
                    : read_rows<DT>(at, 16 * j + l16, g, q);
#pragma unroll
      for (int t = 0; t < NR; ++t)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[t][j] = product<DT>(w[j], x.f[t][q], acc[t][j]);
    }
  };
  // Whole steps, two ahead.  Every step makes the same number of loads (past the last
  // one the last again) with no branch around any, so that a count of them waits for
  // the step's own.
  auto load = [&](int i, int slot, Rows& x) {
    const int k = i < nk ? i : nk - 1;
    // the slot's reads are done before its place is filled again
    __builtin_amdgcn_s_waitcnt(wait_all_lds(63));
    asm volatile("" ::: "memory");
    load_w(k, slot, KS);
    asm volatile("" ::: "memory");
#pragma unroll
    for (int t = 0; t < NR; ++t)
#pragma unroll
      for (int q = 0; q < QS; ++q)
#pragma unroll
        for (int h = 0; h < XV; ++h)
          x.f[t][q].v[h] =
              reinterpret_cast<const bk_u32x4*>(xp[t] + (int64_t)k * 512 + q * 32 * ES)[h];
    asm volatile("" ::: "memory");
  };
  constexpr int LOADS = WL + NR * QS * XV;
  if (nk > 0) {
    Rows x[2];
    load(0, 0, x[0]);
    load(1, 1, x[1]);
    auto step = [&](int i, int slot, Rows& now) {
      wait_loads<LOADS>();
      asm volatile("" ::: "memory");
      multiply(slot, now);
      load(i + 2, slot, now);
      return i + 1 < nk;
    };
    for (int i = 0;; i += 2) {
      if (!step(i, 0, x[0])) break;
      if (!step(i + 1, 1, x[1])) break;
    }
    wait_loads<0>();
  }
  // The reduction's end, where it is no whole step: zeros past it.
  const int left = hi - lo - whole_steps * KS;
  if (left > 0 && wave == (whole_steps & 3)) {
    Rows x;
    load_w(nk, 0, left);
#pragma unroll
    for (int t = 0; t < NR; ++t)
#pragma unroll
      for (int q = 0; q < QS; ++q)
#pragma unroll
        for (int h = 0; h < XV; ++h) {
          const char* p = xp[t] + (int64_t)nk * 512 + q * 32 * ES + 16 * h;
          x.f[t][q].v[h] =
              *reinterpret_cast<const bk_u32x4*>(32 * q + 8 * g + 4 * h < left ? p : zeros());
        }
    wait_loads<0>();
    asm volatile("" ::: "memory");
    multiply(0, x);
  }
  // a lane holds ranks 4 g .. 4 g + 3 of every rank tile, of row l16 of every row tile
  constexpr int RB = 16 * NT, LD = RB + 4;
  float* const sums = reinterpret_cast<float*>(lds);
  __syncthreads();
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const bool in = 16 * t + l16 < rows;
#pragma unroll
    for (int j = 0; j < NT; ++j)
      *reinterpret_cast<bk_f32x4*>(sums + (wave * 64 + 16 * t + l16) * LD + 16 * j + 4 * g) =
          in && t < NR ? acc[t < NR ? t : 0][j] : bk_f32x4{0.f, 0.f, 0.f, 0.f};
  }
  __syncthreads();
  const int q = kOut ? s : a.S + s;
  const bool whole = a.chunk >= len;
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int o = (i * 256 + (int)threadIdx.x) * 4, row = o / RB, r = o % RB;
    bk_f32x4* p = reinterpret_cast<bk_f32x4*>(sums + row * LD + r);
    bk_f32x4 v = *p;
#pragma unroll
    for (int w = 1; w < 4; ++w) v += *reinterpret_cast<bk_f32x4*>(sums + (w * 64 + row) * LD + r);
    if (whole)
      *p = v;
    else
      *reinterpret_cast<bk_f32x4*>(
          a.partial + (((int64_t)part * 2 * a.S + q) * a.slots + tile * 64 + row) * a.padded +
          rank0 + r) = v;
  }
  if (!whole) return;
  __syncthreads();
  finish_ranks<DT, 16 * NT>(a, sums, q, tile, rank0);
}

__device__ __forceinline__ int parts_of(int len, int chunk) { return (len + chunk - 1) / chunk; }

// A tile's rows, if they and its slot are in range.
__device__ __forceinline__ bool take_tile(const DeltaArgs& a, int tile, int& slot, int& rows,
                                          int& first) {
  const int32_t* rec = a.tiles + 4 * tile;
  slot = rec[0];
  rows = rec[1];
  first = rec[2];
  return slot >= 0 && slot < a.max_loras && rows > 0 && rows <= kDeltaTileRows && first >= 0 &&
         first <= a.rows - rows;
}

template <int DT, int NT>
__global__ __launch_bounds__(256, 2) void ranks_kernel(DeltaArgs a) {
  __shared__ __attribute__((aligned(16))) char lds[ranks_lds<DT, NT>()];
  // All tiles' first job before the second, so that a compute unit gets jobs of every
  // length.  (Neighbouring tiles on one XCD, whose L2 they would share: 55 us against
  // 56 for 8704 x 4096 x 4096, 200 against 194 for gate/up of 8960 rows, 19.8 against 14.4
  // for 256 rows of 43 adapters.)
  int job = blockIdx.x / a.num_tiles, slot, rows, first;
  const int tile = blockIdx.x - job * a.num_tiles;
  if (!take_tile(a, tile, slot, rows, first)) return;
  const int rank0 = job % a.blocks * 16 * NT;
  job /= a.blocks;
  int s = 0;
  for (; s < a.S; ++s) {
    const int n = parts_of(a.out[s], a.chunk);
    if (job < n) break;
    job -= n;
  }
  const bool out = s < a.S;
  if (!out) {
    const int n = parts_of(a.K, a.chunk);
    s = job / n;
    job %= n;
  }
  // (few rows: a quarter of the products; 256 rows of 43 adapters 14.4 us against 15.9)
  if (rows <= 16) {
    if (out)
      ranks_tile<DT, NT, true, 1>(a, lds, tile, slot, rows, first, s, rank0, job);
    else
      ranks_tile<DT, NT, false, 1>(a, lds, tile, slot, rows, first, s, rank0, job);
  } else {
    if (out)
      ranks_tile<DT, NT, true, 4>(a, lds, tile, slot, rows, first, s, rank0, job);
    else
      ranks_tile<DT, NT, false, 4>(a, lds, tile, slot, rows, first, s, rank0, job);
  }
}

// ------------------------------------------------------- 2: parts of the sums
//
// 64 rows by 16 ranks a workgroup.  8 to 9.5 us for 2 parts of 8704 rows (u and v of 64
// ranks: 18 MB in, 9 out), half of it a launch and its latency.
template <int DT>
__global__ __launch_bounds__(256) void join_kernel(DeltaArgs a) {
  constexpr int LD = 16 + 4;
  __shared__ __attribute__((aligned(16))) float sums[64 * LD];
  const int tile = blockIdx.x, q = blockIdx.y, rank0 = blockIdx.z * 16;
  const int n = parts_of(q < a.S ? a.out[q] : a.K, a.chunk);
  if (n == 1) return;
  const int row = threadIdx.x / 4, r = threadIdx.x % 4 * 4;
  const float* from = a.partial + (((int64_t)q * a.slots + tile * 64 + row) * a.padded + rank0 + r);
  bk_f32x4 v = *reinterpret_cast<const bk_f32x4*>(from);
#pragma unroll 4
  for (int p = 1; p < n; ++p) v += *reinterpret_cast<const bk_f32x4*>(from + p * turned_values(a));
  *reinterpret_cast<bk_f32x4*>(sums + row * LD + r) = v;
  __syncthreads();
  finish_ranks<DT, 16>(a, sums, q, tile, rank0);
}

// ------------------------------------------------------------- 3: the input's
//
// 64 rows of one adapter (or none: a copy) by 256 bytes of columns: the ranks' rows of
// A for these columns in LDS, 128 ranks at a time, a wave's 16 rows of u and of dx_in
// straight to registers, u 64 ranks at a time.  The columns are dealt to the output's
// index so that a lane's are neighbours in memory.  Alone 44 us for 8704 x 4096 of 64 ranks (143 MB in
// and out: 3.2 TB/s).
constexpr int kDxLds = 128 * 256;
template <int DT>
__device__ __forceinline__ void dx_tile(const DeltaArgs& a, char* lds, int block) {
  constexpr int ES = es(DT), RB = 256, CB = RB / ES, RANKS = kDxLds / RB;
  constexpr int CT = CB / 16, V = 16 / ES;  // column tiles; columns of a 16-byte piece
  constexpr int TV = V / 4, NV = CT / TV;   // tiles a piece spans; a lane's pieces
  constexpr int P = DT == LORA_BF16 ? kPlanes : 1;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  // (where the groups are a multiple of 8, one XCD takes a column group of all tiles)
  const int tile = block / a.dx_groups, c0 = (block - tile * a.dx_groups) * CB;
  int slot, rows, first;
  const bool none = tile >= a.num_tiles;
  if (none) {
    const int32_t* rec = a.tiles + 4 * tile;
    rows = rec[1];
    first = rec[2];
    if (a.dx_in == a.dx || rows < 1 || rows > kDeltaTileRows || first < a.rows ||
        first > a.all - rows)
      return;
  } else if (!take_tile(a, tile, slot, rows, first)) {
    return;
  }
  const int row = 16 * wave + l16;
  const bool busy = 16 * wave < rows;  // (the wave has a row)
  int t = row < rows ? a.perm[first + row] : -1;
  // a lane's pieces of dx_in: columns c0 + i 4 V + g V ..
  bk_u32x4 base[NV];
  auto fetch = [&]() {
    if (t >= a.all) t = -1;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = c0 + i * 4 * V + g * V;
      base[i] = bk_u32x4{0, 0, 0, 0};
      if (a.dx_in && t >= 0 && c < a.K)
        base[i] = *reinterpret_cast<const bk_u32x4*>(a.dx_in + ((int64_t)t * a.K + c) * ES);
    }
  };
  bk_f32x4 acc[CT] = {};
  const int ranks = none ? 0 : a.S * a.padded;  // of the reduction
  if (none) fetch();
  for (int r0 = 0; r0 < ranks; r0 += RANKS) {
    const int n = ranks - r0 < RANKS ? ranks - r0 : RANKS;
    // rank index i of the reduction is rank i % padded of slice i / padded
    for (int j = wave; j * 4 < ((n + 31) & ~31); j += 4) {
      const int k = j * 4 + g, i = r0 + k, s = i / a.padded, r = i - s * a.padded;
      const int c = c0 + column_place<DT, RB>(l16 * 16, k) / ES;
      const bool in = k < n && r < a.R && c < a.K;
      to_lds(in ? a.A + ((((int64_t)slot * a.S + s) * a.R + r) * a.K + c) * ES : zeros(),
             lds + j * 1024);
    }
    Frag<LORA_F32> u[2];  // of 32 ranks, and of the next 32
    auto load_u = [&](int q) {
      const int i = r0 + 32 * q + 8 * g, s = i / a.padded, r = i - s * a.padded;
      const bk_u32x4* from = reinterpret_cast<const bk_u32x4*>(
          a.straight + ((int64_t)s * a.slots + tile * 64 + row) * a.padded + r);
#pragma unroll
      for (int h = 0; h < 2; ++h) u[q & 1].v[h] = i < r0 + n ? from[h] : bk_u32x4{0, 0, 0, 0};
    };
    if (busy) {
      load_u(0);
      load_u(1);
    }
    if (r0 == 0) fetch();
    wait_loads<0>();
    barrier();
#pragma unroll
    for (int q = 0; q < RANKS / 32; ++q) {
      if (32 * q >= n || !busy) break;
      Frag<DT> f[P];
      pieces_of(u[q & 1], f);
#pragma unroll
      for (int i = 0; i < CT; ++i) {
        const Frag<DT> w =
            read_cols<DT, RB>(lds, 32 * q, i / TV * 4 * V + i % TV * 4, V, l16, g);
#pragma unroll
        for (int p = P - 1; p >= 0; --p) acc[i] = product<DT>(w, f[p], acc[i]);
      }
      if (q + 2 < RANKS / 32 && 32 * (q + 2) < n) load_u(q + 2);
    }
    wait_loads<0>();
    barrier();
  }
  if (t < 0) return;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = c0 + i * 4 * V + g * V;
    if (c >= a.K) continue;
    bk_u32x4 v;
    if constexpr (DT == LORA_BF16) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bk_f32x4& z = acc[2 * i + j / 2];
        v[j] = bk_pack(z[2 * (j & 1)] + bk_lo(base[i][j]), z[2 * (j & 1) + 1] + bk_hi(base[i][j]));
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        v[j] = __float_as_uint(acc[i][j] + __uint_as_float(base[i][j]));
    }
    *reinterpret_cast<bk_u32x4*>(a.dx + ((int64_t)t * a.K + c) * ES) = v;
  }
}

// ------------------------------------------------------ 4: the adapters' own
//
// One workgroup: a piece of an adapter's rows, 512 bytes of columns of x or dy,
// one rank block.  x or dy goes through a ring of stages of 32 rows in LDS, from which
// both reads are of columns (a row of memory is a reduction index); a wave's 16
// ranks of u or v come straight to registers, with the stages.  Half of the columns a
// workgroup take twice as long (8704 x 4096 x 4096: 97 us alone against 50): u and v are
// read once for each.  dx and gradients there together: 79 us, 5.1 TB/s; 2 x 14336 out
// features 250 to 262 us, 4.3 to 4.5 TB/s.
template <int DT, int NT, int NST, bool kOut>  // kOut: dB, from dy and v; else dA, from x and u
__device__ __forceinline__ void grads_tile(const DeltaArgs& a, char* lds, int slot, int rows,
                                           int first, int tile, int partial, int s, int rank0,
                                           int c0) {
  constexpr int ES = es(DT), P = DT == LORA_BF16 ? kPlanes : 1, XV = sizeof(Frag<DT>) / 16;
  constexpr int RB = kDeltaColumnBytes, STAGE = 32 * RB;
  constexpr int RL = 1024 / RB, LOADS = 8 / RL;  // rows of a load, a wave's loads of a stage
  constexpr int CT = RB / ES / 16 / (4 / NT);  // a wave's column tiles
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const int len = kOut ? a.out[s] : a.K;
  const int col = wave / NT * CT * 16, rank = rank0 + wave % NT * 16;
  const int nk = (rows + 31) / 32;

  const char* base = kOut ? a.dy : a.x;
  const int64_t stride = (int64_t)(kOut ? a.O : a.K) * ES;
  const int lr = lane / (RB / 16);  // a lane's row of a load
  int xc[LOADS];  // column in memory of a lane's piece, or -1
#pragma unroll
  for (int j = 0; j < LOADS; ++j) {
    const int k = 8 * wave + RL * j + lr;
    const int c = column_place<DT, RB>(lane % (RB / 16) * 16, k) / ES;
    xc[j] = c0 + c < len ? (kOut ? a.off[s] : 0) + c0 + c : -1;
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
  auto load = [&](int kt, int slot, const Tokens& tok) {
    char* to = lds + slot * STAGE + wave * 8 * RB;
#pragma unroll
    for (int j = 0; j < LOADS; ++j) {
      int t = tok.t[RL * j];
#pragma unroll
      for (int r = 1; r < RL; ++r) t = lr == r ? tok.t[RL * j + r] : t;
      const bool in = kt * 32 + 8 * wave + RL * j + lr < rows && t >= 0 && t < a.all && xc[j] >= 0;
      to_lds(in ? base + t * stride + (int64_t)xc[j] * ES : zeros(), to + j * 1024);
    }
  };
  // (rank, row 8 g) of the piece's first step; a piece begins with a tile
  const char* const up =
      a.turned + (((int64_t)(kOut ? a.S + s : s) * a.padded + rank + l16) * a.slots + tile * 64 +
                  8 * g) * ES;
  const int64_t apart = turned_values(a) * ES;
  struct Ranks {
    Frag<DT> f[P];
  };
  auto load_u = [&](int kt, Ranks& u) {
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int h = 0; h < XV; ++h) {
        const char* from = up + p * apart + (int64_t)kt * 32 * ES + 16 * h;
        u.f[p].v[h] = *reinterpret_cast<const bk_u32x4*>(kt < nk ? from : zeros());
      }
  };
  bk_f32x4 acc[CT] = {};
  Ranks u[NST];
#pragma unroll
  for (int i = 0; i < NST - 1; ++i) load_u(i, u[i]);
  asm volatile("" ::: "memory");
  Tokens tok = fetch(0);
#pragma unroll
  for (int i = 0; i < NST - 1; ++i) {
    const Tokens next = fetch(i + 1);
    load(i, i, tok);
    tok = next;
  }
  // step kt, whose stage is in `slot` (a constant: the loop below is over the ring)
  auto step = [&](int kt, int slot) {
    const int last = (slot + NST - 1) % NST;
    wait_loads<(NST - 2) * LOADS>();
    barrier();
    load_u(kt + NST - 1, u[last]);
    const Tokens next = fetch(kt + NST);
    load(kt + NST - 1, last, tok);
    tok = next;
    const char* at = lds + slot * STAGE;
#pragma unroll
    for (int i = 0; i < CT; ++i) {
      const Frag<DT> x = read_cols<DT, RB>(at, 0, col + 16 * i, 4, l16, g);
#pragma unroll
      for (int p = P - 1; p >= 0; --p)  // the smallest first
        acc[i] = kOut ? product<DT>(u[slot].f[p], x, acc[i]) : product<DT>(x, u[slot].f[p], acc[i]);
    }
    return kt + 1 < nk;
  };
  wait_loads<(NST - 1) * LOADS>();
  for (int kt = 0;; kt += NST) {
    if (!step(kt, 0)) break;
    if (!step(kt + 1, 1)) break;
    if constexpr (NST > 2)
      if (!step(kt + 2, 2)) break;
  }
  wait_loads<0>();

  const int64_t values = (int64_t)a.R * ((int64_t)a.S * a.K + a.O);
  const bool add = partial < 0 && a.accumulate;
  auto put = [&](float* to, const bk_f32x4& v) {
    bk_f32x4* p = reinterpret_cast<bk_f32x4*>(to);
    *p = add ? *p + v : v;
  };
  if constexpr (!kOut) {
    // a lane holds columns 4 g .. 4 g + 3 of every column tile, of rank l16
    float* to = partial < 0 ? a.dA + (int64_t)slot * a.S * a.R * a.K : a.grads + partial * values;
    const int r = rank + l16;
    if (r >= a.R) return;
    to += ((int64_t)s * a.R + r) * a.K;
#pragma unroll
    for (int i = 0; i < CT; ++i) {
      const int c = c0 + col + 16 * i + 4 * g;
      if (c < a.K) put(to + c, acc[i]);
    }
  } else {
    // ranks 4 g .. 4 g + 3 of column l16 of every column tile
    float* to = partial < 0 ? a.dB + (int64_t)slot * a.O * a.R
                            : a.grads + partial * values + (int64_t)a.S * a.R * a.K;
    const int r = rank + 4 * g;
    if (r >= a.R) return;
#pragma unroll
    for (int i = 0; i < CT; ++i) {
      const int c = c0 + col + 16 * i + l16;
      if (c < len) put(to + (int64_t)(a.off[s] + c) * a.R + r, acc[i]);
    }
  }
}

template <int DT>
__global__ __launch_bounds__(256, 4) void dx_kernel(DeltaArgs a) {
  __shared__ __attribute__((aligned(16))) char lds[kDxLds];
  dx_tile<DT>(a, lds, blockIdx.x);
}

// NST: stages of the ring.  Three, 48 KB, let three workgroups share a compute unit
// (four and five stages: slower); pieces of at most two steps take no third (256 rows of
// 64 adapters 50 us, with the third 56).
template <int DT, int NT, int NST>
__global__ __launch_bounds__(256, 2) void grads_kernel(DeltaArgs a) {
  constexpr int LDS = NST * 32 * kDeltaColumnBytes;
  __shared__ __attribute__((aligned(16))) char lds[LDS > kDxLds ? LDS : kDxLds];
  constexpr int CB = kDeltaColumnBytes / es(DT);
  const int nb = gridDim.x - a.dx_blocks;
  if ((int)blockIdx.x >= nb) {
    dx_tile<DT>(a, lds, blockIdx.x - nb);
    return;
  }
  const int jobs = nb / a.num_parts, part = blockIdx.x / jobs;
  int job = blockIdx.x - part * jobs, slot, n, first;
  const int32_t* rec = a.parts + 4 * part;  // (the longest first)
  const int rows = rec[1], tile = rec[2], partial = rec[3];
  if (tile < 0 || tile >= a.num_tiles || !take_tile(a, tile, slot, n, first) || slot != rec[0] ||
      rows < 1 || rows > a.longest || first > a.rows - rows || (rows + 63) / 64 > a.num_tiles - tile ||
      partial < -1 || partial >= a.partials)
    return;
  const int rank0 = job % a.blocks * 16 * NT;
  job /= a.blocks;
  int s = 0;
  for (; s < a.S; ++s) {
    n = parts_of(a.out[s], CB);
    if (job < n) break;
    job -= n;
  }
  if (s < a.S)
    return grads_tile<DT, NT, NST, true>(a, lds, slot, rows, first, tile, partial, s, rank0, job * CB);
  n = parts_of(a.K, CB);
  grads_tile<DT, NT, NST, false>(a, lds, slot, rows, first, tile, partial, job / n, rank0, job % n * CB);
}

// ----------------------------------------------------- 5: cut adapters' sums
// 1024 values a workgroup.  5 us where two adapters of 8704 x 4096 x 4096 are cut (12 MB).
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
int32_t run(DeltaArgs& a, hipStream_t st) {
  // Jobs of the out slices, and behind them those of x, whose v (as u ranks outside) is for
  // dA and dB: a call for dx alone leaves them out (8704 x 4096 x 4096 105 -> 81 us, gate/up
  // of 8960 rows 260 -> 224, 256 rows of 43 adapters 27 -> 23).
  auto count = [&](int32_t width) {
    int64_t n = a.dA ? (int64_t)a.S * ((a.K + width - 1) / width) : 0;
    for (int s = 0; s < a.S; ++s) n += (a.out[s] + width - 1) / width;
    return n * a.blocks;
  };
  const int64_t jobs = count(a.chunk);
  const int64_t blocks = a.num_tiles * jobs;
  const int64_t grads =
      a.dA && a.rows ? a.num_parts * count(kDeltaColumnBytes / es(DT)) : 0;
  const int64_t dx = a.dx ? (int64_t)(a.num_tiles + a.none_tiles) * a.dx_groups : 0;
  const int64_t values = (int64_t)a.R * ((int64_t)a.S * a.K + a.O);
  if (blocks > kMaxGroups || grads + dx > kMaxGroups || values / 1024 >= kMaxGroups)
    return fail(LORA_E_SHAPE, "too many workgroups");
  if (a.rows) {
    hipLaunchKernelGGL((ranks_kernel<DT, NT>), dim3((uint32_t)blocks), dim3(256), 0, st, a);
    bool cut = a.dA && a.K > a.chunk;
    for (int s = 0; s < a.S; ++s) cut |= a.out[s] > a.chunk;
    if (cut)
      hipLaunchKernelGGL(join_kernel<DT>, dim3(a.num_tiles, a.dA ? 2 * a.S : a.S, a.padded / 16),
                         dim3(256), 0, st, a);
  }
  const bool one = grads && dx;
  a.dx_blocks = one ? (int32_t)dx : 0;
  if (dx && !one)
    hipLaunchKernelGGL(dx_kernel<DT>, dim3((uint32_t)dx), dim3(256), 0, st, a);
  if (grads) {
    const dim3 grid((uint32_t)(grads + a.dx_blocks));
    if (a.longest <= 64)
      hipLaunchKernelGGL((grads_kernel<DT, NT, 2>), grid, dim3(256), 0, st, a);
    else
      hipLaunchKernelGGL((grads_kernel<DT, NT, 3>), grid, dim3(256), 0, st, a);
  }
  if (a.dA && a.num_multi) {
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
  // (offsets inside 64 ranks' rows of A have 32 bits)
  if (g.K > kMaxFeatures || g.R > kMaxRank)
    return fail(LORA_E_SHAPE, "in_features and max_lora_rank must be at most %d and %d",
                kMaxFeatures, kMaxRank);
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
  // Later launches read x, dy and the pools again, so that nothing may be written over them.
  const int64_t e = elem_bytes(g.dtype), of_a = (int64_t)g.max_loras * g.S * g.R * g.K,
                of_b = (int64_t)g.max_loras * g.O * g.R;
  const int64_t sizes[] = {of_a * e,      of_b * e,      T * (int64_t)g.K * e, T * (int64_t)g.O * e,
                           T * (int64_t)g.K * e, T * (int64_t)g.K * e, of_a * 4, of_b * 4,
                           plan->image_bytes,    l.total};
  constexpr int kDxIn = 4, kDx = 5, kDA = 6, kDB = 7, kWs = 9;
  for (int i : {kDx, kDA, kDB, kWs})
    for (int j = 0; j <= kWs; ++j) {
      if (i == j || !ptrs[i] || !ptrs[j] || (i == kDx && j == kDxIn && dx == dx_in)) continue;
      const uintptr_t p = (uintptr_t)ptrs[i], q = (uintptr_t)ptrs[j];
      if (p < q + (uint64_t)sizes[j] && q < p + (uint64_t)sizes[i])
        return fail(LORA_E_ARG, "an output or the workspace overlaps another buffer");
    }

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
  a.turned = (char*)ws + l.turned;
  a.straight = (float*)((char*)ws + l.straight);
  a.partial = (float*)((char*)ws + l.partial);
  a.grads = (float*)((char*)ws + l.grads);
  a.num_tiles = plan->tiles;
  a.none_tiles = plan->none_tiles;
  a.num_parts = plan->parts;
  a.num_multi = plan->multi;
  a.rows = plan->rows;
  a.slots = (int64_t)plan->tiles * kDeltaTileRows;
  a.partials = plan->partials;
  a.longest = plan->longest;
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
  const int32_t cb = 256 / (int32_t)elem_bytes(g.dtype);
  a.dx_groups = (g.K + cb - 1) / cb;
  const hipStream_t st = (hipStream_t)stream;
  if (g.dtype == LORA_BF16)
    return r.tiles == 1   ? run<LORA_BF16, 1>(a, st)
           : r.tiles == 2 ? run<LORA_BF16, 2>(a, st)
                          : run<LORA_BF16, 4>(a, st);
  return r.tiles == 1   ? run<LORA_F32, 1>(a, st)
         : r.tiles == 2 ? run<LORA_F32, 2>(a, st)
                        : run<LORA_F32, 4>(a, st);
}
