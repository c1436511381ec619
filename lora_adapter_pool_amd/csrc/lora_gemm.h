// The matrix product of the decoder-block operators, for one operand type.
//
//   z[m][n] = sum_k A[m][k] B[n][k],  both row-major, reduction contiguous
//
// Everything but the matrix instruction itself is written in bytes: a tile
// step takes 128 bytes of every row (64 bf16, 128 e4m3 or 32 fp32 values), a
// lane reads 16-byte chunks, and lane group g = lane / 16 takes chunks g and
// 4 + g of its row.  Which reduction index a chunk holds does not matter as
// long as both operands agree, so one layout serves all three types:
//   bf16  two v_mfma_f32_16x16x32 a pair of chunks
//   e4m3  one v_mfma_f32_16x16x128_f8f6f4 (unit block scales), or, where the
//         sums have to be exact to fp32, conversion to bf16 (exact) and four
//         bf16 instructions: the 8-bit instructions of gfx950 add neighbouring
//         products on a grid of 2^-11 of the larger one before the fp32 sum
//         (measured: two terms alone are off by up to 2^-10.8 of the larger,
//         terms in different lanes by 2^-23.7), less than bf16 outputs keep
//         and more than fp32 outputs do
//   fp32  eight v_mfma_f32_16x16x4, one a word
// B is the instruction's first operand, so a lane ends with four consecutive
// columns n of one row m.
//
// LDS rows are 128 bytes and chunk c of row r sits at position c ^ (r / 2 % 8):
// 16 lanes that read one chunk of 16 consecutive rows then cover all 64 banks.
// Direct global -> LDS loads write 1 KB runs (8 rows) in lane order, so the
// permutation is made by the lane's choice of its global chunk.
//
// Rows past the end are clamped to the last row (their results are never
// stored).  What a step has past the end of the reduction is loaded from 16
// bytes of zeros instead: no masks, and nothing of the next row can come in.
//
// The gradients sum over what their operands store as rows, so an operand may
// also be reduction-major (bf16 and fp32): A[k][m], m contiguous.  A step of
// it is the same number of bytes, 128 / size rows of k; it lies in LDS as it
// does in memory, and the read turns it into the fragments above:
//   bf16  ds_read_b64_tr_b16: 16 lanes read four rows of 16 values and lane i
//         gets column i.  Two a chunk; 32 bytes a row, so the 32-byte units of
//         a row are permuted by k until the eight rows that 32 lanes read
//         cover all 64 banks.
//   fp32  one value is one matrix instruction's word, so a lane reads NT
//         consecutive columns of one row k and has that word for NT tiles: its
//         tile i holds column NT l16 + i, and the epilogue puts it back.
// Transposed copies instead cost 420 us of the 1820 us of the gradients of
// 4096 rows (4096 x 14336 bf16).
#pragma once

#include "lora_block.h"

namespace lora {
namespace gemm {

constexpr int kE4m3Exact = 3;  // a fourth operand type: e4m3 with fp32 sums

// eight e4m3 values (two words) as bf16
__device__ __forceinline__ bk_bf16x8 widen(uint32_t lo, uint32_t hi) {
  const bk_bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)lo, 1.f, false);
  const bk_bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)lo, 1.f, true);
  const bk_bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)hi, 1.f, false);
  const bk_bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)hi, 1.f, true);
  return bk_bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

template <int DT>
__device__ __forceinline__ bk_f32x4 mma(const bk_u32x4 (&a)[2], const bk_u32x4 (&b)[2],
                                        bk_f32x4 c) {
  if constexpr (DT == LORA_BF16) {
    c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bk_bf16x8, a[0]),
                                                __builtin_bit_cast(bk_bf16x8, b[0]), c, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(
        __builtin_bit_cast(bk_bf16x8, a[1]), __builtin_bit_cast(bk_bf16x8, b[1]), c, 0, 0, 0);
  } else if constexpr (DT == LORA_E4M3) {
    const bk_i32x8 x = {(int)a[0][0], (int)a[0][1], (int)a[0][2], (int)a[0][3],
                        (int)a[1][0], (int)a[1][1], (int)a[1][2], (int)a[1][3]};
    const bk_i32x8 y = {(int)b[0][0], (int)b[0][1], (int)b[0][2], (int)b[0][3],
                        (int)b[1][0], (int)b[1][1], (int)b[1][2], (int)b[1][3]};
    // block scales are powers of two with a bias of 127: 0x7f is 1
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, c, 0, 0, 0, 0x7f7f7f7f, 0,
                                                            0x7f7f7f7f);
  } else if constexpr (DT == kE4m3Exact) {
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int h = 0; h < 4; h += 2)
        c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen(a[s][h], a[s][h + 1]),
                                                    widen(b[s][h], b[s][h + 1]), c, 0, 0, 0);
    return c;
  } else {
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a[s][j]),
                                                 __uint_as_float(b[s][j]), c, 0, 0, 0);
    return c;
  }
}

// s_waitcnt operand (gfx9 encoding): at most n vector memory operations
// outstanding, LDS operations not waited for
__host__ __device__ constexpr int wait_vm(int n) {
  return (n & 15) | ((n >> 4) << 14) | 0x0F70;
}

// the same with every LDS operation waited for
__host__ __device__ constexpr int wait_all_lds(int n) { return wait_vm(n) & ~0x0F00; }

__device__ __forceinline__ void barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Workgroup -> tile and K part.  The whole tiles come first (their number is a
// multiple of 8 unless all are whole), then the parts of the others.
__device__ __forceinline__ void tile_of(const GemmArgs& p, int b, int& tm, int& tn, int& tile,
                                        int& sp) {
  const int rest = p.tiles_m * p.tiles_n - p.whole;
  sp = 0;
  if (b < p.whole) {
    tile = xcd_item(b, p.whole);
  } else {
    const int id = xcd_item(b - p.whole, rest * p.splits);
    sp = id / rest;
    tile = p.whole + id - sp * rest;
  }
  tile_place(p, tile, tm, tn);
}

template <int V>
struct Int {
  static constexpr int value = V;
};

constexpr int type_size(int dt) { return dt == LORA_F32 ? 4 : dt == LORA_BF16 ? 2 : 1; }

// Loaded in place of what lies past the end of the reduction.
static __device__ const uint32_t kZeros[4] __attribute__((aligned(16))) = {0, 0, 0, 0};

// 16 bytes a lane from `base` (uniform) + `off`: one instruction and no vector
// arithmetic, which the loops below do not hide (a 128 x 128 bf16 tile: 0.72 us
// a step against 0.78 with addresses of 64 bits and a comparison a load).
// kOnce: non-temporal.
template <bool kOnce = false>
__device__ __forceinline__ void load_lds(const char* base, uint32_t off, char* to) {
  asm("" : "+s"(base), "+v"(off));  // (no 64-bit sums by lane are kept instead)
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(base + off),
                                   (__attribute__((address_space(3))) void*)to, 16, 0,
                                   kOnce ? 2 : 0);
}
// the same where the reduction may end in the step.  The large kernel's waves
// multiply in pairs, one while the other loads, which hides the sums; there it
// is the faster form (8192^3 e4m3 428 us against 463).
__device__ __forceinline__ void load_lds_end(const char* base, uint32_t off, bool past, char* to) {
  const char* from = past ? reinterpret_cast<const char*>(kZeros) : base + off;
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)from,
                                   (__attribute__((address_space(3))) void*)to, 16, 0, 0);
}

// Four rows of 16 values, read as columns.  The argument is `restrict` so that
// the read is known apart from the direct loads into LDS: without it the
// compiler waits for all of these before each such read, which the waits and
// barriers of the kernels below order already (gradients of 4096 x 4096 x 14336
// 1538 -> 1496 us, of 300 x 2048 x 2048 54 -> 48 us).
typedef short bk_half4 __attribute__((ext_vector_type(4)));
typedef uint32_t bk_u32x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ bk_u32x2 read_columns(
    __attribute__((address_space(3))) bk_half4* __restrict p) {
  return __builtin_bit_cast(bk_u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(p));
}

// A reduction-major tile of ROWS columns m: rows of RB bytes, one a k.
template <int DT, int ROWS>
struct ColTile {
  static constexpr int ES = type_size(DT), RB = ROWS * ES;
  static_assert(DT == LORA_F32 ? RB >= 128 : RB == 32 || RB == 64 || RB == 128 || RB == 256, "");
  // position of column byte `c` of row k (its own inverse)
  static __device__ __forceinline__ int swizzle(int c, int k) {
    if constexpr (DT == LORA_F32) return c ^ (((k >> 2) & 1) << (RB == 128 ? 6 : 7));
    // four rows of 64 bytes, two of 128 or one of 256 cover the banks once
    if constexpr (RB == 64) return c ^ (((k >> 3) & 1) << 5);
    if constexpr (RB == 128) return c ^ ((((k >> 1) & 1) | ((k >> 3) & 1) << 1) << 5);
    return c ^ (((k & 3) | ((k >> 3) & 1) << 2) << 5);
  }
  // the fragments of NT tiles from column `col` on (a multiple of 16 NT)
  template <int NT>
  static __device__ __forceinline__ void read(const char* tile, int col, int l16, int g,
                                              bk_u32x4 (&f)[NT][2]) {
    if constexpr (DT == LORA_F32) {
      typedef uint32_t vec __attribute__((ext_vector_type(NT)));
      const int at = swizzle(ES * (col + NT * l16), 4 * g);
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const vec v = *reinterpret_cast<const vec*>(tile + (16 * s + 4 * g + w) * RB + at);
#pragma unroll
          for (int i = 0; i < NT; ++i) f[i][s][w] = v[i];
        }
    } else {
      const int k = 8 * g + (l16 >> 2);
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const char* at = tile + k * RB + swizzle(ES * (col + 16 * i + 4 * (l16 & 3)), k);
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const bk_u32x2 v = read_columns(
                (__attribute__((address_space(3))) bk_half4*)(at + (32 * s + 4 * h) * RB));
            f[i][s][2 * h] = v[0];
            f[i][s][2 * h + 1] = v[1];
          }
      }
    }
  }
};

// Column (of NT tiles) that index r of tile i is, as the reads above deal them.
template <int DT, bool kCol, int NT>
__device__ __forceinline__ int tile_index(int i, int r) {
  return kCol && DT == LORA_F32 ? NT * r + i : 16 * i + r;
}

// A wave's products of one row of tiles into its part of LDS.
template <int DT, bool kBCol, int NT>
__device__ __forceinline__ void put_row(float* row, int g, const bk_f32x4 (&acc)[NT]) {
#pragma unroll
  for (int j = 0; j < NT; ++j)
    if constexpr (kBCol && DT == LORA_F32) {
#pragma unroll
      for (int r = 0; r < 4; ++r) row[tile_index<DT, kBCol, NT>(j, 4 * g + r)] = acc[j][r];
    } else {
      *reinterpret_cast<bk_f32x4*>(row + j * 16 + 4 * g) = acc[j];
    }
}

// The rows of a wave's products, from its part of LDS (row-major, LDE floats a
// row) to the partials or through the epilogue.  ROWS rows from m on, COLS
// output columns from n on (gated: the up products lie COLS to the right);
// row and col are the wave's place in the tile of BM x BN.
template <bool kGated, int BM, int BN, int ROWS, int COLS, int LDE>
__device__ __forceinline__ void finish_rows(const GemmArgs& p, const float* reg, int lane, int m,
                                            int n, int tile, int sp, int row, int col) {
  constexpr int LPR = COLS / 8;   // lanes a row
  constexpr int RPI = 64 / LPR;   // rows an iteration
  constexpr int NI = ROWS / RPI > 0 ? ROWS / RPI : 1;
  constexpr int GRP = NI < 4 ? NI : 4;
  const int r0 = lane / LPR, c = lane % LPR * 8;
  n += c;
  auto get = [&](int r, float (&z)[8], float (&u)[8]) {
    const float* from = reg + r * LDE + c;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const bk_f32x4 v = *reinterpret_cast<const bk_f32x4*>(from + 4 * h);
#pragma unroll
      for (int j = 0; j < 4; ++j) z[4 * h + j] = v[j];
      if constexpr (kGated) {
        const bk_f32x4 w = *reinterpret_cast<const bk_f32x4*>(from + COLS + 4 * h);
#pragma unroll
        for (int j = 0; j < 4; ++j) u[4 * h + j] = w[j];
      }
    }
  };
  if (tile >= p.whole) {
    float* to = p.part + (int64_t)((tile - p.whole) * p.splits + sp) * (BM * BN);
    for (int r = r0; r < ROWS; r += RPI) {
      if (m + r >= p.M || n >= p.N) continue;
      float z[8], u[8];
      get(r, z, u);
      float* d = to + (row + r) * BN + col + c;
      *reinterpret_cast<bk_f32x4*>(d) = bk_f32x4{z[0], z[1], z[2], z[3]};
      *reinterpret_cast<bk_f32x4*>(d + 4) = bk_f32x4{z[4], z[5], z[6], z[7]};
      if constexpr (kGated) {
        d += BN / 2;
        *reinterpret_cast<bk_f32x4*>(d) = bk_f32x4{u[0], u[1], u[2], u[3]};
        *reinterpret_cast<bk_f32x4*>(d + 4) = bk_f32x4{u[4], u[5], u[6], u[7]};
      }
    }
  } else if (p.out_dtype == LORA_BF16) {
    for (int i0 = 0; i0 < NI; i0 += GRP) {
      Extra<kGated> x[GRP];
#pragma unroll
      for (int i = 0; i < GRP; ++i) fetch_extra<kGated>(p, m + r0 + (i0 + i) * RPI, n, x[i]);
#pragma unroll
      for (int i = 0; i < GRP; ++i) {
        const int r = r0 + (i0 + i) * RPI;
        if (r >= ROWS || m + r >= p.M || n >= p.N) continue;
        float z[8], u[8];
        get(r, z, u);
        epilogue8<kGated, true>(p, m + r, n, z, u, x[i]);
      }
    }
  } else {
    for (int r = r0; r < ROWS; r += RPI) {
      if (m + r >= p.M || n >= p.N) continue;
      float z[8], u[8];
      get(r, z, u);
      epilogue8<kGated, false>(p, m + r, n, z, u, Extra<kGated>{});
    }
  }
}

// A tile of BM x BN, waves of WM x WN, a ring of NST stages filled by direct
// global -> LDS loads.  One barrier a step: after it stage kt has landed for
// every wave and stage kt - 1 has been read by every wave, so its place takes
// the loads of step kt + NST - 1.  The epilogue goes through LDS (a wave's own
// region) so that it is a rolled loop over whole row pieces.
//
// kOnce: one row of tiles covers A, so that B is read once: the weights of a
// decode step, which are gone from the caches before the next step wants them.
// Its loads are non-temporal (1 x 14336 x 4096 bf16 26.7 -> 24.6 us, gated 1 x
// 4096 x 14336 47.1 -> 42.8 us).
//
// kLines: rows that do not start at a cache line.  Loads of 128 bytes from a
// row's start would touch every line twice, a step apart.  Stage L holds whole
// lines instead, from 16 sh bytes before the row's chunk 8 L on, where sh =
// (address / 16) mod 8 repeats every eight rows, and step kt reads its chunks
// from stages kt and kt + 1.  The swizzle stays free of conflicts: (x + 2 n q)
// mod 8, then xor q, is a permutation of 0 .. 7 in q for every x and n.  This
// pays where the loads come from memory (gated bf16 44 x 9112 x 9408 93 -> 82
// us, 64 x 4104 x 4096 16.4 -> 14.5 us) and costs a short product time (gated
// 777 x 1032 x 520 9.6 -> 11.3 us): the plan decides by the operands' size.
template <int BM, int BN, int WM, int WN, int NST>
constexpr int ring_bytes() {
  constexpr int stages = (BM + BN) * kStepBytes * NST;
  constexpr int epilogue = BM / WM * (BN / WN) * WM * (WN + 4) * 4;
  return stages > epilogue ? stages : epilogue;
}
template <int DT, Form kForm, int BM, int BN, int WM, int WN, int NST, bool kOnce, bool kLines>
__device__ __forceinline__ void ring_tile(const GemmArgs& p, int block, char* lds) {
  constexpr bool kGated = kForm == kGatedForm, kACol = kForm == kGradW;
  constexpr bool kBCol = kForm == kGradX || kForm == kGradW;
  constexpr int ES = type_size(DT);
  using TileA = ColTile<DT, BM>;
  using TileB = ColTile<DT, BN>;
  constexpr int NWN = BN / WN, NW = BM / WM * NWN;
  constexpr int STAGE = (BM + BN) * kStepBytes;
  constexpr int P = (BM + BN) / 8 / NW;  // loads a wave makes for a stage
  static_assert(P * NW * 8 == BM + BN, "rows divide over the waves");
  constexpr int LDE = WN + 4;            // floats a row of the epilogue's region

  int tm, tn, tile, sp;
  tile_of(p, block, tm, tn, tile, sp);
  const int m0 = tm * BM, n0 = tn * (kGated ? BN / 2 : BN);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, g = lane >> 4;

  const int nk_all = (int)((p.kb + kStepBytes - 1) / kStepBytes);
  const int per = tile < p.whole ? nk_all : (nk_all + p.splits - 1) / p.splits;
  const int k_lo = sp * per, nk = (k_lo + per < nk_all ? k_lo + per : nk_all) - k_lo;

  // Loads: the first half of the waves fills A, the other B.  A lane's offset
  // from the tile's first stored row in the step, and how many bytes of the
  // reduction lie before its own in the step.
  static_assert(NW % 2 == 0 && BM == BN, "");
  const bool of_a = wave < NW / 2;
  const int run = of_a ? wave * P : wave * P - BM / 8;  // first 1 KB run of the operand's
  const int64_t ld = of_a ? p.lda : p.ldb;
  const int64_t advance =
      (of_a ? kACol : kBCol) ? (int64_t)(kStepBytes / ES) * ld : (int64_t)kStepBytes;
  const char* base = of_a ? p.A + (kACol ? (int64_t)m0 * ES : m0 * ld)
                          : p.B + (kBCol ? (int64_t)n0 * ES : n0 * ld);
  base += k_lo * advance;
  // (chunk units; the tile's first row and a wave's tiles are multiples of
  // eight rows apart)
  auto shift_of = [&](const char* at, int64_t stride, int row) {
    return kLines ? (int)(((uintptr_t)at >> 4) + row * (stride >> 4)) & 7 : 0;
  };
  const int sh = shift_of(base, ld, lane >> 3);
  const int lines = kLines ? nk + 1 : nk;  // stages to load
  const int64_t up = kGated && !of_a ? p.N * ld : 0;  // from a gate row to its up row
  uint32_t off[P];
  auto before = [&](int j) {
    if constexpr (kACol && kBCol) return ((run + j) * 1024 + lane * 16) / TileA::RB * ES;
    if constexpr (kBCol)
      if (!of_a) return ((run + j) * 1024 + lane * 16) / TileB::RB * ES;
    return 16 * (((lane & 7) ^ ((4 * (run + j) + (lane >> 4)) & 7)) - sh);
  };
  // gated: a wave's WN rows of B are WN / 2 gate rows, then the up rows of the
  // same columns
  auto is_up = [&](int j) { return kGated && !of_a && (run + j) * 8 % WN >= WN / 2; };
#pragma unroll
  for (int j = 0; j < P; ++j) {
    const int o = (run + j) * 1024 + lane * 16;
    if (of_a ? kACol : kBCol) {
      const int rb = of_a ? TileA::RB : TileB::RB, k = o / rb;
      int c = of_a ? TileA::swizzle(o % rb, k) : TileB::swizzle(o % rb, k);
      if ((of_a ? m0 : n0) + c / ES >= (of_a ? p.M : p.N)) c = 0;
      off[j] = (uint32_t)c + (uint32_t)k * (uint32_t)ld;
    } else {
      int r = o / kStepBytes;
      if (kGated && !of_a) r = r / WN * (WN / 2) + r % (WN / 2);
      const int left = of_a ? p.M - m0 : p.N - n0;
      // (kLines: from a line before the row, so that it is not negative)
      off[j] = (uint32_t)(r < left ? r : left - 1) * (uint32_t)ld +
               (uint32_t)(before(j) + (kLines ? kStepBytes : 0));
    }
  }
  auto issue = [&](int kt, int slot) {
    const int64_t left = p.kb - (int64_t)(k_lo + kt) * kStepBytes;
    const char* from = base + kt * advance - (kLines ? kStepBytes : 0);
    char* to = lds + slot * STAGE + wave * P * 1024;
    if (kLines && k_lo + kt == 0) {  // what lies before the row is not read
#pragma unroll
      for (int j = 0; j < P; ++j) {
        const int b = before(j);
        load_lds_end(from + (is_up(j) ? up : 0), off[j] + (b < 0 ? -b : 0), b >= left,
                     to + j * 1024);
      }
    } else if (left >= kStepBytes) {
#pragma unroll
      for (int j = 0; j < P; ++j)
        load_lds<kOnce>(from + (is_up(j) ? up : 0), off[j], to + j * 1024);
    } else {
#pragma unroll
      for (int j = 0; j < P; ++j)
        load_lds_end(from + (is_up(j) ? up : 0), off[j], before(j) >= left, to + j * 1024);
    }
  };

  const int wr = wave / NWN, wc = wave % NWN;
  bk_f32x4 acc[WM / 16][WN / 16];
#pragma unroll
  for (int i = 0; i < WM / 16; ++i)
#pragma unroll
    for (int j = 0; j < WN / 16; ++j) acc[i][j] = bk_f32x4{0.f, 0.f, 0.f, 0.f};

#pragma unroll
  for (int s = 0; s < NST - 1; ++s)
    if (s < lines) issue(s, s);

  // a lane's two chunks: place in a stage's row, and whether in the next stage
  const int sha = shift_of(p.A + m0 * p.lda, p.lda, l16);
  const int shb = shift_of(p.B + n0 * p.ldb, p.ldb, l16);
  auto place = [&](int chunk) { return ((chunk & 7) ^ (l16 >> 1)) * 16; };
  const int a0 = place(g + sha), a1 = place(g + 4 + sha);
  const int b0 = place(g + shb), b1 = place(g + 4 + shb);

  int slot = 0;
  for (int kt = 0; kt < nk; ++kt) {
    // (kLines: stage kt + 1 has landed too)
    if (kt + NST - 1 <= lines)
      __builtin_amdgcn_s_waitcnt(wait_vm((NST - (kLines ? 3 : 2)) * P));
    else
      __builtin_amdgcn_s_waitcnt(wait_vm(0));
    barrier();
    if (kt + NST - 1 < lines) issue(kt + NST - 1, slot == 0 ? NST - 1 : slot - 1);

    const char* stage = lds + slot * STAGE;
    const int next = kLines ? (slot == NST - 1 ? -(NST - 1) * STAGE : STAGE) : 0;
    const int at_a0 = a0 + (g + sha > 7 ? next : 0), at_a1 = a1 + (g + sha > 3 ? next : 0);
    const int at_b0 = b0 + (g + shb > 7 ? next : 0), at_b1 = b1 + (g + shb > 3 ? next : 0);
    bk_u32x4 fa[WM / 16][2], fb[WN / 16][2];
    if constexpr (kACol) {
      TileA::read(stage, wr * WM, l16, g, fa);
    } else {
      const char* sA = stage + (wr * WM + l16) * kStepBytes;
#pragma unroll
      for (int i = 0; i < WM / 16; ++i) {
        fa[i][0] = *reinterpret_cast<const bk_u32x4*>(sA + i * 16 * kStepBytes + at_a0);
        fa[i][1] = *reinterpret_cast<const bk_u32x4*>(sA + i * 16 * kStepBytes + at_a1);
      }
    }
    if constexpr (kBCol) {
      TileB::read(stage + BM * kStepBytes, wc * WN, l16, g, fb);
    } else {
      const char* sB = stage + (BM + wc * WN + l16) * kStepBytes;
#pragma unroll
      for (int j = 0; j < WN / 16; ++j) {
        fb[j][0] = *reinterpret_cast<const bk_u32x4*>(sB + j * 16 * kStepBytes + at_b0);
        fb[j][1] = *reinterpret_cast<const bk_u32x4*>(sB + j * 16 * kStepBytes + at_b1);
      }
    }
#pragma unroll
    for (int i = 0; i < WM / 16; ++i)
#pragma unroll
      for (int j = 0; j < WN / 16; ++j) acc[i][j] = mma<DT>(fb[j], fa[i], acc[i][j]);
    slot = slot == NST - 1 ? 0 : slot + 1;
  }

  // epilogue: the wave's products, row-major, in its own part of LDS
  __builtin_amdgcn_s_waitcnt(0xC07F);  // this wave's LDS reads are done
  barrier();
  float* reg = reinterpret_cast<float*>(lds) + wave * WM * LDE;
#pragma unroll
  for (int i = 0; i < WM / 16; ++i)
    put_row<DT, kBCol>(reg + tile_index<DT, kACol, WM / 16>(i, l16) * LDE, g, acc[i]);
  __builtin_amdgcn_s_waitcnt(0xC07F);
  asm volatile("" ::: "memory");
  __builtin_amdgcn_wave_barrier();

  constexpr int WCOLS = kGated ? WN / 2 : WN;  // output columns of a wave
  finish_rows<kGated, BM, BN, WM, WCOLS, LDE>(p, reg, lane, m0 + wr * WM, n0 + wc * WCOLS, tile,
                                              sp, wr * WM, wc * WCOLS);
}

template <int DT, Form kForm, int BM, int BN, int WM, int WN, int NST, bool kOnce, bool kLines>
__global__ __launch_bounds__(BM / WM * (BN / WN) * 64) void gemm_ring_kernel(GemmArgs p) {
  __shared__ __align__(1024) char lds[ring_bytes<BM, BN, WM, WN, NST>()];
  ring_tile<DT, kForm, BM, BN, WM, WN, NST, kOnce, kLines>(p, blockIdx.x, lds);
}

// Both gradients' products in one launch: they need each other's results for
// nothing, and together they fill compute units that either leaves idle.
// `first` workgroups belong to the product with the longer reduction.
template <int DT, int BM, int BN, int WM, int WN, int NST>
__global__ __launch_bounds__(BM / WM * (BN / WN) * 64) void gemm_pair_kernel(GemmArgs x,
                                                                             GemmArgs w,
                                                                             int first,
                                                                             bool x_first) {
  __shared__ __align__(1024) char lds[ring_bytes<BM, BN, WM, WN, NST>()];
  const int b = blockIdx.x;
  if ((b < first) == x_first)
    ring_tile<DT, kGradX, BM, BN, WM, WN, NST, false, false>(x, b < first ? b : b - first, lds);
  else
    ring_tile<DT, kGradW, BM, BN, WM, WN, NST, false, false>(w, b < first ? b : b - first, lds);
}

// The large product: a 256 x 256 tile, 8 waves of 128 x 64 (two a SIMD), and
// two LDS buffers of one step each, cut into four pieces of 16 KB (A0, A1: the
// two halves of the rows of A; B0, B1: of B) that are read and refilled apart.
//
// A step is two phases, one half of a wave's rows each:
//   phase 0: read A0, B0, B1, multiply A0 B0, A0 B1;  load A1 of the next step
//   phase 1: read A1, multiply A1 B1, A1 B0;  load A0, B0, B1 of the step after
// and a phase is two slots with a barrier after each: one for memory (LDS
// reads into registers, direct loads) and one for the products (32 matrix
// instructions of 16 cycles).  Waves 4 to 7 run one slot behind waves 0 to 3,
// so on every SIMD one wave multiplies while the other reads.  Four phases of
// half this length spent 23% of their time in the barriers between them.
//
// What orders the accesses.  A wave's LDS reads are complete at the end of the
// memory slot that issued them; a piece is refilled in the next phase's memory
// slot at the earliest, two slots later.  Loads of a wave complete in order
// and eight may be outstanding when it leaves a memory slot: those issued
// before have landed, which are the ones that the next phase reads, and do so
// for every wave once all have passed the barriers of that slot and the next.
template <int DT, Form kForm>
__global__ __launch_bounds__(512, 2) void gemm_phase_kernel(GemmArgs p) {
  constexpr bool kGated = kForm == kGatedForm, kACol = kForm == kGradW;
  constexpr bool kBCol = kForm == kGradX || kForm == kGradW;
  constexpr int ES = type_size(DT);
  using Piece = ColTile<DT, 128>;
  constexpr int PIECE = 128 * kStepBytes, BUF = 4 * PIECE;
  constexpr int LDE = 64 + 4;             // floats a row of the epilogue's region
  constexpr int EPI = 8 * 64 * LDE * 4;   // half of every wave's rows at a time
  __shared__ __align__(1024) char lds[EPI > 2 * BUF ? EPI : 2 * BUF];

  int tm, tn, tile, sp;
  tile_of(p, blockIdx.x, tm, tn, tile, sp);
  const int m0 = tm * 256, n0 = tn * (kGated ? 128 : 256);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const int wr = wave >> 2, wc = wave & 3;

  const int nk_all = (int)((p.kb + kStepBytes - 1) / kStepBytes);
  const int per = tile < p.whole ? nk_all : (nk_all + p.splits - 1) / p.splits;
  const int k_lo = sp * per, nk = (k_lo + per < nk_all ? k_lo + per : nk_all) - k_lo;
  const int64_t rest = p.kb - (int64_t)(k_lo + nk - 1) * kStepBytes;
  const int tail = rest < kStepBytes ? (int)rest : kStepBytes;  // bytes of the last step

  // loads: a wave fills 1 KB runs w and w + 8 of every piece, so the chunk of a
  // row that a lane takes is the same in every load of a row-major operand
  const int chunk16 = 16 * ((lane & 7) ^ ((wave & 1) * 4 + (lane >> 4)));
  const int64_t step_a = kACol ? kStepBytes / ES * p.lda : kStepBytes;
  const int64_t step_b = kBCol ? kStepBytes / ES * p.ldb : kStepBytes;
  const char* baseA = p.A + (kACol ? (int64_t)m0 * ES : m0 * p.lda) + k_lo * step_a;
  const char* baseB0 = p.B + (kBCol ? (int64_t)n0 * ES : n0 * p.ldb) + k_lo * step_b;
  const char* baseB1 = kGated ? baseB0 + p.N * p.ldb : baseB0;
  uint32_t offA[2][2], offB[2][2];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int o = 1024 * (wave + 8 * j) + 16 * lane, r = o / kStepBytes, k = o / Piece::RB;
      const int c = Piece::swizzle(o % Piece::RB, k) / ES;  // first of the chunk's columns
      // linear: a wave's 64 columns are consecutive, 32 from each half of B
      int m = h * 128 + (kACol ? c : r), n = kBCol ? c : r;
      if constexpr (!kGated) n = (n >> 5) * 64 + h * 32 + (n & 31);
      if constexpr (kACol)
        offA[h][j] = (uint32_t)((m0 + m < p.M ? m : 0) * ES) + (uint32_t)k * (uint32_t)p.lda;
      else
        offA[h][j] = (uint32_t)(m0 + m < p.M ? m : p.M - 1 - m0) * (uint32_t)p.lda + chunk16;
      if constexpr (kBCol)
        offB[h][j] = (uint32_t)((n0 + n < p.N ? n : 0) * ES) + (uint32_t)k * (uint32_t)p.ldb;
      else
        offB[h][j] = (uint32_t)(n0 + n < p.N ? n : p.N - 1 - n0) * (uint32_t)p.ldb + chunk16;
    }
  auto fill = [&](auto col, const char* base, int64_t step, const uint32_t (&off)[2], int piece,
                  int kt) {
    constexpr bool kCol = decltype(col)::value;
    char* to = lds + (kt & 1) * BUF + piece * PIECE + wave * 1024;
    const char* from = base + kt * step;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int before = kCol ? (1024 * (wave + 8 * j) + 16 * lane) / Piece::RB * ES : chunk16;
      load_lds_end(from, off[j], kt == nk - 1 && before >= tail, to + j * 8192);
    }
  };
  auto fill_a = [&](int h, int kt) {
    fill(Int<kACol>{}, baseA, step_a, offA[h], h, kt);
  };
  auto fill_b = [&](int kt) {
    fill(Int<kBCol>{}, baseB0, step_b, offB[0], 2, kt);
    fill(Int<kBCol>{}, baseB1, step_b, offB[1], 3, kt);
  };

  bk_f32x4 acc[2][2][4][2];
#pragma unroll
  for (int a = 0; a < 2; ++a)
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[a][b][i][j] = bk_f32x4{0.f, 0.f, 0.f, 0.f};
  bk_u32x4 fa[4][2], fb[2][2][2];

  const int c0 = (g ^ (l16 >> 1)) * 16, c1 = c0 ^ 64;
  const char* rdA = lds + (wr * 64 + l16) * kStepBytes;
  const char* rdB = lds + 2 * PIECE + (wc * 32 + l16) * kStepBytes;

  auto read_a = [&](int h, int kt) {
    if constexpr (kACol) {
      Piece::read(lds + (kt & 1) * BUF + h * PIECE, wr * 64, l16, g, fa);
      return;
    }
    const char* s = rdA + (kt & 1) * BUF + h * PIECE;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      fa[i][0] = *reinterpret_cast<const bk_u32x4*>(s + i * 16 * kStepBytes + c0);
      fa[i][1] = *reinterpret_cast<const bk_u32x4*>(s + i * 16 * kStepBytes + c1);
    }
  };
  auto read_b = [&](int h, int kt) {
    if constexpr (kBCol) {
      Piece::read(lds + (kt & 1) * BUF + (2 + h) * PIECE, wc * 32, l16, g, fb[h]);
      return;
    }
    const char* s = rdB + (kt & 1) * BUF + h * PIECE;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      fb[h][j][0] = *reinterpret_cast<const bk_u32x4*>(s + j * 16 * kStepBytes + c0);
      fb[h][j][1] = *reinterpret_cast<const bk_u32x4*>(s + j * 16 * kStepBytes + c1);
    }
  };
  auto products = [&](int ha) {
    if constexpr (DT == kE4m3Exact) {
      // Eight values at a time, A widened anew for each half of B: all of
      // the widened fragments at once do not fit in the registers.
      __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int hb = 0; hb < 2; ++hb)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            bk_bf16x8 wb[2];
#pragma unroll
            for (int j = 0; j < 2; ++j)
              wb[j] = widen(fb[hb][j][s][2 * q], fb[hb][j][s][2 * q + 1]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t lo = fa[i][s][2 * q], hi = fa[i][s][2 * q + 1];
              asm volatile("" : "+v"(lo), "+v"(hi));  // (no reuse of the other half's)
              const bk_bf16x8 wa = widen(lo, hi);
#pragma unroll
              for (int j = 0; j < 2; ++j)
                acc[ha][hb][i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                    wb[j], wa, acc[ha][hb][i][j], 0, 0, 0);
            }
            __builtin_amdgcn_sched_barrier(0);
          }
        }
      __builtin_amdgcn_s_setprio(0);
      return;
    }
    __builtin_amdgcn_s_setprio(1);
    if constexpr (DT == LORA_BF16) {
      // one operand for four instructions, and never the sum of the one before
      // (gradients of 4096 x 4096 x 14336 1484 -> 1470 us)
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int i0 = 0; i0 < 4; ++i0) {
            const int hb = q >> 1, j = q & 1, i = j ? 3 - i0 : i0;
            acc[ha][hb][i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                __builtin_bit_cast(bk_bf16x8, fb[hb][j][c]), __builtin_bit_cast(bk_bf16x8, fa[i][c]),
                acc[ha][hb][i][j], 0, 0, 0);
          }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int hb = 0; hb < 2; ++hb)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            acc[ha][hb][i][j] = mma<DT>(fb[hb][j], fa[i], acc[ha][hb][i][j]);
    }
    __builtin_amdgcn_s_setprio(0);
  };
  auto slot_end = [&]() {
    __builtin_amdgcn_sched_barrier(0);
    barrier();
    __builtin_amdgcn_sched_barrier(0);
  };
  // kLeft: steps after this one (2: two or more, all loads are made)
  auto step = [&](int kt, auto left_tag) {
    constexpr int kLeft = decltype(left_tag)::value;
    read_a(0, kt);
    read_b(0, kt);
    read_b(1, kt);
    if constexpr (kLeft >= 1) fill_a(1, kt + 1);
    __builtin_amdgcn_s_waitcnt(wait_all_lds(kLeft >= 1 ? 8 : 0));
    slot_end();
    products(0);
    slot_end();

    read_a(1, kt);
    if constexpr (kLeft >= 2) {
      fill_a(0, kt + 2);
      fill_b(kt + 2);
    }
    __builtin_amdgcn_s_waitcnt(wait_all_lds(kLeft >= 2 ? 8 : kLeft == 1 ? 2 : 0));
    slot_end();
    products(1);
    slot_end();
  };

  fill_a(0, 0);
  fill_b(0);
  fill_a(1, 0);
  if (nk > 1) {
    fill_a(0, 1);
    fill_b(1);
    __builtin_amdgcn_s_waitcnt(wait_vm(8));
  } else {
    __builtin_amdgcn_s_waitcnt(wait_vm(2));
  }
  slot_end();
  if (wave >= 4) slot_end();  // one slot behind
  int kt = 0;
  for (; kt < nk - 2; ++kt) step(kt, Int<2>{});
  if (nk > 1) step(kt++, Int<1>{});
  step(kt, Int<0>{});
  if (wave < 4) slot_end();

  // epilogue: 64 rows of every wave at a time through its own part of LDS
  float* reg = reinterpret_cast<float*>(lds) + wave * 64 * LDE;
  constexpr int WCOLS = kGated ? 32 : 64;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    barrier();  // (all waves are past their LDS reads; the pass before is read)
#pragma unroll
    for (int hb = 0; hb < 2; ++hb)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        put_row<DT, kBCol>(reg + tile_index<DT, kACol, 4>(i, l16) * LDE + hb * 32, g,
                           acc[h][hb][i]);
    __builtin_amdgcn_s_waitcnt(0xC07F);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_wave_barrier();
    finish_rows<kGated, 256, 256, 64, WCOLS, LDE>(p, reg, lane, m0 + h * 128 + wr * 64,
                                                  n0 + wc * WCOLS, tile, sp, h * 128 + wr * 64,
                                                  wc * WCOLS);
    __builtin_amdgcn_s_waitcnt(0xC07F);
  }
}

// Few rows: 16 MT rows by 16 columns a workgroup (gated: their gate and up
// rows of B).  The eight waves share the reduction: wave w takes steps w, w + 8,
// ..., straight from memory into the fragments (a row of B is wanted by this
// workgroup alone, so LDS has nothing to share), and one sum over the waves
// through LDS ends in the epilogue.  No second launch joins parts, and a
// workgroup is 16 columns, so that few of them fill the compute units.  What
// bounds it is its own loads: 26 KB of B a microsecond, and A once more for
// every 16 columns.  Against the ring and its join, bf16: 1 x 4096 x 4096
// 9.3 us (ring 11.1), gated 1 x 4096 x 4096 16.3 (19.6), 16 x 2048 x 2048 6.4
// (8.8), but 1 x 14336 x 4096 27 (23) and 32 x 14336 x 4096 50 (28); e4m3 1 x
// 4096 x 4096 7.2 (10.7).  B's loads are non-temporal also where rows do not start at a
// cache line and two waves share one, unlike the ring's: 15 such sizes take the
// same time within 1% either way, from memory and from the caches (1 x 4104 x
// 4096 bf16 9.0 and 6.6 us).
template <int DT, Form kForm, int MT>
__global__ __launch_bounds__(64 * kRowsWaves) void gemm_rows_kernel(GemmArgs p) {
  constexpr bool kGated = kForm == kGatedForm;
  constexpr int NB = kGated ? 2 : 1, NF = MT * NB;
  constexpr int U = MT + NB <= 3 ? 4 : 2;  // steps in flight a wave
  __shared__ bk_f32x4 sums[kRowsWaves][NF][64];
  const int n0 = blockIdx.x * 16;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const int nk = (int)((p.kb + kStepBytes - 1) / kStepBytes);

  uint32_t offa[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int m = 16 * i + l16;
    offa[i] = (uint32_t)(m < p.M ? m : p.M - 1) * (uint32_t)p.lda + 16 * g;
  }
  const uint32_t offb = (uint32_t)(n0 + l16 < p.N ? l16 : p.N - 1 - n0) * (uint32_t)p.ldb + 16 * g;
  const char* gate = p.B + n0 * p.ldb;
  const char* up = gate + p.N * p.ldb;

  bk_f32x4 acc[MT][NB];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[i][j] = bk_f32x4{0.f, 0.f, 0.f, 0.f};

  for (int k0 = wave; k0 < nk; k0 += kRowsWaves * U) {
    bk_u32x4 fa[U][MT][2], fb[U][NB][2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + kRowsWaves * u;
      if (k >= nk) break;
      const int64_t at = (int64_t)k * kStepBytes, left = p.kb - at;
      auto get = [&](const char* base, uint32_t off, bk_u32x4 (&f)[2], bool once) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          // past the reduction's end: zeros, from the step's first chunk
          const bool past = 16 * g + 64 * s >= left;
          const bk_u32x4* from = reinterpret_cast<const bk_u32x4*>(
              base + at + (past ? off - 16 * g : off + 64 * s));
          f[s] = once ? __builtin_nontemporal_load(from) : *from;
          if (left < kStepBytes) f[s] = past ? bk_u32x4{0, 0, 0, 0} : f[s];
        }
      };
#pragma unroll
      for (int i = 0; i < MT; ++i) get(p.A, offa[i], fa[u][i], false);
      get(gate, offb, fb[u][0], true);
      if constexpr (kGated) get(up, offb, fb[u][1], true);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (k0 + kRowsWaves * u >= nk) break;
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j) acc[i][j] = mma<DT>(fb[u][j], fa[u][i], acc[i][j]);
    }
  }
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) sums[wave][i * NB + j][lane] = acc[i][j];
  __syncthreads();
  // eight columns a thread: lanes 16 (2 h) + m and 16 (2 h + 1) + m of a tile
  const int t = threadIdx.x;
  if (t >= MT * 32) return;
  const int m16 = t & 15, h = t >> 4 & 1, i = t >> 5;
  const int m = 16 * i + m16, n = n0 + 8 * h;
  if (m >= p.M || n >= p.N) return;
  float z[8], u[8];
  auto total = [&](int f, float (&v)[8]) {
    bk_f32x4 lo = {0.f, 0.f, 0.f, 0.f}, hi = lo;
#pragma unroll
    for (int w = 0; w < kRowsWaves; ++w) {
      lo += sums[w][f][32 * h + m16];
      hi += sums[w][f][32 * h + 16 + m16];
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] = lo[r], v[4 + r] = hi[r];
  };
  total(i * NB, z);
  if constexpr (kGated) total(i * NB + 1, u);
  epilogue8<kGated, false>(p, m, n, z, u, Extra<kGated>{});
}

template <int DT, Form kForm>
void launch_rows(const GemmArgs& a, hipStream_t st) {
  const dim3 grid((a.N + 15) / 16);
  if (a.M <= 16)
    hipLaunchKernelGGL((gemm_rows_kernel<DT, kForm, 1>), grid, dim3(64 * kRowsWaves), 0, st, a);
  else
    hipLaunchKernelGGL((gemm_rows_kernel<DT, kForm, 2>), grid, dim3(64 * kRowsWaves), 0, st, a);
}

template <int DT, Form kForm, int BM, int BN, int WM, int WN, int NST, bool kOnce, bool kLines>
void launch_ring_as(const GemmArgs& a, hipStream_t st) {
  hipLaunchKernelGGL((gemm_ring_kernel<DT, kForm, BM, BN, WM, WN, NST, kOnce, kLines>),
                     dim3(a.whole + (a.tiles_m * a.tiles_n - a.whole) * a.splits),
                     dim3(BM / WM * (BN / WN) * 64), 0, st, a);
}
// NSL: stages with kLines, where one more is in use
template <int DT, Form kForm, int BM, int BN, int WM, int WN, int NST, int NSL>
void launch_ring(const GemmArgs& a, hipStream_t st) {
  if constexpr (kForm == kLinearForm || kForm == kGatedForm) {
    const bool off_lines = ((uintptr_t)a.A | (uintptr_t)a.B | (uint64_t)a.kb) % kStepBytes != 0;
    // (fp32, and e4m3 that is widened, are bound by their products there)
    constexpr bool kMay = BM >= 64 && (DT == LORA_BF16 || DT == LORA_E4M3);
    const bool lines = kMay && off_lines && a.lines;
    const bool once = BM <= 64 && a.tiles_m == 1 && (lines || !off_lines);
    if constexpr (kMay && BM == 64)
      if (once && lines) return launch_ring_as<DT, kForm, BM, BN, WM, WN, NSL, true, true>(a, st);
    if constexpr (BM <= 64)
      if (once) return launch_ring_as<DT, kForm, BM, BN, WM, WN, NST, true, false>(a, st);
    if constexpr (kMay)
      if (lines) return launch_ring_as<DT, kForm, BM, BN, WM, WN, NSL, false, true>(a, st);
  }
  launch_ring_as<DT, kForm, BM, BN, WM, WN, NST, false, false>(a, st);
}

template <int DT, Form kForm>
int32_t launch_form(int shape, const GemmArgs& a, hipStream_t st) {
  // gated: a wave's rows of B are the gate and the up rows of the same columns
  constexpr bool kGated = kForm == kGatedForm;
  if constexpr (kForm == kLinearForm || kForm == kGatedForm) {
    if (shape == kRowsShape) {
      launch_rows<DT, kForm>(a, st);
      return check_launch("product of few rows");
    }
  }
  if (shape == 0)
    launch_ring<DT, kForm, 32, 32, 16, kGated ? 32 : 16, 6, 6>(a, st);
  else if (shape == 1)
    launch_ring<DT, kForm, 64, 64, kGated ? 16 : 32, kGated ? 64 : 32, 4, 5>(a, st);
  else if (shape == 2)
    launch_ring<DT, kForm, 128, 128, 64, 64, 3, 4>(a, st);
  else {
    const dim3 grid(a.whole + (a.tiles_m * a.tiles_n - a.whole) * a.splits);
    hipLaunchKernelGGL((gemm_phase_kernel<DT, kForm>), grid, dim3(512), 0, st, a);
  }
  return check_launch("product");
}

template <int DT, int BM, int BN, int WM, int WN, int NST>
void launch_pair_of(const GemmArgs& x, const GemmArgs& w, hipStream_t st) {
  const int nx = x.whole + (x.tiles_m * x.tiles_n - x.whole) * x.splits;
  const int nw = w.whole + (w.tiles_m * w.tiles_n - w.whole) * w.splits;
  const bool x_first = x.kb / x.splits >= w.kb / w.splits;
  hipLaunchKernelGGL((gemm_pair_kernel<DT, BM, BN, WM, WN, NST>), dim3(nx + nw),
                     dim3(BM / WM * (BN / WN) * 64), 0, st, x, w, x_first ? nx : nw, x_first);
}
template <int DT>
int32_t launch_pair(int shape, const GemmArgs& x, const GemmArgs& w, hipStream_t st) {
  if (shape == 0)
    launch_pair_of<DT, 32, 32, 16, 16, 6>(x, w, st);
  else if (shape == 1)
    launch_pair_of<DT, 64, 64, 32, 32, 4>(x, w, st);
  else
    launch_pair_of<DT, 128, 128, 64, 64, 3>(x, w, st);
  return check_launch("products of the gradients");
}

// the forms of the forward pass, and those of the gradients
template <int DT>
int32_t launch(Form form, int shape, const GemmArgs& a, hipStream_t st) {
  return form == kGatedForm ? launch_form<DT, kGatedForm>(shape, a, st)
                            : launch_form<DT, kLinearForm>(shape, a, st);
}
template <int DT>
int32_t launch_any(Form form, int shape, const GemmArgs& a, hipStream_t st) {
  if (form == kGradX) return launch_form<DT, kGradX>(shape, a, st);
  if (form == kGradW) return launch_form<DT, kGradW>(shape, a, st);
  return launch<DT>(form, shape, a, st);
}

}  // namespace gemm
}  // namespace lora
