// Host plan of the gradients of the adapters' delta: rows sorted by adapter, row
// tiles, and the pieces of each adapter's rows whose gradients one workgroup sums.
#include <algorithm>
#include <cstring>

#include "lora_delta.h"

namespace lora {

namespace {

int64_t column_tiles(const Geo& g) {
  const int64_t c = delta_column_tile(g);
  int64_t n = g.S * ((g.K + c - 1) / c);
  for (int s = 0; s < g.S; ++s) n += (g.out[s] + c - 1) / c;
  return n * delta_ranks(g.R).blocks;
}

// Rows of a piece: with pieces no longer than this the workgroups of the
// gradients hold no more than their share of the rows (their time is their
// rows'), and an adapter's rows are cut only where that needs it: every piece of
// a cut run writes a partial of its adapter's gradients.
int64_t piece_rows(const Geo& g, int64_t rows) {
  const int64_t share = (rows * column_tiles(g) + kDeltaAim - 1) / kDeltaAim;
  return align_up(share < 128 ? 128 : share, 64);
}

// A bound of the pieces that write partials, and that does not fall as T grows:
// only runs longer than a piece are cut, so that two pieces hold more rows than one.
int64_t most_partials(const Geo& g, int64_t T) {
  const int64_t by_rows = 2 * T / 128, by_share = 2 * kDeltaAim / column_tiles(g);
  return by_rows < by_share ? by_rows : by_share;
}

int64_t shrinks(const Geo& g, int64_t chunk) {
  int64_t n = g.S * ((g.K + chunk - 1) / chunk);
  for (int s = 0; s < g.S; ++s) n += (g.out[s] + chunk - 1) / chunk;
  return n;
}

// Columns of a part of the shrink's reductions: the fewest parts that give every
// compute unit four workgroups.
int64_t shrink_chunk(const Geo& g, int64_t tiles) {
  int64_t len = g.K;
  for (int s = 0; s < g.S; ++s) len = g.out[s] > len ? g.out[s] : len;
  int64_t chunk = align_up(len, 64);
  for (int parts = 2; parts <= kDeltaMaxSplits; ++parts) {
    if (tiles * delta_ranks(g.R).blocks * shrinks(g, chunk) >= kDeltaShrinks) break;
    const int64_t c = align_up((len + parts - 1) / parts, 64);
    if (c < 256) break;
    chunk = c;
  }
  return chunk;
}

struct Words {
  int64_t perm, tiles, parts, multi, total;
};
// Capacities for any batch of T rows: every adapter adds at most one partial
// tile, and so do the rows without one.
Words capacity(const Geo& g, int32_t T) {
  const int64_t runs = (T < g.max_loras ? T : g.max_loras) + 1;
  const int64_t tiles = T / kDeltaTileRows + runs + 1, parts = T / 128 + runs + 1;
  Words w;
  w.perm = 0;
  w.tiles = align_up(T, 4);
  w.parts = w.tiles + 4 * tiles;
  w.multi = w.parts + 4 * parts;
  w.total = w.multi + 4 * (T / 128 + 1);
  return w;
}

}  // namespace

DeltaLayout delta_layout(const Geo& g, int32_t T) {
  const DeltaRanks r = delta_ranks(g.R);
  const int64_t sides = 2 * g.S, tile = kDeltaTileRows, e = elem_bytes(g.dtype);
  // Every adapter adds at most one tile that is not full, and no tile is empty.
  const int64_t runs = T < g.max_loras ? T : g.max_loras;
  const int64_t tiles = T < T / tile + runs ? T : T / tile + runs;
  // Reductions are cut only while the unsplit workgroups are fewer than wanted.
  const int64_t few = kDeltaShrinks / (sides * r.blocks) + 1;
  const int64_t planes = g.dtype == LORA_BF16 ? 3 : 1;
  DeltaLayout l;
  l.turned = 0;
  l.straight = l.turned + align_up(planes * sides * tiles * tile * r.padded * e, 256);
  l.partial = l.straight + align_up(g.S * tiles * tile * r.padded * 4, 256);
  l.grads = l.partial + align_up((int64_t)kDeltaMaxSplits * sides * (tiles < few ? tiles : few) *
                                     tile * r.padded * 4,
                                 256);
  l.total = l.grads + align_up(most_partials(g, T) * delta_grad_values(g) * 4, 256);
  return l;
}

int32_t delta_check_plan(const Geo& g, int32_t T, const lora_delta_plan* p) {
  if (!p) return fail(LORA_E_ARG, "plan is NULL");
  const Words w = capacity(g, T);
  const int64_t tiles = (int64_t)p->tiles + p->none_tiles;
  const bool fits =
      p->rows >= 0 && p->none >= 0 && (int64_t)p->rows + p->none == T && p->tiles >= 0 &&
      p->none_tiles >= 0 && p->parts >= 0 && p->multi >= 0 && p->partials >= 0 &&
      p->partials <= most_partials(g, T) && p->chunk >= 64 && p->chunk % 64 == 0 &&
      p->off_perm == 0 && p->off_tiles == align_up(T, 4) &&
      p->off_parts == p->off_tiles + 4 * tiles &&
      p->off_multi == p->off_parts + 4 * (int64_t)p->parts &&
      p->image_bytes == 4 * (p->off_multi + 4 * (int64_t)p->multi) &&
      p->image_bytes <= 4 * w.total && (p->tiles > 0) == (p->rows > 0) &&
      (p->none_tiles > 0) == (p->none > 0) && (p->parts > 0) == (p->rows > 0) &&
      p->longest >= 0 && p->longest <= p->rows && p->max_loras == g.max_loras;
  if (!fits || p->chunk != shrink_chunk(g, p->tiles))
    return fail(LORA_E_ARG, "the plan is not lora_delta_backward_plan's for this pool and T");
  return LORA_OK;
}

}  // namespace lora

using namespace lora;

static int32_t check_batch(const lora_pool_desc* desc, int32_t T, Geo* g) {
  if (int32_t e = check_desc(desc, g)) return e;
  if (T < 0) return fail(LORA_E_ARG, "T must be >= 0, got %d", T);
  if (T > 1 << 21) return fail(LORA_E_SHAPE, "T must be at most %d, got %d", 1 << 21, T);
  g->T = T;
  return LORA_OK;
}

extern "C" int64_t lora_delta_backward_image_bytes(const lora_pool_desc* desc, int32_t T) {
  clear_error();
  Geo g;
  if (int32_t e = check_batch(desc, T, &g)) return e;
  // (the counters of the sort lie behind the image)
  return 4 * (capacity(g, T).total + g.max_loras + 2);
}

extern "C" int64_t lora_delta_backward_workspace_bytes(const lora_pool_desc* desc, int32_t T) {
  clear_error();
  Geo g;
  if (int32_t e = check_batch(desc, T, &g)) return e;
  return delta_layout(g, T).total;
}

extern "C" int32_t lora_delta_backward_plan(const lora_pool_desc* desc, int32_t T,
                                            const int32_t* ids, void* image, int64_t image_bytes,
                                            lora_delta_plan* plan) {
  clear_error();
  Geo g;
  if (int32_t e = check_batch(desc, T, &g)) return e;
  if (!plan) return fail(LORA_E_ARG, "plan is NULL");
  if (T && !ids) return fail(LORA_E_ARG, "ids is NULL");
  const Words w = capacity(g, T);
  const int64_t need = 4 * (w.total + g.max_loras + 2);
  if (!image) return fail(LORA_E_ARG, "image is NULL");
  if (image_bytes < need)
    return fail(LORA_E_WORKSPACE, "image holds %lld bytes, the plan needs %lld",
                (long long)image_bytes, (long long)need);
  for (int32_t t = 0; t < T; ++t)
    if (ids[t] < -1 || ids[t] >= g.max_loras)
      return fail(LORA_E_ID, "ids[%d] = %d, outside [-1, %d)", t, ids[t], g.max_loras);

  // Rows by adapter, in token order; those without one at the end.
  int32_t* const at = (int32_t*)image;
  int32_t* const next = at + w.total;  // [max_loras + 1]: each run's next place
  std::memset(next, 0, (size_t)(g.max_loras + 2) * 4);
  auto run_of = [&](int32_t t) { return ids[t] < 0 ? g.max_loras : ids[t]; };
  for (int32_t t = 0; t < T; ++t) ++next[run_of(t) + 1];
  for (int32_t a = 0; a <= g.max_loras; ++a) next[a + 1] += next[a];
  const int32_t rows = next[g.max_loras];
  for (int32_t t = 0; t < T; ++t) at[next[run_of(t)]++] = t;
  // (next[a] is now the end of run a)

  lora_delta_plan p{};
  p.rows = rows;
  p.none = T - rows;
  int32_t* put = at + w.tiles;
  auto record = [&put](int32_t a, int32_t b, int32_t c, int32_t d) {
    put[0] = a;
    put[1] = b;
    put[2] = c;
    put[3] = d;
    put += 4;
  };
  auto cut_tiles = [&](int32_t slot, int32_t from, int32_t to) {
    int32_t n = 0;
    for (int32_t r = from; r < to; r += kDeltaTileRows, ++n)
      record(slot, to - r < kDeltaTileRows ? to - r : kDeltaTileRows, r, 0);
    return n;
  };
  for (int32_t a = 0; a < g.max_loras; ++a)
    p.tiles += cut_tiles(a, a ? next[a - 1] : 0, next[a]);
  p.none_tiles = cut_tiles(-1, rows, T);
  p.off_perm = 0;
  p.off_tiles = w.tiles;
  p.off_parts = put - at;
  const int64_t most = piece_rows(g, rows);
  for (int32_t a = 0, tile = 0; a < g.max_loras; ++a) {
    const int32_t n = next[a] - (a ? next[a - 1] : 0);
    if (!n) continue;
    // equal pieces, whole steps of 64 rows; a cut costs about what 256 rows do
    const int64_t k = n > most + 256 ? (n + most - 1) / most : 1;
    const int64_t each = align_up((n + k - 1) / k, 64);
    for (int64_t r = 0; r < n; r += each, ++p.parts)
      record(a, (int32_t)(n - r < each ? n - r : each), tile + (int32_t)(r / kDeltaTileRows),
             k > 1 ? p.partials++ : -1);
    tile += (n + kDeltaTileRows - 1) / kDeltaTileRows;
  }
  p.off_multi = put - at;
  struct Record {
    int32_t w[4];
  };
  for (int32_t i = 0, q = 0; i < p.parts; ++i) {
    const int32_t* part = at + p.off_parts + 4 * i;
    if (part[3] < 0) continue;
    if (i == 0 || part[0] != part[-4]) {
      record(part[0], q, 0, 0);
      ++p.multi;
    }
    ++put[-2];
    ++q;
  }
  // the longest pieces first (ties in order)
  Record* const parts = reinterpret_cast<Record*>(at + p.off_parts);
  std::sort(parts, parts + p.parts, [](const Record& a, const Record& b) {
    return a.w[1] != b.w[1] ? a.w[1] > b.w[1] : a.w[2] < b.w[2];
  });
  p.max_loras = g.max_loras;
  p.longest = p.parts ? parts[0].w[1] : 0;
  p.chunk = (int32_t)shrink_chunk(g, p.tiles);
  p.image_bytes = (put - at) * 4;
  *plan = p;
  return LORA_OK;
}
