// The plan of the delta's gradients (lora_delta_plan.cpp) under AddressSanitizer and
// UndefinedBehaviorSanitizer: random pools and batches, the image exactly as large as
// lora_delta_backward_image_bytes says, every row in one tile and one piece, the
// workspace's parts in order.  Built with g++ on the CPU (no HIP code).
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "lora_delta.h"

static int g_fail = 0;
#define CHECK(c)                                                              \
  do {                                                                        \
    if (!(c)) {                                                               \
      std::fprintf(stderr, "check failed at line %d: %s\n", __LINE__, #c);    \
      if (++g_fail > 20) std::exit(1);                                        \
    }                                                                         \
  } while (0)

int main(int argc, char** argv) {
  const int trials = argc > 1 ? std::atoi(argv[1]) : 300;
  std::mt19937 rng(5);
  auto draw = [&](int lo, int hi) { return (int)(lo + rng() % (uint32_t)(hi - lo + 1)); };
  for (int trial = 0; trial < trials; ++trial) {
    lora_pool_desc d{};
    d.dtype = draw(0, 1);
    d.max_loras = trial % 7 == 0 ? draw(1, 5000) : draw(1, 40);
    d.max_lora_rank = 8 * draw(1, 20);
    d.in_features = 8 * draw(1, 700);
    d.num_slices = draw(1, LORA_MAX_SLICES);
    for (int s = 0; s < d.num_slices; ++s) d.out_features[s] = 8 * draw(1, 900);
    const int T = trial % 5 == 0 ? draw(0, 70000) : draw(0, 900);
    std::vector<int32_t> ids(T);
    const int kind = draw(0, 3);
    for (int t = 0; t < T; ++t)
      ids[t] = kind == 0   ? draw(-1, d.max_loras - 1)
               : kind == 1 ? d.max_loras - 1
               : kind == 2 ? (draw(0, 9) ? 0 : draw(-1, d.max_loras - 1))
                           : t % d.max_loras;
    const int64_t bytes = lora_delta_backward_image_bytes(&d, T);
    CHECK(bytes > 0);
    int32_t* image = (int32_t*)std::malloc((size_t)bytes);
    lora_delta_plan p;
    CHECK(lora_delta_backward_plan(&d, T, ids.data(), image, bytes - 1, &p) == LORA_E_WORKSPACE);
    CHECK(lora_delta_backward_plan(&d, T, ids.data(), image, bytes, &p) == LORA_OK);
    std::vector<int> seen(T, 0), in_part(T, 0);
    for (int i = 0; i < p.tiles + p.none_tiles; ++i) {
      const int32_t* r = image + p.off_tiles + 4 * i;
      for (int k = 0; k < r[1]; ++k) {
        CHECK(ids[image[r[2] + k]] == r[0]);
        ++seen[image[r[2] + k]];
      }
    }
    int partials = 0;
    for (int i = 0; i < p.parts; ++i) {
      const int32_t* r = image + p.off_parts + 4 * i;
      const int first = image[p.off_tiles + 4 * r[2] + 2];
      CHECK(r[1] <= p.longest);
      partials += r[3] >= 0;
      for (int k = 0; k < r[1]; ++k) {
        CHECK(ids[image[first + k]] == r[0]);
        ++in_part[image[first + k]];
      }
    }
    for (int t = 0; t < T; ++t) CHECK(seen[t] == 1 && in_part[t] == (ids[t] >= 0));
    CHECK(partials == p.partials && p.rows + p.none == T);
    lora::Geo g;
    CHECK(lora::check_desc(&d, &g) == LORA_OK);
    if (T) CHECK(lora::delta_check_plan(g, T, &p) == LORA_OK);
    const lora::DeltaLayout l = lora::delta_layout(g, T);
    const int64_t slots = (int64_t)p.tiles * lora::kDeltaTileRows;
    const int64_t padded = lora::delta_ranks(g.R).padded, e = lora::elem_bytes(g.dtype);
    const int64_t planes = g.dtype == LORA_BF16 ? 3 : 1, two = g.dtype == LORA_BF16 ? 2 : 1;
    CHECK(l.straight - l.turned >= planes * 2 * g.S * slots * padded * e);
    CHECK(l.partial - l.straight >= two * g.S * slots * padded * e);
    int64_t longest = g.K;
    for (int s = 0; s < g.S; ++s) longest = g.out[s] > longest ? g.out[s] : longest;
    const int64_t splits = (longest + p.chunk - 1) / p.chunk;
    if (p.rows && splits > 1)
      CHECK(l.grads - l.partial >= splits * 2 * g.S * slots * padded * 4);
    CHECK(l.total - l.grads >= p.partials * lora::delta_grad_values(g) * 4);
    if (T) {
      ids[draw(0, T - 1)] = draw(0, 1) ? -2 : d.max_loras;
      CHECK(lora_delta_backward_plan(&d, T, ids.data(), image, bytes, &p) == LORA_E_ID);
    }
    std::free(image);
  }
  std::printf("%d failed checks\n", g_fail);
  return g_fail != 0;
}
