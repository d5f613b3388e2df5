// Runs on the host: the arithmetic that divides attention over the paged cache, against
// counting.  Prints "ok" and exits 0, or names the first case that differs.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdio>
#include <cstdlib>
#include <vector>

#include "../../consumer_gemm_chain_gb300/csrc/cs_kv_sched.cuh"

using namespace cskv;

static unsigned long long seed = 12345;
static int draw(int a, int b) {  // a .. b
  seed = seed * 6364136223846793005ull + 1442695040888963407ull;
  return a + static_cast<int>((seed >> 33) % static_cast<unsigned long long>(b - a + 1));
}
template <int N>
static int pick(const int (&v)[N]) {
  return v[draw(0, N - 1)];
}

int main() {
  for (int it = 0; it < 1500; ++it) {
    Cut c{};
    c.shift = draw(6, 7);
    const int windows[] = {0, 0, 1, 5, 100, 128, 129, 1000, 1024, 3000}, sinks[] = {0, 1, 4, 64, 128, 130, 500, 4000};
    const int per[] = {1, 2, 3, 4, 16, 20, 36, 50, 64, 84, 256};
    c.per_item = pick(per);
    c.window = pick(windows);
    c.sinks = c.window ? pick(sinks) : 0;
    c.item_cost = draw(0, 2);
    Seq s{0, draw(1, 3) == 1 ? draw(1, 4) : draw(1, 2000), 0};
    const int old[] = {0, 0, 1, 77, 5000};
    s.m = s.n + pick(old) - (draw(0, 9) == 0 ? draw(0, s.n) : 0);
    if (s.m < 0) s.m = 0;
    if (draw(0, 5) == 0) c.flat = 1, c.window = c.sinks = 0, c.flat_len = s.m = draw(1, 5000);
    const int tile = 1 << c.shift;
    unsigned long long sum = 0;
    for (int k = 0; k <= items_of(c, s); ++k) {
      if (units_before(c, s, k) != sum) {
        printf("units before item %d: %llu, counted %llu (shift %d per %d window %d sinks %d n %d m %d)\n", k,
               units_before(c, s, k), sum, c.shift, c.per_item, c.window, c.sinks, s.n, s.m);
        return 1;
      }
      if (k == items_of(c, s)) break;
      // tiles that hold a key some token of the item sees
      const int a = k * c.per_item, e = a + c.per_item < s.n ? a + c.per_item : s.n, base = s.m - s.n;
      std::vector<char> seen(s.m / tile + 2, 0);
      for (int t = a; t < e; ++t) {
        const int pos = base + t, end = c.flat ? s.m : pos + 1, lo = c.window ? (pos - c.window + 1 > 0 ? pos - c.window + 1 : 0) : 0;
        for (int j = lo; j < end; j = (j / tile + 1) * tile) seen[j / tile] = 1;
        for (int j = 0; j < c.sinks && j < end; j += tile) seen[j / tile] = 1;
      }
      const int lo = item_lo(c, s, k), lead = sink_tiles(c, lo), tiles = item_tiles(c, s, k);
      std::vector<char> listed(seen.size() + tiles, 0);
      for (int i = 0; i < tiles; ++i) listed[i < lead ? i : lo / tile + i - lead] += 1;
      for (size_t j = 0; j < seen.size(); ++j)
        if (seen[j] && listed[j] != 1) {
          printf("tile %d of item %d is listed %d times\n", static_cast<int>(j), k, listed[j]);
          return 1;
        }
      sum += tiles + c.item_cost;
    }
  }
  printf("ok\n");
  return 0;
}
