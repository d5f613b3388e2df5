// Runs on the host: an MMA warp of the attention over the paged cache begins an item only when
// the item's queries have arrived, however late the copies are that it does not read itself.
// Prints "ok" and exits 0, or names the items.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdio>
#include <vector>

#include "../../consumer_gemm_chain_gb300/csrc/cs_kv_attn.cuh"

using namespace cskv;

// A query buffer's barrier: copies are issued in the items' order, and one lands only when
// somebody waits for it (the latest that it can).
struct Barrier {
  int issued = 0, landed = 0;
  bool wait(unsigned parity) {
    while ((landed & 1u) == parity) {  // the phase with this parity is not complete
      if (landed == issued) return false;  // a wait for a copy that was never issued
      ++landed;
    }
    return true;
  }
};

// Waiting for what the warp reads, and for nothing else: the mistake that this test has to find.
struct OwnOnly {
  uint32_t phase = 0;
  template <typename Wait>
  bool arrived(bool two, int w, Wait wait) {
    const int b = two ? w : 0;
    const bool ok = wait(b, phase >> b & 1u);
    phase ^= two ? 3u : 1u;
    return ok;
  }
};

template <typename Q>
static bool sound(const std::vector<bool>& items, int w) {
  Barrier bar[2];
  Q queries;
  for (bool two : items) {
    ++bar[0].issued;
    if (two) ++bar[1].issued;
    if (!queries.arrived(two, w, [&](int b, uint32_t parity) { return bar[b].wait(parity); })) return false;
    const Barrier& own = bar[two ? w : 0];
    if (own.landed != own.issued) return false;
  }
  return true;
}

int main() {
  int found = 0;
  for (int count = 1; count <= 10; ++count)
    for (int bits = 0; bits < 1 << count; ++bits) {
      std::vector<bool> items;
      for (int i = 0; i < count; ++i) items.push_back(bits >> i & 1);
      for (int w = 0; w < 2; ++w) {
        found += !sound<OwnOnly>(items, w);
        if (!sound<Queries>(items, w)) {
          printf("warp %d, items of two row tiles (bit by bit, %d): %d\n", w, count, bits);
          return 1;
        }
      }
    }
  if (found == 0) {
    printf("a warp that waits for its own queries only was not noticed\n");
    return 1;
  }
  printf("ok\n");
  return 0;
}
