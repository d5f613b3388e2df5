// Runs on the host: the limit of the waits inside the attention kernels, and which copies the
// few-rows kernel has on their way when one of its waits runs out.  Prints "ok" and exits 0.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdio>

#define CS_KV_WAIT_TRIES 1000
#include "../../consumer_gemm_chain_gb300/csrc/cs_kv_rows.cuh"

using namespace cskv;

#define REQUIRE(x)                                     \
  do {                                                 \
    if (!(x)) {                                        \
      printf("line %d: not true: %s\n", __LINE__, #x); \
      return 1;                                        \
    }                                                  \
  } while (0)

template <int ST>
static int copies() {
  for (int k1 = 1; k1 < 40; ++k1)  // a segment's tiles, after `before` of others
    for (unsigned before = 0; before < 9; ++before)
      for (int stop = 0; stop < k1; ++stop)
        for (int at_values = 0; at_values < 2; ++at_values) {
          unsigned issued[2][ST] = {}, total[2] = {before, before};
          for (unsigned n = 0; n < before; ++n) ++issued[0][n % ST], ++issued[1][n % ST];
          auto load = [&](int which, int k) {
            if (k < k1) ++issued[which][total[which]++ % ST];
          };
          for (int k = 0; k < ST; ++k) load(0, k), load(1, k);
          for (int k = 0; k <= stop; ++k) {
            if (k == stop && !at_values) break;
            load(0, k + ST);  // K of tile k is read
            if (k == stop) break;
            load(1, k + ST);
          }
          for (int which = 0; which < 2; ++which)
            for (int s = 0; s < ST; ++s)
              REQUIRE(rows_issued<ST>(which, s, at_values, before + stop, k1 - stop) == issued[which][s]);
        }
  return 0;
}

int main() {
  // what never comes: the limit once, and then no wait that is not satisfied at once
  volatile int abort = 0;
  int tries = 0;
  REQUIRE(!wait_bounded(&abort, [&] { return ++tries, false; }));
  REQUIRE(abort == 1 && tries == 1000);
  for (int i = 0; i < 5; ++i) {
    tries = 0;
    REQUIRE(!wait_bounded(&abort, [&] { return ++tries, false; }));
    REQUIRE(tries == 1);
  }
  REQUIRE(wait_bounded(&abort, [] { return true; }));
  abort = 0;
  tries = 0;
  REQUIRE(wait_bounded(&abort, [&] { return ++tries == 1000; }) && abort == 0);
  if (copies<2>() || copies<4>()) return 1;
  printf("ok\n");
  return 0;
}
