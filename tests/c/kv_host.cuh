// The paged cache operators in one program with a stand-in for the chain: what the calls of
// cs_attn_cached_forward reach is counted, and nothing of it runs.
#pragma once
#include "../../consumer_gemm_chain_gb300/csrc/cs_kv.cu"

#include <cstdarg>
#include <cstdio>

static char last_error[512];
cs_status cs_fail(cs_status s, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(last_error, sizeof(last_error), fmt, ap);
  va_end(ap);
  return s;
}

struct cs_chain_s {
  cs_chain_desc d{};
  cs_chain_info info{};
  int device = 0;
  int stages_run = 0;
};
const cs_chain_desc* cs_chain_desc_of(cs_chain_t chain) { return &chain->d; }
int cs_chain_device_of(cs_chain_t chain) { return chain->device; }
cs_status cs_chain_query(cs_chain_t chain, cs_chain_info* info) {
  *info = chain->info;
  return CS_OK;
}
cs_status cs_chain_forward_stage(cs_chain_t chain, const void*, int, void*) {
  ++chain->stages_run;
  return CS_OK;
}

#define REQUIRE(x)                                                                \
  do {                                                                            \
    if (!(x)) {                                                                   \
      printf("line %d: not true: %s (last error: %s)\n", __LINE__, #x, last_error); \
      return 1;                                                                   \
    }                                                                             \
  } while (0)
