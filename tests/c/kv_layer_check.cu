// Runs on the host: what cs_attn_cached_forward refuses, before any stage of the chain has run.
// The plans are filled in by hand.  Prints "ok" and exits 0.
#include "kv_host.cuh"

int main() {
  constexpr int HEADS = 2, M = 5, F = HEADS * 128;
  cs_kv_s plan;
  if (cs_kv_desc_init(&plan.d) != CS_OK) return 1;
  plan.d.heads = plan.d.kv_heads = HEADS;
  plan.d.num_pages = 4;
  plan.d.max_tokens = 16;
  plan.d.max_seqs = 2;
  plan.d.rotary_dim = 128;
  plan.num_sms = 152;
  alignas(16) static char memory[64];
  cs_chain_s chain;
  chain.d.kind = CS_CHAIN_ATTN;
  chain.d.dtype = plan.d.dtype;
  chain.d.heads = HEADS;
  chain.d.M = M;
  chain.d.F = F;
  chain.info.split_k[0] = chain.info.split_k[1] = chain.info.split_k[2] = 1;
  alignas(16) static char qkv[M * 3 * F * 2], o[M * F * 2];
  chain.info.intermediate[0] = qkv;
  chain.info.intermediate[1] = o;
  static int cu[3], lens[2], table[2];
  const cs_kv_batch batch{M, 2, M, 1, cu, lens, table};
  const cs_attn_args args{memory, memory, memory, memory};
  cs_kv_append_args append{};
  append.k_cache = memory;
  append.v_cache = memory + 32;
  append.rope = reinterpret_cast<const float*>(memory);
  append.rope_rows = 1;
  auto refused = [&](const cs_kv_append_args& a, const char* why) {
    const cs_status s = cs_attn_cached_forward(&chain, &plan, &batch, &args, &a, nullptr);
    return s == CS_ERR_INVALID_ARG && std::strstr(last_error, why) != nullptr && chain.stages_run == 0;
  };
  chain.device = 1;
  REQUIRE(refused(append, "device 1"));
  chain.device = 0;
  // arguments of the append
  cs_kv_append_args a = append;
  a.rope = nullptr;
  REQUIRE(refused(a, "rope is required"));
  a = append;
  a.rope_rows = 0;
  REQUIRE(refused(a, "rope is required"));
  a = append;
  a.rope = reinterpret_cast<const float*>(memory + 4);
  REQUIRE(refused(a, "16-byte aligned"));
  a = append;
  a.k_cache = nullptr;
  REQUIRE(refused(a, "k_cache and v_cache"));
  a = append;
  a.v_cache = memory + 8;
  REQUIRE(refused(a, "16-byte aligned"));
  printf("ok\n");
  return 0;
}
