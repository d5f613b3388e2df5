// Runs on the host: what the operators of the cache in 4 bits refuse, overlaps above all, and what
// cs_attn_cached4_forward refuses before any stage of the chain has run.  Prints "ok" and exits 0.
#include "kv_host.cuh"

#include "../../consumer_gemm_chain_gb300/csrc/cs_kv4.cu"

int main() {
  constexpr int HEADS = 4, KV_HEADS = 2, DIM = 64, TOKENS = 3, PAGES = 2, PAGE = 16;
  constexpr long long Q = HEADS * DIM, KV = KV_HEADS * DIM, W = Q + 2 * KV, CODES = PAGES * PAGE * KV / 2, SCALES = PAGES * PAGE * KV / 32;
  cs_kv_s plan;
  if (cs_kv_desc_init(&plan.d) != CS_OK) return 1;
  plan.d.heads = HEADS;
  plan.d.kv_heads = KV_HEADS;
  plan.d.head_dim = DIM;
  plan.d.num_pages = PAGES;
  plan.d.max_tokens = plan.d.max_seqs = TOKENS;
  plan.num_sms = 152;
  static int cu[2], lens[1], table[1];
  const cs_kv_batch batch{TOKENS, 1, TOKENS, 1, cu, lens, table};
  alignas(32) static char store[1 << 20];
  auto mem = [&](int i) { return store + i * 65536; };  // places that do not overlap
  const cs_kv4_cache k{mem(2), mem(3)}, v{mem(4), mem(5)};

  // append
  cs_kv4_append_args good{};
  good.qkv = mem(0);
  good.q_out = mem(1);
  good.k = k;
  good.v = v;
  cskv::Four4P f;
  auto append = [&](const cs_kv4_append_args& a) { return check_append4(&plan, &batch, &a, f); };
  REQUIRE(append(good) == CS_OK);
  REQUIRE(check_append4(&plan, &batch, nullptr, f) == CS_ERR_INVALID_ARG);
  void* cs_kv4_cache::*const parts[2] = {&cs_kv4_cache::codes, &cs_kv4_cache::scales};
  cs_kv4_cache cs_kv4_append_args::*const caches[2] = {&cs_kv4_append_args::k, &cs_kv4_append_args::v};
  const long long bytes[2] = {CODES, SCALES};
  cs_kv4_append_args a;
  for (auto cache : caches)
    for (int part = 0; part < 2; ++part) {
      a = good;
      a.*cache.*parts[part] = nullptr;
      REQUIRE(append(a) == CS_ERR_INVALID_ARG);
      a.*cache.*parts[part] = mem(7) + 8;
      REQUIRE(append(a) == CS_ERR_INVALID_ARG);
      a = good;
      char* at = static_cast<char*>(a.*cache.*parts[part]);
      a.q_out = at + bytes[part] - 16;
      REQUIRE(append(a) == CS_ERR_INVALID_ARG);
      a.q_out = at + bytes[part];
      REQUIRE(append(a) == CS_OK);
      a = good;
      a.qkv = at - TOKENS * W * 2 + 16;
      REQUIRE(append(a) == CS_ERR_INVALID_ARG);
      a.qkv = at - TOKENS * W * 2;
      REQUIRE(append(a) == CS_OK);
      // every part against every other one
      for (auto other : caches)
        for (int which = 0; which < 2; ++which) {
          if (other == cache && which == part) continue;
          a = good;
          a.*cache.*parts[part] = static_cast<char*>(a.*other.*parts[which]) + bytes[which] - 16;
          REQUIRE(append(a) == CS_ERR_INVALID_ARG);
          a.*cache.*parts[part] = static_cast<char*>(a.*other.*parts[which]) + bytes[which];
          REQUIRE(append(a) == CS_OK);
        }
    }
  a = good;  // in place
  a.q_out = mem(0);
  REQUIRE(append(a) == CS_ERR_INVALID_ARG);
  a.q_stride = W;
  REQUIRE(append(a) == CS_OK);
  a.qkv_stride = a.q_stride = W + 4;
  REQUIRE(append(a) == CS_ERR_INVALID_ARG);
  plan.d.rotary_dim = 32;
  REQUIRE(append(good) == CS_ERR_INVALID_ARG);
  plan.d.rotary_dim = 0;

  // reading
  cs_kv4_read_args some{};
  some.k = k;
  some.v = v;
  some.k_out = mem(0);
  some.v_out = mem(1);
  auto read = [&](const cs_kv4_read_args& x) { return check_read4(&plan, &batch, &x, f); };
  REQUIRE(read(some) == CS_OK && f.units == 2 * KV / 16);
  REQUIRE(check_read4(&plan, &batch, nullptr, f) == CS_ERR_INVALID_ARG);
  cs_kv4_read_args r = some;
  r.k_out = nullptr;
  r.k = cs_kv4_cache{};
  REQUIRE(read(r) == CS_OK && f.units == KV / 16);
  r.v_out = nullptr;
  REQUIRE(read(r) == CS_ERR_INVALID_ARG);
  r = some;
  r.v = cs_kv4_cache{};
  REQUIRE(read(r) == CS_ERR_INVALID_ARG);
  r = some;
  r.v_out = mem(0);
  REQUIRE(read(r) == CS_ERR_INVALID_ARG);
  r.v_out = mem(0) + KV * 2;  // side by side
  REQUIRE(read(r) == CS_ERR_INVALID_ARG);
  r.k_stride = r.v_stride = 2 * KV;
  REQUIRE(read(r) == CS_OK);
  r.k_stride = KV - 8;
  REQUIRE(read(r) == CS_ERR_INVALID_ARG);
  r = some;
  r.k_out = mem(0) + 8;
  REQUIRE(read(r) == CS_ERR_INVALID_ARG);
  for (int place = 2; place < 6; ++place) {
    r = some;
    r.v_out = mem(place) + bytes[place & 1] - 16;
    REQUIRE(read(r) == CS_ERR_INVALID_ARG);
    r.v_out = mem(place) + bytes[place & 1];
    REQUIRE(read(r) == CS_OK);
  }

  // attention
  cs_kv4_attn_args fine{};
  fine.q = mem(0);
  fine.out = mem(1);
  fine.k = k;
  fine.v = v;
  fine.lse = reinterpret_cast<float*>(mem(6));
  cskv::AttnP p;
  auto attend = [&](const cs_kv4_attn_args& x) { return check_attn4(&plan, &batch, &x, p); };
  REQUIRE(attend(fine) == CS_OK);
  REQUIRE(check_attn4(&plan, &batch, nullptr, p) == CS_ERR_INVALID_ARG);
  cs_kv4_attn_args t = fine;
  t.v = k;  // read only: may be one
  REQUIRE(attend(t) == CS_OK);
  t.v.scales = nullptr;
  REQUIRE(attend(t) == CS_ERR_INVALID_ARG);
  t = fine;
  t.out = mem(0);
  REQUIRE(attend(t) == CS_ERR_INVALID_ARG);
  for (int place = 2; place < 6; ++place) {
    t = fine;
    t.out = mem(place) + bytes[place & 1] - 16;
    REQUIRE(attend(t) == CS_ERR_INVALID_ARG);
    t.out = mem(place) + bytes[place & 1];
    REQUIRE(attend(t) == CS_OK);
  }
  for (int other = 0; other < 6; ++other) {
    t = fine;
    t.lse = reinterpret_cast<float*>(mem(other) + 16);
    REQUIRE(attend(t) == CS_ERR_INVALID_ARG);
  }

  // a layer
  constexpr int M = 5, F = 2 * 128;
  cs_kv_s layer;
  if (cs_kv_desc_init(&layer.d) != CS_OK) return 1;
  layer.d.heads = layer.d.kv_heads = 2;
  layer.d.num_pages = PAGES;
  layer.d.max_tokens = 16;
  layer.d.max_seqs = 2;
  layer.d.rotary_dim = 128;
  layer.num_sms = 152;
  cs_chain_s chain;
  chain.d.kind = CS_CHAIN_ATTN;
  chain.d.dtype = layer.d.dtype;
  chain.d.heads = 2;
  chain.d.M = M;
  chain.d.F = F;
  chain.info.split_k[0] = chain.info.split_k[1] = chain.info.split_k[2] = 1;
  chain.info.intermediate[0] = mem(0);
  chain.info.intermediate[1] = mem(1);
  const cs_kv_batch step{M, 2, M, 1, cu, lens, table};
  const cs_attn_args args{mem(8), mem(8), mem(8), mem(8)};
  cs_kv4_append_args into{};
  into.k = k;
  into.v = v;
  into.rope = reinterpret_cast<const float*>(mem(6));
  into.rope_rows = 1;
  auto refused = [&](const cs_kv4_append_args& x, const char* why) {
    const cs_status s = cs_attn_cached4_forward(&chain, &layer, &step, &args, &x, nullptr);
    return s == CS_ERR_INVALID_ARG && std::strstr(last_error, why) != nullptr && chain.stages_run == 0;
  };
  chain.device = 1;
  REQUIRE(refused(into, "device 1"));
  chain.device = 0;
  a = into;
  a.rope = nullptr;
  REQUIRE(refused(a, "rope is required"));
  a = into;
  a.v.scales = nullptr;
  REQUIRE(refused(a, "scales of v"));
  a = into;
  a.v = k;
  REQUIRE(refused(a, "overlap"));
  layer.d.heads = 4;
  REQUIRE(refused(into, "plans differ"));

  // calls without a plan, and of a plan that holds an error
  REQUIRE(cs_kv4_append(nullptr, &batch, &good, nullptr) == CS_ERR_INVALID_ARG);
  REQUIRE(cs_kv4_read(nullptr, &batch, &some, nullptr) == CS_ERR_INVALID_ARG);
  REQUIRE(cs_kv4_attention(nullptr, &batch, &fine, nullptr) == CS_ERR_INVALID_ARG);
  REQUIRE(cs_kv4_attention_shared(nullptr, &batch, nullptr, 0, &fine, nullptr) == CS_ERR_INVALID_ARG);
  REQUIRE(cs_attn_cached4_forward(nullptr, nullptr, &batch, &args, &into, nullptr) == CS_ERR_INVALID_ARG);
  REQUIRE(cs_kv4_attention_shared(&plan, &batch, nullptr, 0, &fine, nullptr) == CS_ERR_INVALID_ARG);  // not asked for
  plan.d.shared = 1;
  REQUIRE(cs_kv4_attention_shared(&plan, &batch, nullptr, 1, &fine, nullptr) == CS_ERR_INVALID_ARG);
  REQUIRE(cs_kv4_attention_shared(&plan, &batch, table, -1, &fine, nullptr) == CS_ERR_INVALID_ARG);
  cs_kv_batch big = batch;
  big.tokens = TOKENS + 1;
  REQUIRE(cs_kv4_read(&plan, &big, &some, nullptr) == CS_ERR_INVALID_ARG);
  plan.error_latched = true;
  REQUIRE(cs_kv4_append(&plan, &batch, &good, nullptr) == CS_ERR_NEEDS_RESET);
  REQUIRE(cs_kv4_read(&plan, &batch, &some, nullptr) == CS_ERR_NEEDS_RESET);
  REQUIRE(cs_kv4_attention(&plan, &batch, &fine, nullptr) == CS_ERR_NEEDS_RESET);
  printf("ok\n");
  return 0;
}
