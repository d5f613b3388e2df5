// Runs on the host: which overlapping arguments append and attention refuse.  Prints "ok" and exits 0.
#include "kv_host.cuh"

#include <vector>

static unsigned long long seed = 7;
static int draw(int a, int b) {  // a .. b
  seed = seed * 6364136223846793005ull + 1442695040888963407ull;
  return a + static_cast<int>((seed >> 33) % static_cast<unsigned long long>(b - a + 1));
}

int main() {
  // rows against a contiguous range, by marking bytes
  std::vector<char> at(6000);
  for (int it = 0; it < 20000; ++it) {
    const int rows = draw(0, 5), width = 8 * draw(1, 6), stride = width + 8 * draw(0, 20), bytes = draw(0, 1) ? draw(1, 60) : draw(1, 2000);
    const int a = 16 * draw(0, 120), c = draw(0, 3900);
    std::fill(at.begin(), at.end(), 0);
    for (int r = 0; r < rows; ++r) std::fill_n(at.begin() + a + 2 * r * stride, 2 * width, 1);
    bool both = false;
    for (int i = c; i < c + bytes; ++i) both |= at[i] != 0;
    REQUIRE(rows_over(at.data() + a, stride, width, rows, at.data() + c, bytes) == both);
  }

  constexpr int HEADS = 4, KV_HEADS = 2, DIM = 64, TOKENS = 3, PAGES = 2, PAGE = 16;
  constexpr long long Q = HEADS * DIM, W = Q + 2 * KV_HEADS * DIM, CACHE = PAGES * PAGE * KV_HEADS * DIM * 2;
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

  cs_kv_append_args good{};
  good.qkv = mem(0);
  good.q_out = mem(1);
  good.k_cache = mem(2);
  good.v_cache = mem(3);
  cskv::AppendP ak;
  auto append = [&](const cs_kv_append_args& a) { return check_append(&plan, &batch, &a, ak); };
  REQUIRE(append(good) == CS_OK);
  cs_kv_append_args a = good;
  a.v_cache = mem(2);  // both caches the same
  REQUIRE(append(a) == CS_ERR_INVALID_ARG);
  a.v_cache = mem(2) + CACHE - 16;
  REQUIRE(append(a) == CS_ERR_INVALID_ARG);
  a.v_cache = mem(2) + CACHE;  // one behind the other
  REQUIRE(append(a) == CS_OK);
  for (int cache = 0; cache < 2; ++cache) {
    char* c = mem(2 + cache);
    a = good;
    a.q_out = c + CACHE - 32;
    REQUIRE(append(a) == CS_ERR_INVALID_ARG);
    a.q_out = c - TOKENS * Q * 2;
    REQUIRE(append(a) == CS_OK);
    a = good;
    a.qkv = c - TOKENS * W * 2 + 16;
    REQUIRE(append(a) == CS_ERR_INVALID_ARG);
    a.qkv = c + CACHE;
    REQUIRE(append(a) == CS_OK);
  }
  a = good;  // in place
  a.q_out = mem(0);
  a.q_stride = W;
  REQUIRE(append(a) == CS_OK);

  // one row in place: its stride means nothing
  const cs_kv_batch single{1, 1, 1, 1, cu, lens, table};
  a.q_stride = 0;
  REQUIRE(append(a) == CS_ERR_INVALID_ARG);
  REQUIRE(check_append(&plan, &single, &a, ak) == CS_OK);
  a.q_out = mem(0) + 16;
  REQUIRE(check_append(&plan, &single, &a, ak) == CS_ERR_INVALID_ARG);

  cs_kv_attn_args fine{};
  fine.q = mem(0);
  fine.out = mem(1);
  fine.k_cache = mem(2);
  fine.v_cache = mem(3);
  fine.lse = reinterpret_cast<float*>(mem(4));
  cskv::AttnP k;
  auto attend = [&](const cs_kv_attn_args& x) { return check_attn(&plan, &batch, &x, k); };
  REQUIRE(attend(fine) == CS_OK);
  cs_kv_attn_args t = fine;
  t.v_cache = mem(2);  // read only: may be one
  REQUIRE(attend(t) == CS_OK);
  for (int cache = 0; cache < 2; ++cache) {
    t = fine;
    t.out = mem(2 + cache) + 64;
    REQUIRE(attend(t) == CS_ERR_INVALID_ARG);
  }
  for (int other = 0; other < 4; ++other) {
    t = fine;
    t.lse = reinterpret_cast<float*>(mem(other) + 16);
    REQUIRE(attend(t) == CS_ERR_INVALID_ARG);
    t.lse = reinterpret_cast<float*>(mem(other) - TOKENS * HEADS * 4);
    REQUIRE(other == 0 || attend(t) == CS_OK);
  }
  t = fine;  // between the rows of out
  t.out_stride = Q + 64;
  t.lse = reinterpret_cast<float*>(mem(1) + Q * 2);
  REQUIRE(attend(t) == CS_OK);
  printf("ok\n");
  return 0;
}
