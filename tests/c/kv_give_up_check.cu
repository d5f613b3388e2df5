// Runs on a GPU, built with a limit of no tries: every wait inside the attention kernels runs
// out at once, with copies on their way.  Each call must end soon and leave the status and
// nothing else.  Prints "ok" and exits 0.
#define CS_KV_WAIT_TRIES 0
#include "kv_host.cuh"

#include <chrono>
#include <vector>

static int run(int dtype, int head_dim, int tokens_each, int prefix, int window) {
  constexpr int SEQS = 3, HEADS = 8, KV_HEADS = 2, PAGE = 16, COLS = 140;
  const int lens[SEQS] = {900, 300, 2200}, tokens = SEQS * tokens_each;
  const int pages = SEQS * COLS + (prefix + PAGE - 1) / PAGE;
  cs_kv_desc d;
  REQUIRE(cs_kv_desc_init(&d) == CS_OK);
  d.dtype = dtype;
  d.heads = HEADS;
  d.kv_heads = KV_HEADS;
  d.head_dim = head_dim;
  d.num_pages = pages;
  d.max_tokens = tokens;
  d.max_seqs = SEQS;
  d.window = window;
  d.shared = prefix > 0;
  cs_kv_t plan = nullptr;
  REQUIRE(cs_kv_plan(&d, &plan) == CS_OK);
  std::vector<int> table(SEQS * COLS), cu(SEQS + 1), prefix_pages;
  for (int i = 0; i < SEQS * COLS; ++i) table[i] = i;
  for (int i = 0; i <= SEQS; ++i) cu[i] = i * tokens_each;
  for (int i = SEQS * COLS; i < pages; ++i) prefix_pages.push_back(i);
  prefix_pages.push_back(0);
  const size_t rows = static_cast<size_t>(tokens) * HEADS * head_dim * 2, cache = static_cast<size_t>(pages) * PAGE * KV_HEADS * head_dim * 2;
  void *q, *out, *k, *v;
  int *cu_d, *lens_d, *table_d, *prefix_d;
  float* lse;
  REQUIRE(cudaMalloc(&q, rows) == cudaSuccess && cudaMalloc(&out, rows) == cudaSuccess && cudaMalloc(&k, cache) == cudaSuccess &&
          cudaMalloc(&v, cache) == cudaSuccess && cudaMalloc(&lse, tokens * HEADS * 4) == cudaSuccess);
  REQUIRE(cudaMalloc(&cu_d, sizeof(int) * cu.size()) == cudaSuccess && cudaMalloc(&lens_d, sizeof(lens)) == cudaSuccess &&
          cudaMalloc(&table_d, sizeof(int) * table.size()) == cudaSuccess &&
          cudaMalloc(&prefix_d, sizeof(int) * prefix_pages.size()) == cudaSuccess);
  REQUIRE(cudaMemset(q, 0, rows) == cudaSuccess && cudaMemset(k, 0, cache) == cudaSuccess && cudaMemset(v, 0, cache) == cudaSuccess &&
          cudaMemset(out, 0x47, rows) == cudaSuccess);
  REQUIRE(cudaMemcpy(cu_d, cu.data(), sizeof(int) * cu.size(), cudaMemcpyHostToDevice) == cudaSuccess &&
          cudaMemcpy(lens_d, lens, sizeof(lens), cudaMemcpyHostToDevice) == cudaSuccess &&
          cudaMemcpy(table_d, table.data(), sizeof(int) * table.size(), cudaMemcpyHostToDevice) == cudaSuccess &&
          cudaMemcpy(prefix_d, prefix_pages.data(), sizeof(int) * prefix_pages.size(), cudaMemcpyHostToDevice) == cudaSuccess);
  cs_kv_batch b{};
  b.tokens = tokens;
  b.seqs = SEQS;
  b.max_q = tokens_each;
  b.table_cols = COLS;
  b.cu_q = cu_d;
  b.kv_lens = lens_d;
  b.page_table = table_d;
  cs_kv_attn_args a{};
  a.q = q;
  a.k_cache = k;
  a.v_cache = v;
  a.out = out;
  a.lse = lse;
  auto call = [&] { return prefix ? cs_kv_attention_shared(plan, &b, prefix_d, prefix, &a, nullptr) : cs_kv_attention(plan, &b, &a, nullptr); };
  REQUIRE(cudaDeviceSynchronize() == cudaSuccess);
  const auto t0 = std::chrono::steady_clock::now();
  REQUIRE(call() == CS_OK);
  REQUIRE(cudaDeviceSynchronize() == cudaSuccess);
  REQUIRE(std::chrono::duration<double>(std::chrono::steady_clock::now() - t0).count() < 1.0);
  REQUIRE(cs_kv_status(plan) == CS_ERR_WATCHDOG);
  REQUIRE(call() == CS_ERR_NEEDS_RESET);
  std::vector<unsigned char> got(rows);
  REQUIRE(cudaMemcpy(got.data(), out, rows, cudaMemcpyDeviceToHost) == cudaSuccess);
  for (unsigned char x : got) REQUIRE(x == 0x47);
  REQUIRE(cs_kv_reset(plan) == CS_OK && cs_kv_status(plan) == CS_OK);
  REQUIRE(cs_kv_destroy(plan) == CS_OK);
  for (void* x : {q, out, k, v, static_cast<void*>(lse), static_cast<void*>(cu_d), static_cast<void*>(lens_d),
                  static_cast<void*>(table_d), static_cast<void*>(prefix_d)})
    REQUIRE(cudaFree(x) == cudaSuccess);
  return 0;
}

int main() {
  for (int dtype : {CS_F16, CS_BF16})
    for (int head_dim : {64, 128})
      for (int tokens : {1, 4, 200})
        for (int form = 0; form < 3; ++form)  // plain, behind a prefix, under a window
          if (run(dtype, head_dim, tokens, form == 1 ? 500 : 0, form == 2 ? 700 : 0)) {
            printf("dtype %d, %d dimensions, %d tokens, form %d\n", dtype, head_dim, tokens, form);
            return 1;
          }
  printf("ok\n");
  return 0;
}
