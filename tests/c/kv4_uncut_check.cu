// Runs on the host: which items of few rows stay whole.  However unequal a batch's sequences are, no CTA walks more
// than a short item's tiles beyond an equal range.  Prints "ok" and exits 0.
#include <random>
#include <vector>

#include "kv_host.cuh"

#include "../../consumer_gemm_chain_gb300/csrc/cs_kv4.cu"

struct Case {
  cs_kv_s plan;
  int seqs, keys;
  cskv::AttnP k{};
  Kernels use;
  bool uncut;
  Case(int dim, int heads, int kv_heads, int layout, int seqs, int keys, int window = 0, int sinks = 0, int sms = 152) : seqs(seqs), keys(keys) {
    cs_kv_desc_init(&plan.d);
    plan.d.dtype = CS_BF16;
    plan.d.head_dim = dim;
    plan.d.heads = heads;
    plan.d.kv_heads = kv_heads;
    plan.d.cache_layout = layout;
    plan.d.max_tokens = plan.d.max_seqs = seqs;
    plan.d.window = window;
    plan.d.sinks = sinks;
    plan.num_sms = sms;
    const cs_kv_batch b{seqs, seqs, 1, (keys + 15) / 16, nullptr, nullptr, nullptr};
    k.b = device_batch(&plan, &b);
    const int rows = rows_of(k, 1);
    use = kernels(&plan, rows);
    k.c.window = window;
    k.c.sinks = sinks;
    k.c.item_cost = 1;
    k.c.per_item = cskv::ROWS / k.b.group;
    k.c.shift = use.rows_shift;
    uncut = rows_uncut(k, use, plan.d);
  }
};

int main() {
  // batches whose number of items is that of the CTAs, or nearly: long tables are cut
  for (int seqs : {56, 57, 113, 114, 171, 228})
    for (int keys : {700, 1100, 2000, 32000}) REQUIRE(!Case(128, 32, 8, CS_KV_TOKEN, seqs, keys).uncut);
  REQUIRE(!Case(128, 12, 12, CS_KV_TOKEN, 38, 32000).uncut);
  REQUIRE(!Case(64, 40, 8, CS_KV_HEAD, 76, 9000).uncut);
  REQUIRE(!Case(64, 40, 8, CS_KV_HEAD, 76, 9000, 1024, 4).uncut);
  // short ones stay whole where that loads the CTAs evenly enough, and only there
  REQUIRE(Case(128, 32, 8, CS_KV_TOKEN, 57, 500).uncut);
  REQUIRE(Case(128, 32, 8, CS_KV_TOKEN, 6, 250).uncut);
  REQUIRE(Case(64, 40, 8, CS_KV_HEAD, 76, 500).uncut);
  REQUIRE(Case(128, 32, 8, CS_KV_TOKEN, 50, 9000, 100, 0).uncut);
  REQUIRE(!Case(128, 32, 8, CS_KV_TOKEN, 60, 500).uncut);
  // a prefix's items are cut
  Case prefix(128, 32, 8, CS_KV_TOKEN, 57, 500);
  prefix.k.c.flat = 1;
  REQUIRE(!rows_uncut(prefix.k, prefix.use, prefix.plan.d));
  // the longest CTA, item after item as the kernel takes them (that of an item's middle), against an equal range
  std::mt19937 r(1);
  auto draw = [&](int a, int b) { return a + static_cast<int>(r() % static_cast<unsigned>(b - a + 1)); };
  int whole = 0;
  for (int it = 0; it < 20000; ++it) {
    const int kv_heads = draw(1, 12), most = draw(0, 3) ? draw(1, 600) : draw(1, 40000);
    const bool windowed = draw(0, 3) == 0;
    Case c(draw(0, 1) ? 128 : 64, kv_heads * draw(1, 16), kv_heads, draw(0, 1), draw(1, 300), most, windowed ? draw(1, 600) : 0,
           windowed ? draw(0, 200) : 0, draw(0, 3) ? 152 : draw(1, 200));
    if (!c.uncut) continue;
    ++whole;
    std::vector<unsigned> units;  // of a head's items
    for (int b = 0; b < c.seqs; ++b) {
      const cskv::Seq s{b, 1, draw(0, 2) ? draw(1, most) : most};
      units.push_back(cskv::item_tiles(c.k.c, s, 0) + c.k.c.item_cost);
    }
    const int heads = c.use.head_ctas ? 1 : kv_heads, ctas = c.use.head_ctas ? c.use.head_ctas : c.use.rows_grid;
    unsigned long long total = 0;
    for (unsigned u : units) total += u * heads;
    const unsigned long long quota = std::max<unsigned long long>((total + ctas - 1) / ctas, c.use.least);
    std::vector<unsigned long long> load(ctas);
    unsigned long long x = 0;
    for (int h = 0; h < heads; ++h)
      for (unsigned u : units) {
        load[(2 * x + u - 1) / 2 / quota] += u;
        x += u;
      }
    REQUIRE(*std::max_element(load.begin(), load.end()) <= quota + c.use.uncut + c.k.c.item_cost);
  }
  REQUIRE(whole > 1000);
  printf("ok\n");
}
