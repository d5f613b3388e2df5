// Attention over the paged key/value cache (include/cs_kv.h) on the tensor cores.
//
// Mathematics.  For one sequence and key head, the rows of a product are the
// (token, query head) pairs that read that head: S = Q K^T, running row maximum
// and sum, P = 2^(c S - max), O += P V, and O / sum at the end.
//
// Work.  An item is 2 x 128 such rows (whole tokens) of one sequence and key head; it
// needs one or more tiles of 128 keys.  The tiles of all items, laid end to end, are
// cut into one equal range per CTA (one CTA per SM): long and short sequences, one or
// many, prompts and single tokens all load the SMs alike, without a launch per
// kind.  Items cut by a range's border leave their state (O, max, sum) in the
// workspace, and the last CTA to arrive joins the pieces in their order, so the
// result does not depend on who is last.
#pragma once
#include "cs_kv_append.cuh"

namespace cskv {

// ---------------------------------------------------------------- which tiles
struct Cut {
  int per_tile;   // tokens of a 128-row tile: 128 / group, rounded down
  int per_item;   // tokens of an item: two tiles
  int window, sinks;
  int flat;       // every row sees keys 0 .. flat_len - 1 of one common table (a shared prefix)
  int flat_len;
};

constexpr int KT = 128;  // keys per tile

struct Seq {
  int t0, n, m;
};

// Sequence b of the batch, or with `flat` all tokens of the batch over the prefix.
__device__ __forceinline__ bool load_seq(const Batch& B, const Cut& C, int b, Seq& s) {
  if (!C.flat) return sequence(B, b, s.t0, s.n, s.m);
  s.t0 = __ldg(B.cu_q);
  const int t1 = __ldg(B.cu_q + B.seqs);
  s.n = t1 - s.t0;
  s.m = C.flat_len;
  if (s.t0 >= 0 && t1 >= s.t0 && t1 <= B.tokens) return true;
  record(B.ctrl, ERR_INVALID, WHAT_LENGTHS, static_cast<uint32_t>(B.seqs - 1));
  return false;
}

// First key of the window of the item's first token (0 without a window), and the
// end of the keys that its last token sees.
__device__ __forceinline__ int item_lo(const Cut& C, const Seq& s, int item) {
  return C.window > 0 ? max(0, s.m - s.n + item * C.per_item - C.window + 1) : 0;
}
__device__ __forceinline__ int item_hi(const Cut& C, const Seq& s, int item) {
  return C.flat ? s.m : max(0, s.m - s.n + min(s.n, (item + 1) * C.per_item));
}
// Tiles of the sinks before the window's first tile.
__device__ __forceinline__ int sink_tiles(const Cut& C, int lo) { return min((C.sinks + KT - 1) / KT, lo / KT); }
// Key tiles of an item; at least one, so that rows without keys are written too.
__device__ __forceinline__ int item_tiles(const Cut& C, const Seq& s, int item) {
  const int lo = item_lo(C, s, item), hi = item_hi(C, s, item);
  return (max(1, hi) + KT - 1) / KT - lo / KT + sink_tiles(C, lo);
}
__device__ __forceinline__ int items_of(const Cut& C, const Seq& s) { return (s.n + C.per_item - 1) / C.per_item; }

// sum over i < n of floor((a i + b) / m), a, b >= 0 (the Euclid-like recurrence for
// lattice points under a line)
__device__ __forceinline__ unsigned long long floor_sum(unsigned n, unsigned m, unsigned a, unsigned b) {
  unsigned long long ans = 0;
  while (n > 0) {
    if (a >= m) {
      ans += static_cast<unsigned long long>(n) * (n - 1) / 2 * (a / m);
      a %= m;
    }
    if (b >= m) {
      ans += static_cast<unsigned long long>(n) * (b / m);
      b %= m;
    }
    const unsigned long long y = static_cast<unsigned long long>(a) * n + b;
    if (y < m) break;
    n = static_cast<unsigned>(y / m);
    b = static_cast<unsigned>(y % m);
    const unsigned t = m;
    m = a;
    a = t;
  }
  return ans;
}

// Key tiles of the first k items of a sequence (of one key head).
__device__ __forceinline__ unsigned long long tiles_before(const Cut& C, const Seq& s, int k) {
  if (k == 0) return 0;
  if (C.flat) return static_cast<unsigned long long>(k) * static_cast<unsigned>(item_tiles(C, s, 0));
  const int full = min(k, items_of(C, s) - 1);  // the last item may hold fewer tokens
  unsigned long long sum = 0;
  if (k > full) sum += item_tiles(C, s, full);
  if (full > 0) {
    const int base = s.m - s.n, P = C.per_item;
    // sum of ceil(max(1, base + (i + 1) P) / KT)
    const int early = base < 0 ? min(full, -base / P) : 0;
    sum += early + floor_sum(full - early, KT, P, base + (early + 1) * P + KT - 1);
    if (C.window > 0) {
      // minus what lies between the sinks' tiles and the window's first tile
      const int b2 = base - C.window + 1 - (C.sinks + KT - 1) / KT * KT;
      const int k2 = b2 >= 0 ? 0 : (-b2 + P - 1) / P;
      if (full > k2) sum -= floor_sum(full - k2, KT, P, b2 + k2 * P);
    }
  }
  return sum;
}

// A piece of work of one CTA: key tiles [k0, k1) of an item.
struct Seg {
  Seq s;
  int b, kvh, item, k0, k1, tiles, lo, hi, sinks;  // sinks: its leading sink tiles
  unsigned long long x;                            // the item's first tile in the order of all
  __device__ __forceinline__ bool whole() const { return k0 == 0 && k1 == tiles; }
  // first key of the k-th tile
  __device__ __forceinline__ int key0(int k) const { return (k < sinks ? k : lo / KT + k - sinks) * KT; }
};

// Where a CTA's range begins and ends; every warp role walks it by itself.
struct Range {
  unsigned long long x0, x1, total, rem;
  int ctas;
  int b, kvh, item, off;
  __device__ __forceinline__ unsigned long long begin_of(unsigned c) const { return total * c / ctas; }
  // the CTA whose range holds tile x
  __device__ __forceinline__ unsigned cta_of(unsigned long long x) const {
    return static_cast<unsigned>(((x + 1) * ctas + total - 1) / total - 1);
  }
};

struct Walk {
  unsigned long long x, x1;
  int b, kvh, item, off, items;
  Seq s;
  __device__ __forceinline__ Walk(const Batch& B, const Cut& C, const Range& r)
      : x(r.x0), x1(r.x1), b(r.b), kvh(r.kvh), item(r.item), off(r.off), items(0) {
    if (x < x1 && load_seq(B, C, b, s)) items = items_of(C, s);
  }
  __device__ __forceinline__ bool next(const Batch& B, const Cut& C, Seg& g) {
    if (x >= x1) return false;
    if (item == items) {
      item = 0;
      if (++kvh == B.kv_heads) {
        kvh = 0;
        const int seqs = C.flat ? 1 : B.seqs;
        do {
          if (++b >= seqs) return false;
          items = load_seq(B, C, b, s) ? items_of(C, s) : 0;
        } while (items == 0);
      }
    }
    g.s = s;
    g.b = b;
    g.kvh = kvh;
    g.item = item;
    g.lo = item_lo(C, s, item);
    g.hi = item_hi(C, s, item);
    g.sinks = sink_tiles(C, g.lo);
    g.tiles = item_tiles(C, s, item);
    g.k0 = off;
    g.x = x - off;
    const unsigned long long left = x1 - x;
    g.k1 = static_cast<unsigned long long>(g.tiles - off) <= left ? g.tiles : off + static_cast<int>(left);
    x += g.k1 - g.k0;
    off = 0;
    ++item;
    return true;
  }
};

// Every thread of the block: this CTA's range into *r (shared memory).
template <int THREADS>
__device__ __forceinline__ void find_range(const Batch& B, const Cut& C, Range* r, unsigned long long* scratch) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int seqs = C.flat ? 1 : B.seqs;
  const int per = (seqs + THREADS - 1) / THREADS;
  const int b0 = min(tid * per, seqs), b1 = min(b0 + per, seqs);
  unsigned long long mine = 0;
  Seq s;
  for (int b = b0; b < b1; ++b)
    if (load_seq(B, C, b, s)) mine += tiles_before(C, s, items_of(C, s));
  unsigned long long incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const unsigned long long o = __shfl_up_sync(0xFFFFFFFFu, incl, d);
    if (lane >= d) incl += o;
  }
  if (lane == 31) scratch[warp] = incl;
  __syncthreads();
  unsigned long long before = 0, total = 0;
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) before += scratch[w];
    total += scratch[w];
  }
  incl += before;
  total *= B.kv_heads;
  const unsigned ctas = total < gridDim.x ? static_cast<unsigned>(total) : gridDim.x;
  const bool work = blockIdx.x < ctas;
  const unsigned long long x0 = work ? total * blockIdx.x / ctas : 0, x1 = work ? total * (blockIdx.x + 1) / ctas : 0;
  if (tid == 0) {
    r->x0 = x0;
    r->x1 = x1;
    r->total = total;
    r->ctas = static_cast<int>(ctas);
    r->b = r->kvh = r->item = r->off = 0;
  }
  __syncthreads();
  unsigned long long at = (incl - mine) * B.kv_heads;
  if (work && at <= x0 && x0 < incl * B.kv_heads) {
    for (int b = b0; b < b1; ++b) {
      if (!load_seq(B, C, b, s)) continue;
      const unsigned long long c = tiles_before(C, s, items_of(C, s));
      if (x0 < at + c * B.kv_heads) {
        r->b = b;
        r->kvh = static_cast<int>((x0 - at) / c);
        r->rem = (x0 - at) % c;
        break;
      }
      at += c * B.kv_heads;
    }
  }
  __syncthreads();
  if (warp == 0 && work) {
    // the item that holds tile `rem` of its sequence and head: 32 trials at a time
    if (load_seq(B, C, r->b, s)) {
      const unsigned long long rem = r->rem;
      int a = 0, e = items_of(C, s);  // tiles_before(a) <= rem < tiles_before(e)
      while (e - a > 1) {
        const int step = (e - a + 31) / 32;
        const int k = a + lane * step;
        const bool in = k < e && tiles_before(C, s, k) <= rem;
        const int last = 31 - __clz(__ballot_sync(0xFFFFFFFFu, in));
        a += last * step;
        e = min(e, a + step);
      }
      const int off = static_cast<int>(rem - tiles_before(C, s, a));
      __syncwarp();
      if (lane == 0) {
        r->item = a;
        r->off = off;
      }
    }
  }
  __syncthreads();
}

// ---------------------------------------------------------------- the kernel
struct AttnP {
  CUtensorMap q, k, v;
  Batch b;
  Cut c;
  const int* pages;       // flat: the prefix's pages
  void* out;
  float* lse;
  long long out_stride;   // elements
  float scale_log2;       // scale * log2(e): exponents in base 2
  float* part;            // pieces: [CTA][first, last][tile][D / 4 + 1][128 rows] float4
  uint32_t* arrivals;     // [CTA][tile] pieces of the item that starts there and ends elsewhere
  float* flat_o;          // [tokens][heads][D], [tokens][heads]: a prefix's normalised output and
  float* flat_lse;        // base-2 log-sum-exp; written with c.flat, else joined in if not null
  int head_groups;        // 8-slot groups between heads (HEAD layout), 0: heads are a dimension of their own
  unsigned long long wait_ns;
};

constexpr int ATTN_THREADS = 320;  // two softmax warpgroups, the TMA warp, the MMA warp
constexpr uint32_t COL_S = 0, COL_O = 256;
constexpr float RAISE_LOG2 = 8.0f;  // the reference maximum follows a row's when it is exceeded by more than 2^8

template <int D>
struct AttnShape {
  static constexpr int HALVES = D / 64;
  static constexpr int TILE = KT * D * 2;              // bytes of a 128-row tile of Q, K or V
  static constexpr int SLOTS = D == 128 ? 5 : 10;      // ring of K and V tiles: 160 KB in flight
  static constexpr int SMEM = 2 * TILE + SLOTS * TILE + 1024 + 1024;
};

template <int SLOTS>
struct AttnCtl {
  uint64_t full[SLOTS], empty[SLOTS];
  uint64_t q_full, q_empty, s_full[2], p_full[2], o_full[2], stored[2], counted[2], drained;
  unsigned long long scratch[ATTN_THREADS / 32];
  Range range;
  uint32_t tmem;
  volatile int abort;
  volatile int last[2];
  int loads, q_loads;  // tiles and queries whose copies were issued
};

__device__ __forceinline__ void tma_5d(void* dst, const CUtensorMap* map, int x, int c1, int c2, int c3, int c4,
                                       uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, "
      "%6}], [%7];" ::"r"(cs::smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(cs::smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tma_3d(void* dst, const CUtensorMap* map, int x, int c1, int c2, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          cs::smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(c1), "r"(c2), "r"(cs::smem_u32(bar))
      : "memory");
}
// D(tmem) (+)= A(tmem) * B(smem): the 16-bit A operand holds two K values per 32-bit column.
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(acc)
      : "memory");
}

// Bounded wait; false when it ran out, here or in another role.
template <typename Ctl>
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, Ctl* sc, const AttnP& p, uint32_t where) {
  if (cs::mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = cs::globaltimer();
  for (uint32_t i = 1;; ++i) {
    if (cs::mbar_try_wait(bar, parity)) return true;
    if (sc->abort) return false;
    if ((i & 63u) == 0u && cs::globaltimer() - t0 > p.wait_ns) {
      record(p.b.ctrl, ERR_WATCHDOG, WHAT_WAIT, where);
      sc->abort = 1;
      return false;
    }
  }
}

// The same for a whole warp, which goes on or gives up together.
template <typename Ctl>
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, Ctl* sc, const AttnP& p, uint32_t where) {
  const bool ok = wait(bar, parity, sc, p, where);
  return __all_sync(0xFFFFFFFFu, ok);
}

// After a wait that ran out, one thread: this CTA's copies and MMAs in flight
// come to rest (again with a limit) before its memory is given back.
template <int SLOTS>
__device__ void come_to_rest(AttnCtl<SLOTS>* sc, const AttnP& p) {
  const uint64_t t0 = cs::globaltimer();
  auto settle = [&](uint64_t* bar, uint32_t parity) {
    while (!cs::mbar_try_wait(bar, parity) && cs::globaltimer() - t0 < p.wait_ns) {
    }
  };
  for (int i = 0; i < SLOTS; ++i) {
    const int n = (sc->loads - i + SLOTS - 1) / SLOTS;  // loads into slot i
    if (n > 0) settle(&sc->full[i], (n - 1) & 1);
  }
  if (sc->q_loads > 0) settle(&sc->q_full, (sc->q_loads - 1) & 1);
  settle(&sc->drained, 0);
}

// A position in the ring: slot and the parity of its full barrier's current phase.
template <int SLOTS>
struct Ring {
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++slot == SLOTS) slot = 0, phase ^= 1u;
  }
};

// TMA warp: the item's queries, then K and V of each key tile, page by page.  A
// tile lies in shared memory as [8-key group][64-dimension half][8 x 128 bytes],
// so that one box brings a page's slots of a head with all dimensions.
template <int D>
__device__ bool load_role(const AttnP& p, AttnCtl<AttnShape<D>::SLOTS>* sc, uint8_t* qbuf, uint8_t* ring) {
  using Sh = AttnShape<D>;
  const Batch& B = p.b;
  const int lane = threadIdx.x & 31;
  const int pages_per_tile = KT >> B.page_shift, groups = B.page_size >> 3;
  Walk walk(B, p.c, sc->range);
  Seg g;
  Ring<Sh::SLOTS> rp;
  uint32_t q_phase = 1;
  while (walk.next(B, p.c, g)) {
    const int* table = p.c.flat ? p.pages : B.table + static_cast<long long>(g.b) * B.table_cols;
    const bool two = g.s.n - g.item * p.c.per_item > p.c.per_tile;
    if (!wait_warp(&sc->q_empty, q_phase, sc, p, 1)) return false;
    q_phase ^= 1u;
    if (lane == 0) {
      const int tok = g.s.t0 + g.item * p.c.per_item;
      const uint32_t bytes = static_cast<uint32_t>(p.c.per_tile) * B.group * D * 2;
      cs::mbar_arrive_expect_tx(&sc->q_full, two ? 2 * bytes : bytes);
      for (int w = 0; w < (two ? 2 : 1); ++w)
        for (int h = 0; h < Sh::HALVES; ++h)
          tma_3d(qbuf + w * Sh::TILE + h * (KT * 128), &p.q, h * 64, g.kvh * B.group, tok + w * p.c.per_tile, &sc->q_full);
      ++sc->q_loads;
    }
    // the page that this lane brings of tile k, -1: none of its keys is seen
    auto page_of = [&](int k) {
      if (k >= g.k1 || lane >= pages_per_tile) return -1;
      const int j0 = g.key0(k) + (lane << B.page_shift), j1 = j0 + B.page_size;
      if (j0 >= g.hi || (j1 <= g.lo && j0 >= p.c.sinks)) return -1;
      const int page = __ldg(table + (j0 >> B.page_shift));
      if (page >= 0 && page < B.num_pages) return page;
      record(B.ctrl, ERR_INVALID, WHAT_PAGE, p.c.flat ? 0xFFFFFFFFu : static_cast<uint32_t>(g.b));
      return -1;
    };
    int page = page_of(g.k0);
    for (int k = g.k0; k < g.k1; ++k) {
      const uint32_t boxes = __popc(__ballot_sync(0xFFFFFFFFu, page >= 0));
      const int after = page_of(k + 1);
      const int c3 = p.head_groups ? 0 : g.kvh;
      const int c4 = page * (p.head_groups ? p.head_groups * B.kv_heads : groups) + g.kvh * p.head_groups;
      for (int half = 0; half < 2; ++half) {  // K, then V
        if (!wait_warp(&sc->empty[rp.slot], rp.phase ^ 1u, sc, p, 2)) return false;
        if (lane == 0) {
          cs::mbar_arrive_expect_tx(&sc->full[rp.slot], boxes * B.page_size * D * 2);
          ++sc->loads;
        }
        __syncwarp();
        if (page >= 0)
          tma_5d(ring + rp.slot * Sh::TILE + lane * (B.page_size * D * 2), half ? &p.v : &p.k, 0, 0, 0, c3, c4,
                 &sc->full[rp.slot]);
        rp.next();
      }
      page = after;
    }
  }
  return true;
}

// One thread: S of the two row tiles in turn, each P V between them, so that one
// tile's softmax runs while the tensor core works for the other.  P takes the
// place of the first half of S; MMAs execute in the order of their issue.
template <int D>
__device__ bool mma_role(const AttnP& p, AttnCtl<AttnShape<D>::SLOTS>* sc, uint8_t* qbuf, uint8_t* ring, int bf16) {
  using Sh = AttnShape<D>;
  const uint32_t idesc_s = cs::make_idesc_f16(bf16, 0, 128, KT);
  const uint32_t idesc_o = cs::make_idesc_f16(bf16, 1, 128, D);
  Walk walk(p.b, p.c, sc->range);
  Seg g;
  Ring<Sh::SLOTS> rk, rv;
  rv.next();
  uint32_t q_phase = 0, p_phase[2] = {0, 0};
  const uint32_t qa = cs::smem_u32(qbuf), ra = cs::smem_u32(ring);
  auto scores = [&](int w) {
    const uint64_t a = cs::smem_desc_sw128(qa + w * Sh::TILE, 16, 1024);
    const uint64_t b = cs::smem_desc_sw128(ra + rk.slot * Sh::TILE, 16, Sh::HALVES * 1024);
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk)
      cs::tc_mma_f16<1>(sc->tmem + COL_S + w * 128, a + (kk >> 2) * (KT * 128 >> 4) + (kk & 3) * 2,
                        b + (kk >> 2) * (1024 >> 4) + (kk & 3) * 2, idesc_s, kk != 0);
    cs::tc_commit<1>(&sc->s_full[w]);
  };
  auto values = [&](int w, const Ring<Sh::SLOTS>& r, bool acc) {
    if (!wait(&sc->p_full[w], p_phase[w], sc, p, 3)) return false;
    p_phase[w] ^= 1u;
    if (!wait(&sc->full[r.slot], r.phase, sc, p, 4)) return false;
    cs::tc_fence_after();
    const uint64_t b = cs::smem_desc_sw128(ra + r.slot * Sh::TILE, 1024, Sh::HALVES * 1024);
#pragma unroll
    for (int kk = 0; kk < KT / 16; ++kk)
      mma_ts(sc->tmem + COL_O + w * D, sc->tmem + COL_S + w * 128 + kk * 8, b + kk * (Sh::HALVES * 2048 >> 4), idesc_o,
             acc || kk != 0);
    return true;
  };
  while (walk.next(p.b, p.c, g)) {
    const bool two = g.s.n - g.item * p.c.per_item > p.c.per_tile;
    if (!wait(&sc->q_full, q_phase, sc, p, 5)) return false;
    q_phase ^= 1u;
    Ring<Sh::SLOTS> prev;  // the V tile of the previous key tile
    for (int k = g.k0; k < g.k1; ++k) {
      if (!wait(&sc->full[rk.slot], rk.phase, sc, p, 6)) return false;
      cs::tc_fence_after();
      scores(0);
      if (two) {
        if (k > g.k0) {
          if (!values(1, prev, k - 1 > g.k0)) return false;
          cs::tc_commit<1>(&sc->empty[prev.slot]);
        }
        scores(1);
      }
      cs::tc_commit<1>(&sc->empty[rk.slot]);
      if (k + 1 == g.k1) cs::tc_commit<1>(&sc->q_empty);
      rk.next(), rk.next();
      if (!values(0, rv, k > g.k0)) return false;
      if (!two) cs::tc_commit<1>(&sc->empty[rv.slot]);
      if (k + 1 == g.k1) cs::tc_commit<1>(&sc->o_full[0]);
      prev = rv;
      rv.next(), rv.next();
    }
    if (two) {
      if (!values(1, prev, g.k1 - 1 > g.k0)) return false;
      cs::tc_commit<1>(&sc->empty[prev.slot]);
      cs::tc_commit<1>(&sc->o_full[1]);
    }
  }
  return true;
}

// Warpgroup w: the softmax of row tile w, one row per thread, and its output.
template <typename T, int D>
__device__ bool softmax_role(const AttnP& p, AttnCtl<AttnShape<D>::SLOTS>* sc, uint8_t* ring, int w) {
  using Sh = AttnShape<D>;
  const Batch& B = p.b;
  const int r = threadIdx.x & 127;
  const uint32_t lanes = static_cast<uint32_t>(r & ~31) << 16;
  const uint32_t s_tm = sc->tmem + lanes + COL_S + w * 128, o_tm = sc->tmem + lanes + COL_O + w * D;
  const int row_tok = r / B.group, row_head = r - row_tok * B.group;
  Walk walk(B, p.c, sc->range);
  Seg g;
  Ring<Sh::SLOTS> rv;
  rv.next();
  uint32_t s_phase = 0, o_phase = 0, j_phase = 0;
  while (walk.next(B, p.c, g)) {
    const int first = g.item * p.c.per_item + w * p.c.per_tile;  // the tile's first token
    if (first >= g.s.n) {  // the item has one tile
      for (int k = g.k0; k < g.k1; ++k) rv.next(), rv.next();
      continue;
    }
    const int base = g.s.m - g.s.n;
    const int tok = first + row_tok;
    const bool live = row_tok < p.c.per_tile && tok < g.s.n;
    const int end = p.c.flat ? g.s.m : live ? base + tok + 1 : 0;  // keys [.., end) are seen
    const int lo = p.c.window > 0 ? max(0, base + tok + 1 - p.c.window) : 0;
    // keys below `some` and from `all_lo` on are seen by every live row
    const int some = p.c.flat ? g.s.m : base + first + 1;
    const int all_lo = p.c.window > 0 ? max(0, base + first + p.c.per_tile - p.c.window) : 0;
    float m_ref = -INFINITY, l = 0.0f;
    for (int k = g.k0; k < g.k1; ++k) {
      const int j0 = g.key0(k);
      if (!wait_warp(&sc->s_full[w], s_phase, sc, p, 7 + w)) return false;
      s_phase ^= 1u;
      cs::tc_fence_after();
      uint32_t v[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c) cs::tmem_ld32(s_tm + c * 32, v[c]);
      cs::tc_wait_ld();
#pragma unroll
      for (int c = 0; c < 4; ++c) cs::tc_wait_ld_regs(v[c]);
      if (!(j0 + KT <= some && (j0 >= all_lo || j0 + KT <= p.c.sinks))) {
        const int rel_end = end - j0, rel_lo = lo - j0, rel_sinks = p.c.sinks - j0;
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int t = 0; t < 32; ++t) {
            const int j = c * 32 + t;
            if (j >= rel_end || (j < rel_lo && j >= rel_sinks)) v[c][t] = 0xFF800000u;  // -inf
          }
      }
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int t = 0; t < 32; ++t) mx[t & 3] = fmaxf(mx[t & 3], __uint_as_float(v[c][t]));
      const float m_tile = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.scale_log2;
      // P is taken against a reference that is raised only when a row's maximum
      // exceeds it by more than 2^8 (so P <= 2^8, and rounding to the dtype is as
      // good as at 1); then O and l are scaled down first
      const bool raise = m_tile > m_ref + RAISE_LOG2 || (m_ref == -INFINITY && m_tile > -INFINITY);
      const float m_new = raise ? m_tile : m_ref;
      if (k > g.k0 && __any_sync(0xFFFFFFFFu, raise)) {
        // S of this tile was issued after P V of the one before: O is complete
        const float f = raise ? cs::ex2_approx(m_ref - m_new) : 1.0f;
        l *= f;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          cs::tmem_ld32(o_tm + c * 32, o);
          cs::tc_wait_ld();
          cs::tc_wait_ld_regs(o);
#pragma unroll
          for (int t = 0; t < 32; ++t) o[t] = __float_as_uint(__uint_as_float(o[t]) * f);
          cs::tmem_st32(o_tm + c * 32, o);
        }
      }
      m_ref = m_new;
      const float sub = m_ref == -INFINITY ? 0.0f : -m_ref;
      float ls[2] = {0.0f, 0.0f};
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t pk[32];
#pragma unroll
        for (int t = 0; t < 64; t += 2) {
          const float p0 = cs::ex2_approx(fmaf(__uint_as_float(v[2 * c + (t >> 5)][t & 31]), p.scale_log2, sub));
          const float p1 = cs::ex2_approx(fmaf(__uint_as_float(v[2 * c + (t >> 5)][(t & 31) + 1]), p.scale_log2, sub));
          ls[0] += p0;
          ls[1] += p1;
          pk[t >> 1] = Pair<T>::put(p0, p1);
        }
        cs::tmem_st32(s_tm + c * 32, pk);
      }
      l += ls[0] + ls[1];
      // values of keys that no row of the item sees may hold anything: zeros in
      // their place (the first tile's P V is issued first, so w = 0 does it for both)
      if (w == 0 && (j0 + KT > g.hi || (j0 < g.lo && j0 + KT > p.c.sinks))) {
        if (!wait_warp(&sc->full[rv.slot], rv.phase, sc, p, 9)) return false;
        const int j = j0 + r;
        if (j >= g.hi || (j < g.lo && j >= p.c.sinks)) {
          uint8_t* row = ring + rv.slot * Sh::TILE + (r >> 3) * (Sh::HALVES * 1024) + (r & 7) * 128;
          for (int h = 0; h < Sh::HALVES; ++h)
#pragma unroll
            for (int c = 0; c < 8; ++c) *reinterpret_cast<uint4*>(row + h * 1024 + c * 16) = make_uint4(0, 0, 0, 0);
        }
        cs::fence_proxy_async_shared();
      }
      cs::tc_wait_st();
      cs::tc_fence_before();
      cs::mbar_arrive(&sc->p_full[w]);
      rv.next(), rv.next();
    }
    if (!wait_warp(&sc->o_full[w], o_phase, sc, p, 10 + w)) return false;
    o_phase ^= 1u;
    cs::tc_fence_after();
    // this thread's row of O, against m_ref
    float acc[D];
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
      uint32_t o[32];
      cs::tmem_ld32(o_tm + c * 32, o);
      cs::tc_wait_ld();
      cs::tc_wait_ld_regs(o);
#pragma unroll
      for (int t = 0; t < 32; ++t) acc[c * 32 + t] = __uint_as_float(o[t]);
    }
    cs::tc_fence_before();
    if (!g.whole()) {
      constexpr size_t PIECE = static_cast<size_t>(D / 4 + 1) * 128;  // float4s
      float4* part = reinterpret_cast<float4*>(p.part);
      auto piece = [&](unsigned cta, int last) { return part + ((static_cast<size_t>(cta) * 2 + last) * 2 + w) * PIECE + r; };
      float4* mine = piece(blockIdx.x, sc->range.x0 < g.x);
#pragma unroll
      for (int t = 0; t < D / 4; ++t) mine[t * 128] = make_float4(acc[4 * t], acc[4 * t + 1], acc[4 * t + 2], acc[4 * t + 3]);
      mine[D / 4 * 128] = make_float4(m_ref, l, 0.0f, 0.0f);
      const unsigned c0 = sc->range.cta_of(g.x), c1 = sc->range.cta_of(g.x + g.tiles - 1);
      // every thread's stores come before the one arrival at gpu scope; the other
      // pieces are read after it
      cs::mbar_arrive(&sc->stored[w]);
      if (r < 32) {
        if (!wait_warp(&sc->stored[w], j_phase, sc, p, 12)) return false;
        if (r == 0) {
          uint32_t* ctr = p.arrivals + c0 * 2 + w;
          const uint32_t old = cs::atom_add_acq_rel_gpu(ctr, 1u);
          sc->last[w] = old == c1 - c0;
          if (old == c1 - c0) *ctr = 0u;  // for the next call
          cs::mbar_arrive(&sc->counted[w]);
        }
        __syncwarp();
      }
      if (!wait_warp(&sc->counted[w], j_phase, sc, p, 13)) return false;
      j_phase ^= 1u;
      const bool last = sc->last[w] != 0;
      if (!last) continue;
      m_ref = -INFINITY;
      for (unsigned c = c0; c <= c1; ++c)
        m_ref = fmaxf(m_ref, __ldcg(piece(c, sc->range.begin_of(c) < g.x) + D / 4 * 128).x);
      const float sub = m_ref == -INFINITY ? 0.0f : m_ref;
      l = 0.0f;
#pragma unroll
      for (int t = 0; t < D; ++t) acc[t] = 0.0f;
      for (unsigned c = c0; c <= c1; ++c) {
        const float4* src = piece(c, sc->range.begin_of(c) < g.x);
        const float4 ml = __ldcg(src + D / 4 * 128);
        const float f = cs::ex2_approx(ml.x - sub);
        l = fmaf(ml.y, f, l);
#pragma unroll
        for (int t = 0; t < D / 4; ++t) {
          const float4 x = __ldcg(src + t * 128);
          acc[4 * t] = fmaf(x.x, f, acc[4 * t]);
          acc[4 * t + 1] = fmaf(x.y, f, acc[4 * t + 1]);
          acc[4 * t + 2] = fmaf(x.z, f, acc[4 * t + 2]);
          acc[4 * t + 3] = fmaf(x.w, f, acc[4 * t + 3]);
        }
      }
    }
    if (!live) continue;
    const long long row = static_cast<long long>(g.s.t0 + tok) * B.heads + g.kvh * B.group + row_head;
    if (p.c.flat) {
      const float inv = 1.0f / l;
      float4* dst = reinterpret_cast<float4*>(p.flat_o + row * D);
#pragma unroll
      for (int t = 0; t < D / 4; ++t)
        dst[t] = make_float4(acc[4 * t] * inv, acc[4 * t + 1] * inv, acc[4 * t + 2] * inv, acc[4 * t + 3] * inv);
      p.flat_lse[row] = m_ref + log2f(l);
      continue;
    }
    float fold = 0.0f;  // weight of the prefix's output
    const float4* pre = reinterpret_cast<const float4*>(p.flat_o + row * D);
    if (p.flat_o) {
      const float z = p.flat_lse[row];
      const float m_new = fmaxf(m_ref, z);
      const float f = m_ref == -INFINITY ? 0.0f : cs::ex2_approx(m_ref - m_new);
      fold = cs::ex2_approx(z - m_new);
      l = fmaf(l, f, fold);
#pragma unroll
      for (int t = 0; t < D / 4; ++t) {
        const float4 x = pre[t];
        acc[4 * t] = fmaf(acc[4 * t], f, fold * x.x);
        acc[4 * t + 1] = fmaf(acc[4 * t + 1], f, fold * x.y);
        acc[4 * t + 2] = fmaf(acc[4 * t + 2], f, fold * x.z);
        acc[4 * t + 3] = fmaf(acc[4 * t + 3], f, fold * x.w);
      }
      m_ref = m_new;
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(p.out) + (g.s.t0 + tok) * p.out_stride +
                                          (g.kvh * B.group + row_head) * D);
#pragma unroll
    for (int t = 0; t < D / 8; ++t) {
      const float* a = acc + 8 * t;
      dst[t] = make_uint4(Pair<T>::put(a[0] * inv, a[1] * inv), Pair<T>::put(a[2] * inv, a[3] * inv),
                          Pair<T>::put(a[4] * inv, a[5] * inv), Pair<T>::put(a[6] * inv, a[7] * inv));
    }
    if (p.lse) p.lse[row] = l == 0.0f ? -INFINITY : (m_ref + log2f(l)) * 0.6931471805599453f;
  }
  return true;
}

template <typename T, int D>
__global__ void __launch_bounds__(ATTN_THREADS, 1) cs_kv_attn_kernel(const __grid_constant__ AttnP p) {
  using Sh = AttnShape<D>;
  using Ctl = AttnCtl<Sh::SLOTS>;
  static_assert(sizeof(Ctl) <= 1024, "control block");
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* qbuf = smem;
  uint8_t* ring = smem + 2 * Sh::TILE;
  Ctl* sc = reinterpret_cast<Ctl*>(ring + Sh::SLOTS * Sh::TILE);
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int i = 0; i < Sh::SLOTS; ++i) {
      cs::mbar_init(&sc->full[i], 1);
      cs::mbar_init(&sc->empty[i], 1);
    }
    cs::mbar_init(&sc->q_full, 1);
    cs::mbar_init(&sc->q_empty, 1);
    for (int w = 0; w < 2; ++w) {
      cs::mbar_init(&sc->s_full[w], 1);
      cs::mbar_init(&sc->p_full[w], 128);
      cs::mbar_init(&sc->o_full[w], 1);
      cs::mbar_init(&sc->stored[w], 128);
      cs::mbar_init(&sc->counted[w], 1);
    }
    cs::mbar_init(&sc->drained, 1);
    sc->abort = sc->loads = sc->q_loads = 0;
    cs::fence_mbar_init();
    cs::prefetch_tmap(&p.q);
    cs::prefetch_tmap(&p.k);
    cs::prefetch_tmap(&p.v);
  }
  if (warp == 9) {
    cs::tmem_alloc<1>(&sc->tmem, 512);
    cs::tmem_relinquish<1>();
  }
  cs::tc_fence_before();
  __syncthreads();
  cs::tc_fence_after();
  cs::grid_dep_wait();
  cs::grid_dep_launch_dependents();
  find_range<ATTN_THREADS>(p.b, p.c, &sc->range, sc->scratch);
  constexpr int bf16 = sizeof(T) == 2 && !std::is_same<T, __half>::value;
  if (warp < 8)
    softmax_role<T, D>(p, sc, ring, warp >> 2);
  else if (warp == 8)
    load_role<D>(p, sc, qbuf, ring);
  else if ((threadIdx.x & 31) == 0 && !mma_role<D>(p, sc, qbuf, ring, bf16))
    cs::tc_commit<1>(&sc->drained);
  __syncwarp();
  cs::tc_fence_before();
  __syncthreads();
  cs::tc_fence_after();
  if (sc->abort) {
    if (threadIdx.x == 0) come_to_rest(sc, p);
    __syncthreads();
  }
  if (warp == 9) cs::tmem_dealloc<1>(sc->tmem, 512);
}

}  // namespace cskv
