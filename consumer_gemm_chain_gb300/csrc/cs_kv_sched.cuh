// How attention over the paged cache is divided (cs_kv_attn.cuh, cs_kv_rows.cuh).
//
// An item is the rows (token, query head) of some consecutive tokens of one sequence
// and key head; it needs one or more tiles of keys.  The tiles of all items, laid
// end to end, are cut into one equal range per CTA: long and short sequences, one or
// many, prompts and single tokens all load the SMs alike, without a launch per kind.
// Items cut by a range's border leave their state (O, max, sum) in the workspace, and
// the pieces are joined in their order.  Where that would cost more than it evens out,
// items stay whole (Cut::whole; run_attention in cs_kv.cu has the rule).
#pragma once
#include "cs_kv_append.cuh"

namespace cskv {

struct Cut {
  int per_item;   // tokens of an item
  int shift;      // a tile has 1 << shift keys
  int window, sinks;
  int item_cost;  // what starting and ending an item costs, in key tiles
  int flat;       // every row sees keys 0 .. flat_len - 1 of one common table (a shared prefix)
  int flat_len;
  int whole;      // no item is cut: it belongs to the range that holds its middle
};

#define CS_KV_BOTH __host__ __device__ __forceinline__  // the division's arithmetic also runs in a host test

template <typename A>
CS_KV_BOTH A kv_min(A a, A b) {
  return b < a ? b : a;
}
template <typename A>
CS_KV_BOTH A kv_max(A a, A b) {
  return a < b ? b : a;
}

CS_KV_BOTH int kt(const Cut& C) { return 1 << C.shift; }

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
CS_KV_BOTH int item_lo(const Cut& C, const Seq& s, int item) {
  return C.window > 0 ? kv_max(0, s.m - s.n + item * C.per_item - C.window + 1) : 0;
}
CS_KV_BOTH int item_hi(const Cut& C, const Seq& s, int item) {
  return C.flat ? s.m : kv_max(0, s.m - s.n + kv_min(s.n, (item + 1) * C.per_item));
}
// Tiles of the sinks before the window's first tile.
CS_KV_BOTH int sink_tiles(const Cut& C, int lo) { return kv_min((C.sinks + kt(C) - 1) >> C.shift, lo >> C.shift); }
// Key tiles of an item; at least one, so that rows without keys are written too.
CS_KV_BOTH int item_tiles(const Cut& C, const Seq& s, int item) {
  const int lo = item_lo(C, s, item), hi = item_hi(C, s, item);
  return ((kv_max(1, hi) + kt(C) - 1) >> C.shift) - (lo >> C.shift) + sink_tiles(C, lo);
}
CS_KV_BOTH int items_of(const Cut& C, const Seq& s) { return (s.n + C.per_item - 1) / C.per_item; }

// sum over i < n of floor((a i + b) / m), a, b >= 0 (the Euclid-like recurrence for
// lattice points under a line); m a + m fits 32 bits times n
CS_KV_BOTH unsigned long long floor_sum(unsigned n, unsigned m, unsigned a, unsigned b) {
  unsigned long long ans = 0;
#pragma unroll 1
  while (n > 0) {
    ans += static_cast<unsigned long long>(n) * (n - 1) / 2 * (a / m) + static_cast<unsigned long long>(n) * (b / m);
    a %= m;
    b %= m;
    const unsigned y = a * n + b;  // below 128 (n + 1), n <= 2^20 tokens
    n = y / m;
    b = y % m;
    const unsigned t = m;
    m = a;
    a = t;
  }
  return ans;
}

// Units of the first k items of a sequence (of one key head): their key tiles, and
// item_cost for each.
CS_KV_BOTH unsigned long long units_before(const Cut& C, const Seq& s, int k) {
  if (k == 0) return 0;
  if (C.flat) return static_cast<unsigned long long>(k) * static_cast<unsigned>(item_tiles(C, s, 0) + C.item_cost);
  const int full = kv_min(k, items_of(C, s) - 1);  // the last item may hold fewer tokens
  unsigned long long sum = static_cast<unsigned long long>(k) * C.item_cost;
  if (k > full) sum += item_tiles(C, s, full);
  if (full > 0) {
    const int base = s.m - s.n, P = C.per_item;
    // sum of ceil(max(1, base + (i + 1) P) / tile)
    const int early = base < 0 ? kv_min(full, -base / P) : 0;
    sum += early + floor_sum(full - early, kt(C), P, base + (early + 1) * P + kt(C) - 1);
    if (C.window > 0) {
      // minus what lies between the sinks' tiles and the window's first tile
      const int b2 = base - C.window + 1 - (((C.sinks + kt(C) - 1) >> C.shift) << C.shift);
      const int k2 = b2 >= 0 ? 0 : (-b2 + P - 1) / P;
      if (full > k2) sum -= floor_sum(full - k2, kt(C), P, b2 + k2 * P);
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
  __device__ __forceinline__ int key0(const Cut& C, int k) const { return (k < sinks ? k : (lo >> C.shift) + k - sinks) << C.shift; }
};

// Where a CTA's range of units begins and ends (CTA c takes units c * quota and
// on); every warp role walks it by itself.
struct Range {
  unsigned long long x0, x1, rem, quota;
  int b, kvh, item, off;
  Seq s;  // sequence b
};

// An item's units are item_cost of overhead and then its tiles; a range that ends
// in the overhead leaves all tiles to the next CTA.
struct Walk {
  unsigned long long x, x1;
  int b, kvh, item, off, items;
  Seq s;
  __device__ __forceinline__ Walk(const Cut& C, const Range& r)
      : x(r.x0), x1(r.x1), b(r.b), kvh(r.kvh), item(r.item), off(r.off), items(items_of(C, r.s)), s(r.s) {
    if (C.whole && off > 0) {
      const int units = item_tiles(C, s, item) + C.item_cost;
      x -= off;
      if (2 * off > units) {  // the CTA before has this item
        x += units;
        ++item;
      }
      off = 0;
    }
  }
  __device__ __forceinline__ bool next(const Batch& B, const Cut& C, Seg& g) {
    while (x < x1) {
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
      const int units = item_tiles(C, s, item) + C.item_cost;
      const unsigned long long left = x1 - x;
      if (C.whole && 2 * left <= static_cast<unsigned>(units)) return false;  // the next CTA's
      const int to = C.whole || static_cast<unsigned long long>(units - off) <= left ? units : off + static_cast<int>(left);
      g.x = x - off + C.item_cost;
      g.k0 = kv_max(0, off - C.item_cost);
      g.k1 = to - C.item_cost;
      g.item = item;
      x += to - off;
      off = 0;
      ++item;
      if (g.k1 <= g.k0) continue;
      g.s = s;
      g.b = b;
      g.kvh = kvh;
      g.tiles = units - C.item_cost;
      g.lo = item_lo(C, s, g.item);
      g.hi = item_hi(C, s, g.item);
      g.sinks = sink_tiles(C, g.lo);
      return true;
    }
    return false;
  }
};

// a / b; nearly always both fit 32 bits, where the division is much the shorter
__device__ __forceinline__ unsigned long long divide(unsigned long long a, unsigned long long b) {
  if (((a | b) >> 32) == 0) return static_cast<unsigned>(a) / static_cast<unsigned>(b);
  return a / b;
}

// One warp, all lanes: the item that holds unit r.rem of sequence s and a key head;
// 32 trials at a time.
__device__ __forceinline__ void find_item(const Cut& C, const Seq& s, Range& r) {
  const int lane = threadIdx.x & 31;
  int a = 0, e = items_of(C, s);  // units_before(a) <= rem < units_before(e)
  unsigned long long base = 0;    // units_before(a)
#pragma unroll 1
  while (e - a > 1) {
    const int step = (e - a + 31) / 32;
    const int k = a + lane * step;
    const unsigned long long u = k < e ? units_before(C, s, k) : ~0ull;
    const int last = 31 - __clz(__ballot_sync(0xFFFFFFFFu, u <= r.rem));
    base = __shfl_sync(0xFFFFFFFFu, u, last);
    a += last * step;
    e = kv_min(e, a + step);
  }
  r.item = a;
  r.off = static_cast<int>(r.rem - base);
}

__device__ __forceinline__ unsigned long long warp_inclusive(unsigned long long x) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const unsigned long long o = __shfl_up_sync(0xFFFFFFFFu, x, d);
    if ((threadIdx.x & 31) >= d) x += o;
  }
  return x;
}

// This CTA's share of `total` units.
__device__ __forceinline__ void share(unsigned long long total, Range& r) {
  r.quota = divide(total + gridDim.x - 1, gridDim.x);
  r.x0 = kv_min(r.quota * blockIdx.x, total);
  r.x1 = kv_min(r.x0 + r.quota, total);
  r.rem = 0;
  r.b = r.kvh = r.item = r.off = 0;
  r.s = Seq{0, 0, 0};
}

// Every thread of the block: this CTA's range into *out (shared memory).
template <int THREADS>
__device__ __forceinline__ void find_range(const Batch& B, const Cut& C, Range* out, unsigned long long* scratch) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int seqs = C.flat ? 1 : B.seqs;
  if (seqs <= 32) {  // one sequence per lane of one warp: no barrier but the last
    if (warp == 0) {
      Seq s{0, 0, 0};
      const bool ok = lane < seqs && load_seq(B, C, lane, s);
      const unsigned long long c = ok ? units_before(C, s, items_of(C, s)) * B.kv_heads : 0;
      const unsigned long long incl = warp_inclusive(c);
      Range r;
      share(__shfl_sync(0xFFFFFFFFu, incl, 31), r);
      if (r.x0 < r.x1) {
        r.b = __ffs(__ballot_sync(0xFFFFFFFFu, r.x0 < incl)) - 1;
        const unsigned long long in = r.x0 - __shfl_sync(0xFFFFFFFFu, incl - c, r.b);
        const unsigned long long per_head = divide(__shfl_sync(0xFFFFFFFFu, c, r.b), B.kv_heads);
        s.t0 = __shfl_sync(0xFFFFFFFFu, s.t0, r.b);
        s.n = __shfl_sync(0xFFFFFFFFu, s.n, r.b);
        s.m = __shfl_sync(0xFFFFFFFFu, s.m, r.b);
        r.kvh = static_cast<int>(divide(in, per_head));
        r.rem = in - r.kvh * per_head;
        r.s = s;
        find_item(C, s, r);
      }
      if (lane == 0) *out = r;
    }
    __syncthreads();
    return;
  }
  const int per = (seqs + THREADS - 1) / THREADS;
  const int b0 = kv_min(tid * per, seqs);
  int b1 = kv_min(b0 + per, seqs);
  unsigned long long at = 0, x0 = 0;
  Seq s;
  // first the units of all sequences, then, by the thread whose sequences hold unit
  // x0, the one that holds it
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    unsigned long long mine = 0;
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
      if (!load_seq(B, C, b, s)) continue;
      const unsigned long long c = units_before(C, s, items_of(C, s));
      const unsigned long long in = x0 - at - mine * B.kv_heads;
      if (pass == 1 && in < c * B.kv_heads) {
        out->b = b;
        out->kvh = static_cast<int>(divide(in, c));
        out->rem = in - out->kvh * c;
        break;
      }
      mine += c;
    }
    if (pass == 1) break;
    unsigned long long incl = warp_inclusive(mine);
    if (lane == 31) scratch[warp] = incl;
    __syncthreads();
    unsigned long long before = 0, total = 0;
#pragma unroll 1
    for (int w = 0; w < THREADS / 32; ++w) {
      if (w < warp) before += scratch[w];
      total += scratch[w];
    }
    incl = (incl + before) * B.kv_heads;
    Range r;
    share(total * B.kv_heads, r);
    if (tid == 0) *out = r;
    __syncthreads();
    x0 = r.x0;
    at = incl - mine * B.kv_heads;
    if (r.x0 >= r.x1 || x0 < at || x0 >= incl) b1 = b0;
  }
  __syncthreads();
  if (warp == 0 && out->x0 < out->x1 && load_seq(B, C, out->b, s)) {
    Range r = *out;
    r.s = s;
    find_item(C, s, r);
    __syncwarp();
    if (lane == 0) *out = r;
  }
  __syncthreads();
}

}  // namespace cskv
