// Attention over the paged key/value cache (include/cs_kv.h) on the tensor cores.
//
// Mathematics.  For one sequence and key head, the rows of a product are the
// (token, query head) pairs that read that head: S = Q K^T, running row maximum
// and sum, P = 2^(c S - max), O += P V, and O / sum at the end.
//
// Work.  An item is 2 x 128 such rows (whole tokens), its tiles have 128 keys; one CTA
// per SM (cs_kv_sched.cuh).  Pieces of items are joined by a kernel of their own.
//
// Layout.  Q and K, V tiles come by TMA, page by page, into 128-byte-swizzled shared
// memory; both S buffers (128 x 128, fp32) and both O lie in TMEM, and P goes back over
// the first half of its S as the A operand of O += P V.  So a softmax thread owns a row:
// its maximum and sum need no exchange, and while one buffer is at its exponentials the
// other's products run.  Sums, maxima, S and O are fp32; P is rounded to the operands'
// type (off by at most 2^-8 of the weight in bf16, 2^-11 in fp16; a weight is at most 2^8 by
// the row's reference, so fp16 has room for it), O once at the end.
//
// Bound.  Per tile of 128 x 128 weights the tensor core needs 8 x 64 cycles for S and as
// many for P V at 128 dimensions (half at 64), the two softmax warpgroups together about
// 960 issue cycles per scheduler and pair of tiles.  A prompt of 8192 tokens, 32 / 8 heads of 128:
// 401 us, 1370 TFLOP/s, 0.71 of the 1925 that a library product of 8192^3 measured;
// pieces of prompts over 2000 to 20000 keys, 40 / 8 heads of 64: 424 us, 895 TFLOP/s.
// The counters (4096 tokens) have the tensor core busy
// in 58 % of the cycles (38 % at 64 dimensions), issue slots 32 % (42 %), DRAM 7 %: no
// unit is full, the chain S -> softmax -> P V of each buffer sets the pace.  A pair of tiles
// takes about 3500 cycles at 128 dimensions and 2500 at 64, where its products are 2048 and
// 1024: the same 1400 or so of latency in both.
#pragma once
#include "cs_kv_sched.cuh"

namespace cskv {

constexpr int KT = 128;  // keys per tile (Cut.shift 7)

// An item whose tiles several CTAs share.
struct Split {
  int pieces;     // 0: none
  int first;      // its first piece is the CTA's last piece (1) or only (0)
  int token, tokens, kvh;
};

struct AttnP {
  CUtensorMap q, k, v;    // for cs_kv_attn_kernel
  const void *q_raw, *k_raw, *v_raw;  // the tensors themselves: q for cs_kv_rows_kernel, all for mend_row
  long long q_stride;
  Batch b;
  Cut c;
  const int* pages;       // flat: the prefix's pages
  void* out;
  float* lse;
  long long out_stride;   // elements
  float scale_log2;       // scale * log2(e): exponents in base 2
  float* part;            // pieces' states: [CTA][first piece, last piece][tile][128 rows][O, max, sum, 6 unused]
  float4* other;          // warpgroup 1's half of an item of one row tile: [CTA][D / 4 + 1][128 rows]
  Split* splits;          // [CTA] the item that starts there and ends elsewhere
  int num_splits;
  uint32_t* arrivals;     // cs_kv_rows_kernel: [CTA] its pieces that are stored
  uint8_t* mend;          // [tokens][heads]: the row is to be computed again (mend_row)
  float* flat_o;          // [tokens][heads][D], [tokens][heads]: a prefix's normalised output and
  float* flat_lse;        // base-2 log-sum-exp; written with c.flat, else joined in if not null
  int per_tile;           // tokens of a 128-row tile: 128 / group, rounded down; an item has two
  int out_wide;           // rows of out start on 32-byte boundaries
  int head_groups;        // 8-slot groups between heads (HEAD layout), 0: heads are a dimension of their own
};

// Two softmax warpgroups, one per S buffer with a row per thread, and one with the
// TMA warp, two MMA warps and an idle one.
constexpr int ATTN_THREADS = 384;
// Registers: 65536 / 384 gives every thread 168 at launch; a softmax thread holds a
// row of S, so the third warpgroup hands over what it does not need
// (2 x 216 + 72 = 3 x 168).  Nothing may spill: next to 226 KB of shared memory the
// L1 holds nearly nothing, and a spilled register comes back from L2.
constexpr int SOFTMAX_REGS = 216, OTHER_REGS = 72;
static_assert(2 * SOFTMAX_REGS + OTHER_REGS <= 3 * 168, "more registers than the launch holds");
template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
constexpr uint32_t COL_S = 0, COL_O = 256;
constexpr int CTL = 1024;  // bytes of the control block
constexpr float RAISE_LOG2 = 8.0f;  // the reference maximum follows a row's when it is exceeded by more than 2^8

template <int D>
struct AttnShape {
  static constexpr int HALVES = D / 64;
  static constexpr int TILE = KT * D * 2;              // bytes of a 128-row tile of Q, K or V
  static constexpr int SLOTS = D == 128 ? 5 : 10;      // ring of K and V tiles: 160 KB in flight
  static constexpr int SMEM = 2 * TILE + SLOTS * TILE + 1024 + CTL;
};

template <int SLOTS>
struct AttnCtl {
  uint64_t full[SLOTS], empty[SLOTS];
  uint64_t q_full[2], q_empty[2], s_full[2], p_full[2][2], o_full[2];
  uint64_t v_ready[2];                 // the values of the buffer's tile are there
  uint64_t other_full, other_empty;    // warpgroup 1's half of an item of one row tile
  uint64_t drained;
  unsigned long long scratch[ATTN_THREADS / 32];
  Range range;
  uint32_t tmem;
  volatile int abort;
  int turn;               // an MMA warp has the tensor core
  int loads, q_loads[2];  // tiles and queries whose copies were issued
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

// One lane of a converged warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
  return one != 0;
}

// Bounded wait; false when it ran out, here or in another role.  What is waited
// for is always work of this CTA, microseconds away; a try suspends the thread
// for some microseconds, so the limit is a second or two.  (Kept small: with a slow path's
// timer and error record inlined everywhere the kernel had 156 KB of code, and its
// warps waited for instructions; with a suspend-time hint a prompt of 8192 tokens
// took 410 us instead of 397.)
#ifndef CS_KV_WAIT_TRIES  // a test lets its waits run out
#define CS_KV_WAIT_TRIES (1 << 18)
#endif
constexpr int SETTLE_TRIES = 1 << 18;  // for copies and MMAs in flight after a wait that ran out
template <typename Try>
CS_KV_BOTH bool wait_bounded(volatile int* abort, Try complete) {
#pragma unroll 1
  for (int i = 0; i < CS_KV_WAIT_TRIES; ++i) {
    if (complete()) return true;
    if (*abort) return false;
  }
  *abort = 1;
  return false;
}
template <typename Ctl>
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, Ctl* sc) {
  return wait_bounded(&sc->abort, [&] { return cs::mbar_try_wait(bar, parity); });
}

// The same for a whole warp, which goes on or gives up together.
template <typename Ctl>
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, Ctl* sc) {
  if (CS_KV_WAIT_TRIES > 0 && __all_sync(0xFFFFFFFFu, cs::mbar_try_wait(bar, parity))) return true;
  return __all_sync(0xFFFFFFFFu, wait(bar, parity, sc));
}

// After a wait that ran out, one thread: this CTA's copies and MMAs in flight
// come to rest (again with a limit) before its memory is given back.
template <int SLOTS>
__device__ void come_to_rest(AttnCtl<SLOTS>* sc, const AttnP& p) {
  record(p.b.ctrl, ERR_WATCHDOG, WHAT_WAIT, blockIdx.x);
  int tries = 0;
  auto settle = [&](uint64_t* bar, uint32_t parity) {
    while (!cs::mbar_try_wait(bar, parity) && ++tries < SETTLE_TRIES) {
    }
  };
  for (int i = 0; i < SLOTS; ++i) {
    const int n = (sc->loads - i + SLOTS - 1) / SLOTS;  // loads into slot i
    if (n > 0) settle(&sc->full[i], (n - 1) & 1);
  }
  for (int w = 0; w < 2; ++w)
    if (sc->q_loads[w] > 0) settle(&sc->q_full[w], (sc->q_loads[w] - 1) & 1);
  settle(&sc->drained, 0);
}

// The tensor core for a group of MMAs (given back by clearing sc->turn).
template <typename Ctl>
__device__ __forceinline__ void take_turn(Ctl* sc) {
#pragma unroll 1
  for (int i = 0; i < CS_KV_WAIT_TRIES && atomicCAS(&sc->turn, 0, 1) != 0 && !sc->abort; ++i) {
  }
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
  Walk walk(p.c, sc->range);
  Seg g;
  Ring<Sh::SLOTS> rp;
  uint32_t q_phase[2] = {1, 1};
  while (walk.next(B, p.c, g)) {
    const int* table = p.c.flat ? p.pages : B.table + static_cast<long long>(g.b) * B.table_cols;
    const bool two = g.s.n - g.item * p.c.per_item > p.per_tile;
    auto queries = [&](int w) {
      if (!wait_warp(&sc->q_empty[w], q_phase[w], sc)) return false;
      q_phase[w] ^= 1u;
      if (lane == 0) {
        cs::mbar_arrive_expect_tx(&sc->q_full[w], static_cast<uint32_t>(p.per_tile) * B.group * D * 2);
        for (int h = 0; h < Sh::HALVES; ++h)
          tma_3d(qbuf + w * Sh::TILE + h * (KT * 128), &p.q, h * 64, g.kvh * B.group,
                 g.s.t0 + g.item * p.c.per_item + w * p.per_tile, &sc->q_full[w]);
        ++sc->q_loads[w];
      }
      return true;
    };
    if (!queries(0)) return false;
    // the page that this lane brings of tile k, -1: none of its keys is seen
    auto page_of = [&](int k) {
      if (k >= g.k1 || lane >= pages_per_tile) return -1;
      const int j0 = g.key0(p.c, k) + (lane << B.page_shift), j1 = j0 + B.page_size;
      if (j0 >= g.hi || (j1 <= g.lo && j0 >= p.c.sinks)) return -1;
      const int page = __ldg(table + (j0 >> B.page_shift));
      if (page >= 0 && page < B.num_pages) return page;
      record(B.ctrl, ERR_INVALID, WHAT_PAGE, p.c.flat ? 0xFFFFFFFFu : static_cast<uint32_t>(g.b));
      return -1;
    };
    int page = page_of(g.k0);
#pragma unroll 1
    for (int k = g.k0; k < g.k1; ++k) {
      const uint32_t boxes = __popc(__ballot_sync(0xFFFFFFFFu, page >= 0));
      const int after = page_of(k + 1);
      const int c3 = p.head_groups ? 0 : g.kvh;
      const int c4 = page * (p.head_groups ? p.head_groups * B.kv_heads : groups) + g.kvh * p.head_groups;
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {  // K, then V
        if (!wait_warp(&sc->empty[rp.slot], rp.phase ^ 1u, sc)) return false;
        if (lane == 0) {
          cs::mbar_arrive_expect_tx(&sc->full[rp.slot], boxes * B.page_size * D * 2);
          ++sc->loads;
        }
        __syncwarp();
        if (page >= 0)
          tma_5d(ring + rp.slot * Sh::TILE + lane * (B.page_size * D * 2), half ? &p.v : &p.k, 0, 0, 0, c3, c4,
                 &sc->full[rp.slot]);
        rp.next();
        // the second row tile's queries, which the last item may still hold, after the first keys
        if (two && k == g.k0 && half == 0 && !queries(1)) return false;
      }
      page = after;
    }
  }
  return true;
}

// Under a window: the key tiles of a segment of an item of two row tiles in which row
// tile w sees a key, that is its leading sink tiles (k < sinks) and tiles a .. last; if there
// is none, the segment's first, so that the rows' state exists.  (Without a window only an
// item's last tile could be left out; that gained nothing.)
struct Seen {
  int first, last, sinks, a;
  __device__ __forceinline__ Seen(const AttnP& p, const Seg& g, int w) {
    const int tok = g.item * p.c.per_item + w * p.per_tile, base = g.s.m - g.s.n;
    const int lo = max(0, base + tok - p.c.window + 1), end = base + min(g.s.n, tok + p.per_tile);
    // (sinks that reach into the window's first tiles are no tiles of their own: k is the tile's place then)
    sinks = (p.c.sinks + KT - 1) / KT;
    a = g.sinks + lo / KT - g.lo / KT;
    const int b = end > 0 ? g.sinks + (end - 1) / KT - g.lo / KT : -1;
    first = g.k0 >= sinks ? max(g.k0, a) : g.k0;
    last = min(g.k1 - 1, b);
    if (last >= sinks && last < a) last = sinks - 1;
    if (last < first) first = last = g.k0;
  }
  __device__ __forceinline__ int next(int k) const { return k + 1 >= sinks && k + 1 < a ? a : k + 1; }
};

// The phases of the query buffers' barriers.  MMA warp w reads buffer w of an item of two row
// tiles and buffer 0 of an item of one; it waits for every copy into buffer 0 all the
// same: a parity tells two phases apart, so a warp that passed one over could take the
// copy of two items ago for the one it waits for.
struct Queries {
  uint32_t phase = 0;  // bit per buffer
  template <typename Wait>  // wait(buffer, parity)
  CS_KV_BOTH bool arrived(bool two, int w, Wait wait) {
    bool ok = wait(0, phase & 1u);
    if (ok && two && w == 1) ok = wait(1, phase >> 1);
    phase ^= two ? 3u : 1u;
    return ok;
  }
};

// MMA warp w works for S buffer w: S = Q K^T, then, once the softmax has put P into the
// first half of S, O += P V.  An item of two row tiles has one for each buffer; of an item
// of one row tile the buffers take the key tiles in turn (and are joined at the end).
// The issue of an MMA holds its warp for the 64 cycles that the tensor core works
// on one, so whatever else the warp does leaves the tensor core idle, unless the other
// buffer's warp is issuing: with one warp for both buffers a step of 1024 cycles took 2300.
// A buffer's MMAs are issued by one thread and execute in that order, and no
// MMA reads what the other buffer's write.
template <int D, bool WINDOW>
__device__ bool mma_role(const AttnP& p, AttnCtl<AttnShape<D>::SLOTS>* sc, uint8_t* qbuf, uint8_t* ring, int bf16, int w) {
  using Sh = AttnShape<D>;
  const uint32_t idesc_s = cs::make_idesc_f16(bf16, 0, 128, KT);
  const uint32_t idesc_o = cs::make_idesc_f16(bf16, 1, 128, D);
  const uint32_t s_tm = sc->tmem + COL_S + w * 128, o_tm = sc->tmem + COL_O + w * D;
  const uint64_t q_desc = cs::smem_desc_sw128(cs::smem_u32(qbuf), 16, 1024);
  const uint64_t k_desc = cs::smem_desc_sw128(cs::smem_u32(ring), 16, Sh::HALVES * 1024);
  const uint64_t v_desc = cs::smem_desc_sw128(cs::smem_u32(ring), 1024, Sh::HALVES * 1024);
  const bool leader = elect_one();
  Walk walk(p.c, sc->range);
  Seg g;
  // Both warps watch every tile arrive, and give back the ones they do not read
  // too: a barrier's parity tells two phases apart, so no reader may be two behind.
  Ring<Sh::SLOTS> r;
  Queries queries;
  uint32_t p_phase = 0;
  bool ok = true;
  while (ok && walk.next(p.b, p.c, g)) {
    const bool two = g.s.n - g.item * p.c.per_item > p.per_tile;
    const int qw = two ? w : 0, count = g.k1 - g.k0;
    ok = queries.arrived(two, w, [&](int b, uint32_t parity) { return wait_warp(&sc->q_full[b], parity, sc); });
    if (!ok) break;
    // both warps give the first queries back, warp 1 at once where it does not read them (the
    // wait above keeps it from doing so for an item before its queries are loaded)
    if (leader && w == 1 && (two || count == 1)) cs::mbar_arrive(&sc->q_empty[0]);
    // S of the tile whose keys lie in `slot`; the last one gives the queries back
    auto scores = [&](int slot, bool last) {
      uint64_t a = q_desc + qw * (Sh::TILE >> 4), b = k_desc + slot * (Sh::TILE >> 4);
#pragma unroll 1
      for (int h = 0; h < Sh::HALVES; ++h, a += KT * 128 >> 4, b += 1024 >> 4)
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) cs::tc_mma_f16<1>(s_tm, a + kk * 2, b + kk * 2, idesc_s, h + kk);
      cs::tc_commit<1>(&sc->s_full[w]);
      cs::tc_commit<1>(&sc->empty[slot]);
      if (last) cs::tc_commit<1>(&sc->q_empty[qw]);
    };
    // 64 keys' part of P V
    auto values = [&](int slot, int h, bool add) {
      const uint64_t b = v_desc + (slot * (Sh::TILE >> 4) + h * (Sh::HALVES * 8192 >> 4));
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
        mma_ts(o_tm, s_tm + h * 32 + kk * 8, b + kk * (Sh::HALVES * 2048 >> 4), idesc_o, add || kk > 0);
    };
    auto segment = [&](auto pair) {
      constexpr bool TWO = decltype(pair)::value;  // an item of two row tiles
      // this buffer's tiles: first, and then every one, every second one, or what is seen
      const Seen seen(p, g, w);
      const int first = TWO && WINDOW ? seen.first - g.k0 : TWO ? 0 : w;
      const int last = TWO && WINDOW ? seen.last - g.k0 : TWO ? count - 1 : count - 1 - ((count - 1 - w) & 1);
      int own = first;
      bool issued = false;  // S of this tile was issued right behind the last P V
#pragma unroll 1
      for (int t = 0; t < count; ++t) {
        if ((!TWO || WINDOW) && t != own) {
          for (int i = 0; i < 2; ++i) {
            if (!wait_warp(&sc->full[r.slot], r.phase, sc)) return false;
            if (leader) cs::mbar_arrive(&sc->empty[r.slot]);
            r.next();
          }
          continue;
        }
        if (!issued) {
          if (!wait_warp(&sc->full[r.slot], r.phase, sc)) return false;
          cs::tc_fence_after();
          if (leader) scores(r.slot, t == last);
          r.next();
        }
        if (!wait_warp(&sc->full[r.slot], r.phase, sc)) return false;
        const int sv = r.slot;
        r.next();
        if (leader) cs::mbar_arrive(&sc->v_ready[w]);
        own = t == last ? -1 : !TWO ? t + 2 : WINDOW ? seen.next(t + g.k0) - g.k0 : t + 1;
        // with the next tile's keys there, nothing comes between this P V and its S
        issued = TWO && t != last && (!WINDOW || own == t + 1) &&
                 __all_sync(0xFFFFFFFFu, cs::mbar_test_wait(&sc->full[r.slot], r.phase));
        const int sk = r.slot;
        if (!wait_warp(&sc->p_full[w][0], p_phase, sc)) return false;  // the weights of the first 64 keys come before the rest
        cs::tc_fence_after();
        if (leader) values(sv, 0, t != first);
        if (!wait_warp(&sc->p_full[w][1], p_phase, sc)) return false;
        cs::tc_fence_after();
        if (leader) {
          // one buffer's twelve MMAs after the other's: issued side by side, both S would
          // be done late, both softmaxes run at a time, and the tensor core wait for them
          // (64 dimensions: an MMA of P V takes half the time and the softmax bounds the rest)
          if (D == 128 && issued) take_turn(sc);
          values(sv, 1, true);
          if (issued) {
            scores(sk, t + 1 == last);
            if (D == 128) atomicExch(&sc->turn, 0);
          }
          cs::tc_commit<1>(&sc->empty[sv]);
          if (t == last) cs::tc_commit<1>(&sc->o_full[w]);
        }
        p_phase ^= 1u;
        if (issued) r.next();
      }
      return true;
    };
    ok = two ? segment(std::true_type()) : segment(std::false_type());
  }
  if (leader) cs::tc_commit<1>(&sc->drained);  // all MMAs of this warp are done
  return ok;
}

// Store 16 consecutive 32-bit columns of this thread's lane.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// max of three, two multiply-adds and two sums at a time
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ uint64_t pack64(float a, float b) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ void unpack64(uint64_t x, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// A row's state in a piece: O against the maximum, the maximum and the sum.
template <int D>
__device__ __forceinline__ float* piece_state(float* part, unsigned cta, int which, int tile, int r) {
  return part + (((static_cast<size_t>(cta) * 2 + which) * 2 + tile) * 128 + r) * (D + 8);
}

// The log-sum-exp of an output row from its maximum and sum (base 2).
__device__ __forceinline__ void put_lse(const AttnP& p, long long row, float m, float l) {
  if (!p.c.flat && !p.lse) return;
  const float lse2 = l == 0.0f ? -INFINITY : m + log2f(l);
  if (p.c.flat)
    p.flat_lse[row] = lse2;
  else
    p.lse[row] = lse2 * 0.6931471805599453f;
}

// A row whose weights are finite and whose output is not: some value of its tiles is
// not, maybe one at a key that is hidden from this row only (its weight 0 times NaN or
// infinity is NaN).  If there is one, the row is computed again from its visible keys alone.
__device__ __forceinline__ void mark(const AttnP& p, long long row) {
  if (p.c.flat) return;  // no key is hidden from one row and seen by another
  p.mend[row] = 1;
  p.b.ctrl[CTRL_MEND] = 1;
}

// x += f * the 32 values of 8 float4s `stride` apart (written by this grid or an earlier one).
__device__ __forceinline__ void axpy(float (&x)[32], const float4* src, int stride, float f) {
  float4 y[8];
#pragma unroll
  for (int t = 0; t < 8; ++t) y[t] = __ldcg(src + t * stride);
#pragma unroll
  for (int t = 0; t < 8; ++t) {
    x[4 * t] = fmaf(y[t].x, f, x[4 * t]);
    x[4 * t + 1] = fmaf(y[t].y, f, x[4 * t + 1]);
    x[4 * t + 2] = fmaf(y[t].z, f, x[4 * t + 2]);
    x[4 * t + 3] = fmaf(y[t].w, f, x[4 * t + 3]);
  }
}

__device__ __forceinline__ void st32(void* p, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]),
               "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// The bits 0 .. n - 1 (none for n <= 0, all from 32 on).
__device__ __forceinline__ uint32_t below(int n) { return n >= 32 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << n) - 1u; }

// Warpgroup w: the softmax of the steps with S buffer w, one row per thread, and the output.
template <typename T, int D, bool WINDOW>
__device__ bool softmax_role(const AttnP& p, AttnCtl<AttnShape<D>::SLOTS>* sc, uint8_t* ring, int w) {
  using Sh = AttnShape<D>;
  constexpr int CH = D / 32;                                      // chunks of 32 columns of O
  const Batch& B = p.b;
  const int r = threadIdx.x & 127, lane = threadIdx.x & 31;
  const uint32_t lanes = static_cast<uint32_t>(r & ~31) << 16;
  const uint32_t s_tm = sc->tmem + lanes + COL_S + w * 128, o_tm = sc->tmem + lanes + COL_O + w * D;
  const int row_tok = r / B.group, row_head = r - row_tok * B.group;
  float4* const shared_half = p.other + static_cast<size_t>(blockIdx.x) * (D / 4 + 1) * 128 + r;
  auto read_o = [&](int c, uint32_t (&o)[32]) {
    cs::tmem_ld32(o_tm + c * 32, o);
    cs::tc_wait_ld();
    cs::tc_wait_ld_regs(o);
  };
  const uint64_t scale2 = pack64(p.scale_log2, p.scale_log2);
  Walk walk(p.c, sc->range);
  Seg g;
  uint32_t tiles_done = 0;  // key tiles of the segments before this one
  uint32_t s_phase = 0, o_phase = 0, x_phase = 0;
  while (walk.next(B, p.c, g)) {
    const int count = g.k1 - g.k0;
    const uint32_t ring0 = 2 * tiles_done;
    tiles_done += count;
    const bool two = g.s.n - g.item * p.c.per_item > p.per_tile;
    if (!two && w >= count) continue;  // one key tile of one row tile: buffer 0 alone
    const int tile = two ? w : 0;      // this buffer's row tile
    const int first = g.item * p.c.per_item + tile * p.per_tile;  // its first token
    const int base = g.s.m - g.s.n;
    const int tok = first + row_tok;
    const bool live = row_tok < p.per_tile && tok < g.s.n;
    const int end = p.c.flat ? g.s.m : live ? base + tok + 1 : 0;  // keys [.., end) are seen
    const int lo = WINDOW ? max(0, base + tok + 1 - p.c.window) : 0;
    // keys below `some` and from `all_lo` on are seen by every live row
    const int some = p.c.flat ? g.s.m : base + first + 1;
    const int all_lo = WINDOW ? max(0, base + first + p.per_tile - p.c.window) : 0;
    float m_ref = -INFINITY, l = 0.0f;
    const Seen seen(p, g, w);
    const int k_first = two ? WINDOW ? seen.first : g.k0 : g.k0 + w, k_end = WINDOW && two ? seen.last + 1 : g.k1;
#pragma unroll 1
    for (int k = k_first; k < k_end; k = WINDOW && two ? seen.next(k) : k + (two ? 1 : 2)) {
      // what the tile needs, known before its scores are there
      const bool fresh = k == k_first;  // O of this buffer holds nothing yet
      const int j0 = WINDOW ? g.key0(p.c, k) : k * KT;
      const bool mask = !(j0 + KT <= some && (!WINDOW || j0 >= all_lo || j0 + KT <= p.c.sinks));  // some key is hidden from some row
      const bool unseen = j0 + KT > g.hi || (WINDOW && j0 < g.lo && j0 + KT > p.c.sinks);       // from every row of the item
      if (!wait_warp(&sc->s_full[w], s_phase, sc)) return false;
      s_phase ^= 1u;
      cs::tc_fence_after();
      if (__builtin_expect(mask, 0)) {
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {  // hidden scores become -inf in place
          const int j1 = j0 + 32 * c;
          const uint32_t seen = below(end - j1) & (WINDOW ? ~below(lo - j1) | below(p.c.sinks - j1) : 0xFFFFFFFFu);
          uint32_t v[32];
          cs::tmem_ld32(s_tm + c * 32, v);
          cs::tc_wait_ld();
          cs::tc_wait_ld_regs(v);
#pragma unroll
          for (int t = 0; t < 32; ++t)
            if (!(seen >> t & 1u)) v[t] = 0xFF800000u;
          cs::tmem_st32(s_tm + c * 32, v);
        }
        cs::tc_wait_st();
      }
      uint32_t v[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c) cs::tmem_ld32(s_tm + c * 32, v[c]);
      cs::tc_wait_ld();
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        cs::tc_wait_ld_regs(v[c]);
#pragma unroll
        for (int t = 0; t < 32; t += 2)
          mx[(t >> 1) & 3] = max3(mx[(t >> 1) & 3], __uint_as_float(v[c][t]), __uint_as_float(v[c][t + 1]));
      }
      const float m_tile = max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]) * p.scale_log2;
      // the reference is raised only when a row's maximum exceeds it by more than
      // 2^8 (so P <= 2^8, and rounding to the dtype is as good as at 1);
      // then O and l are scaled down first
      const bool raise = m_tile > m_ref + RAISE_LOG2 || (m_ref == -INFINITY && m_tile > -INFINITY);
      const float m_new = raise ? m_tile : m_ref;
      if (__builtin_expect(!fresh && __any_sync(0xFFFFFFFFu, raise), 0)) {
        // S of this tile was issued after P V of the buffer's last one: O is complete
        const float f = raise ? cs::ex2_approx(m_ref - m_new) : 1.0f;
        l *= f;
#pragma unroll 1
        for (int c = 0; c < CH; ++c) {
          uint32_t o[32];
          read_o(c, o);
#pragma unroll
          for (int t = 0; t < 32; ++t) o[t] = __float_as_uint(__uint_as_float(o[t]) * f);
          cs::tmem_st32(o_tm + c * 32, o);
        }
      }
      m_ref = m_new;
      // values of keys that no row of the item sees may hold anything: zeros in
      // their place before this buffer's P V (the other buffer's warps write them as well)
      if (__builtin_expect(unseen, 0)) {
        const uint32_t slot = (ring0 + 2 * (k - g.k0) + 1) % Sh::SLOTS;
        if (!wait_warp(&sc->v_ready[w], s_phase ^ 1u, sc)) return false;
        const int j = j0 + r;
        if (j >= g.hi || (WINDOW && j < g.lo && j >= p.c.sinks)) {
          uint8_t* row = ring + slot * Sh::TILE + (r >> 3) * (Sh::HALVES * 1024) + (r & 7) * 128;
          for (int h = 0; h < Sh::HALVES; ++h)
#pragma unroll
            for (int c = 0; c < 8; ++c) *reinterpret_cast<uint4*>(row + h * 1024 + c * 16) = make_uint4(0, 0, 0, 0);
        }
        cs::fence_proxy_async_shared();  // and all warps signal before the MMA reads
      }
      const float sub = m_ref == -INFINITY ? 0.0f : -m_ref;
      const uint64_t sub2 = pack64(sub, sub);
      uint64_t ls[2] = {0, 0};
#pragma unroll
      for (int c = 0; c < 4; ++c) {  // P V of the first 64 keys starts while the rest is computed
        uint32_t pk[16];
#pragma unroll
        for (int t = 0; t < 32; t += 2) {
          float x, y;
          unpack64(fma2(pack64(__uint_as_float(v[c][t]), __uint_as_float(v[c][t + 1])), scale2, sub2), x, y);
          x = cs::ex2_approx(x);
          y = cs::ex2_approx(y);
          pk[t >> 1] = Pair<T>::put(x, y);
          ls[(t >> 1) & 1] = add2(ls[(t >> 1) & 1], pack64(x, y));
        }
        tmem_st16(s_tm + c * 16, pk);
        if (c & 1) {
          cs::tc_wait_st();
          cs::tc_fence_before();
          __syncwarp();
          if (lane == 0) cs::mbar_arrive(&sc->p_full[w][c >> 1]);
        }
      }
      float l0, l1;
      unpack64(add2(ls[0], ls[1]), l0, l1);
      l += l0 + l1;
    }
    if (!wait_warp(&sc->o_full[w], o_phase, sc)) return false;
    cs::tc_fence_after();
    o_phase ^= 1u;
    // the state of this row: O (in tensor memory) and l, both against m_ref
    if (!two && w == 1) {
      // the other key tiles of buffer 0's rows, which joins them
      if (!wait_warp(&sc->other_empty, x_phase ^ 1u, sc)) return false;
      x_phase ^= 1u;
      float4* to = shared_half;
#pragma unroll 1
      for (int c = 0; c < CH; ++c) {
        uint32_t o[32];
        read_o(c, o);
        if (live)
#pragma unroll
          for (int t = 0; t < 8; ++t)
            to[(c * 8 + t) * 128] = make_float4(__uint_as_float(o[4 * t]), __uint_as_float(o[4 * t + 1]),
                                                       __uint_as_float(o[4 * t + 2]), __uint_as_float(o[4 * t + 3]));
      }
      if (live) to[D / 4 * 128] = make_float4(m_ref, l, 0.0f, 0.0f);
      cs::tc_fence_before();
      cs::mbar_arrive(&sc->other_full);
      continue;
    }
    const float4* other = nullptr;
    float f_own = 1.0f, f_other = 0.0f;
    if (!two && count > 1) {
      if (!wait_warp(&sc->other_full, x_phase, sc)) return false;
      x_phase ^= 1u;
      if (live) {
        other = shared_half;
        const float4 ml = __ldcg(other + D / 4 * 128);
        const float m_new = fmaxf(m_ref, ml.x);
        f_own = m_ref == -INFINITY ? 0.0f : cs::ex2_approx(m_ref - m_new);
        f_other = ml.x == -INFINITY ? 0.0f : cs::ex2_approx(ml.x - m_new);
        l = l * f_own + ml.y * f_other;
        m_ref = m_new;
      }
    }
    const long long row = static_cast<long long>(g.s.t0 + tok) * B.heads + g.kvh * B.group + row_head;
    const bool whole = g.whole();
    float f = f_own, fold = 0.0f;
    const float4* pre = nullptr;
    float* to = piece_state<D>(p.part, blockIdx.x, sc->range.x0 < g.x, tile, r);
    if (whole) {
      if (live && !p.c.flat && p.flat_o) {  // join the prefix's output
        pre = reinterpret_cast<const float4*>(p.flat_o + row * D);
        const float z = p.flat_lse[row];
        const float m_new = fmaxf(m_ref, z);
        const float own = m_ref == -INFINITY ? 0.0f : cs::ex2_approx(m_ref - m_new);
        fold = z == -INFINITY ? 0.0f : cs::ex2_approx(z - m_new);
        l = l * own + fold;
        f *= own;
        f_other *= own;
        m_ref = m_new;
      }
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
      f *= inv;
      f_other *= inv;
      fold *= inv;
    }
    float probe = 0.0f;  // NaN if an element of the row is not finite
#pragma unroll 1
    for (int c = 0; c < CH; ++c) {
      float x[32];
      uint32_t o[32];
      read_o(c, o);
#pragma unroll
      for (int t = 0; t < 32; ++t) x[t] = __uint_as_float(o[t]) * f;
      if (other) axpy(x, other + c * 8 * 128, 128, f_other);
#pragma unroll
      for (int t = 0; t < 32; ++t) probe = fmaf(x[t], 0.0f, probe);
      if (!live) continue;
      if (pre) axpy(x, pre + c * 8, 1, fold);
      if (!whole || p.c.flat) {  // 32-bit values: a piece's state, or a prefix's output
        float* dst = whole ? p.flat_o + row * D + c * 32 : to + c * 32;
#pragma unroll
        for (int t = 0; t < 4; ++t) st32(dst + 8 * t, reinterpret_cast<uint32_t*>(x) + 8 * t);
      } else {
        uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(p.out) + (g.s.t0 + tok) * p.out_stride +
                                              (g.kvh * B.group + row_head) * D + c * 32);
        uint32_t y[16];
#pragma unroll
        for (int t = 0; t < 16; ++t) y[t] = Pair<T>::put(x[2 * t], x[2 * t + 1]);
        if (p.out_wide) {
          // a lane's row is another line than its neighbours': whole 32-byte sectors at least
          st32(dst, y);
          st32(dst + 2, y + 8);
        } else {
#pragma unroll
          for (int t = 0; t < 4; ++t) dst[t] = make_uint4(y[4 * t], y[4 * t + 1], y[4 * t + 2], y[4 * t + 3]);
        }
      }
    }
    __syncwarp();
    cs::tc_fence_before();
    if (!two && count > 1) cs::mbar_arrive(&sc->other_empty);  // the other buffer's state is read
    if (whole) {
      if (live) {
        put_lse(p, row, m_ref, l);
        if (probe != 0.0f && isfinite(l)) mark(p, row);
      }
    } else {
      if (live) *reinterpret_cast<float2*>(to + D) = make_float2(m_ref, l);
      if (threadIdx.x == 0 && sc->range.x0 <= g.x) {  // the item starts here: what its joining needs to know
        const unsigned q = static_cast<unsigned>(min(sc->range.quota, 0x80000000ull));
        const unsigned long long end_x = g.x + g.tiles - 1;
        Split sp;
        sp.pieces = static_cast<unsigned>(end_x - sc->range.x1) / q + 2;
        sp.first = sc->range.x0 < g.x;
        sp.token = g.s.t0 + g.item * p.c.per_item;
        sp.tokens = min(p.c.per_item, g.s.n - g.item * p.c.per_item);
        sp.kvh = g.kvh;
        p.splits[blockIdx.x] = sp;
      }
      __syncwarp();
    }
  }
  return true;
}

// One warp: the output of a token and head from its visible keys alone, one key after
// another with the running maximum.
template <typename T, int D>
__device__ __noinline__ void mend_row(const AttnP& p, int t, int h) {
  const Batch& B = p.b;
  const int lane = threadIdx.x & 31, b = sequence_of(B, t);
  int t0, n, m;
  if (!sequence(B, b, t0, n, m) || t < t0 || t >= t0 + n) return;
  const int pos = m - n + t - t0, kh = h / B.group;
  constexpr int W = D / 64;  // 32-bit words per lane
  const int* pages = B.table + static_cast<long long>(b) * B.table_cols;
  const int lo = p.c.window > 0 ? max(0, pos - p.c.window + 1) : 0, sinks = min(p.c.sinks, lo);
  // element offset of key j's row, negative: its page is not in the pool
  auto row_of = [&](int j) {
    const int page = __ldg(pages + (j >> B.page_shift));
    return page < 0 || page >= B.num_pages
               ? -1ll
               : page * B.page_stride + (j & (B.page_size - 1)) * B.slot_stride + kh * B.head_stride;
  };
  // is a value not finite at a key of the item that this row does not see?  (Else the row has
  // what its own keys give, and thousands of rows may see one such value.)
  const int first = (t - t0) / p.c.per_item * p.c.per_item, last = min(n, first + p.c.per_item) - 1;
  bool spoilt = false;
  auto look = [&](int from, int to) {
#pragma unroll 4
    for (int j = from; j < to; ++j) {
      const long long at = row_of(j);
      if (at < 0) continue;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float2 v = Pair<T>::get(reinterpret_cast<const uint32_t*>(static_cast<const T*>(p.v_raw) + at)[lane + 32 * w]);
        spoilt |= !isfinite(v.x) || !isfinite(v.y);
      }
    }
  };
  look(max(0, pos + 1), m - n + last + 1);
  if (p.c.window > 0) look(max(p.c.sinks, m - n + first - p.c.window + 1), lo);
  if (!__any_sync(0xFFFFFFFFu, spoilt)) return;
  float q[2 * W], o[2 * W] = {}, mx = -INFINITY, l = 0.0f;
  const uint32_t* qr = reinterpret_cast<const uint32_t*>(static_cast<const T*>(p.q_raw) + t * p.q_stride + h * D);
#pragma unroll
  for (int w = 0; w < W; ++w) {
    const float2 v = Pair<T>::get(qr[lane + 32 * w]);
    q[2 * w] = v.x, q[2 * w + 1] = v.y;
  }
  for (int i = 0; i < sinks + pos + 1 - lo; ++i) {  // the sinks, then the window
    const int j = i < sinks ? i : lo + i - sinks;
    const long long at = row_of(j);
    if (at < 0) continue;
    const uint32_t* kr = reinterpret_cast<const uint32_t*>(static_cast<const T*>(p.k_raw) + at);
    const uint32_t* vr = reinterpret_cast<const uint32_t*>(static_cast<const T*>(p.v_raw) + at);
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float2 k = Pair<T>::get(kr[lane + 32 * w]);
      s = fmaf(q[2 * w], k.x, fmaf(q[2 * w + 1], k.y, s));
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
    s *= p.scale_log2;
    const float top = fmaxf(mx, s);
    const float f = mx == -INFINITY ? 0.0f : exp2f(mx - top), e = s == -INFINITY ? 0.0f : exp2f(s - top);
    l = l * f + e;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float2 v = Pair<T>::get(vr[lane + 32 * w]);
      o[2 * w] = fmaf(o[2 * w], f, e * v.x), o[2 * w + 1] = fmaf(o[2 * w + 1], f, e * v.y);
    }
    mx = top;
  }
  const long long row = static_cast<long long>(t) * B.heads + h;
  float fold = 0.0f, f = 1.0f;
  if (p.flat_o) {
    const float z = p.flat_lse[row], top = fmaxf(mx, z);
    f = mx == -INFINITY ? 0.0f : exp2f(mx - top);
    fold = z == -INFINITY ? 0.0f : exp2f(z - top);
    l = l * f + fold;
    mx = top;
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<T*>(p.out) + t * p.out_stride + h * D);
#pragma unroll
  for (int w = 0; w < W; ++w) {
    float x = o[2 * w] * f, y = o[2 * w + 1] * f;
    if (fold != 0.0f) {
      const float2 v = *reinterpret_cast<const float2*>(p.flat_o + row * D + 2 * (lane + 32 * w));
      x = fmaf(v.x, fold, x), y = fmaf(v.y, fold, y);
    }
    dst[lane + 32 * w] = Pair<T>::put(x * inv, y * inv);
  }
  if (lane == 0) put_lse(p, row, mx, l);
}

// Joins the pieces of the items that several CTAs of cs_kv_attn_kernel share, a row to a
// warp, D / 32 dimensions to a lane:  O = sum_i 2^(m_i - m) O_i / sum_i 2^(m_i - m) l_i.
// A kernel of its own, because one SM joining ten pieces of 256 rows took 20 us and more
// while the others were done.  Bound by the latency of a row's reads (L2, mostly), so
// all of them start at once.  304 pieces of 256 rows (41 MB, out of DRAM): 21 us, less right
// behind the attention, when they lie in L2.  Then it mends the rows that were marked.
constexpr int JOIN_THREADS = 256;  // at least the grid of cs_kv_attn_kernel
constexpr int JOIN_CTAS = 4;  // per SM
template <typename T, int D>
__global__ void __launch_bounds__(JOIN_THREADS, JOIN_CTAS) cs_kv_join_kernel(const __grid_constant__ AttnP p) {
  __shared__ int before[JOIN_THREADS + 1], sums[JOIN_THREADS / 32];
  __shared__ Split splits[JOIN_THREADS];
  cs::grid_dep_wait();
  cs::grid_dep_launch_dependents();
  const Batch& B = p.b;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // rows of the items that are split, in the order of the CTAs that they start in
  splits[tid].pieces = 0;
  if (tid < p.num_splits) splits[tid] = p.splits[tid];
  const bool mend = !p.c.flat && __ldcg(&B.ctrl[CTRL_MEND]) != 0;
  const int mine = splits[tid].pieces ? splits[tid].tokens * B.group : 0;
  int incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xFFFFFFFFu, incl, d);
    if (lane >= d) incl += o;
  }
  if (lane == 31) sums[warp] = incl;
  __syncthreads();
  for (int w = 0; w < warp; ++w) incl += sums[w];
  before[tid + 1] = incl;
  if (tid == 0) before[0] = 0;
  __syncthreads();
  const int total = before[JOIN_THREADS];
  for (int n = blockIdx.x * (JOIN_THREADS / 32) + warp; n < total; n += gridDim.x * (JOIN_THREADS / 32)) {
    int c0 = 0, e = JOIN_THREADS;  // before[c0] <= n < before[e]
    while (e - c0 > 1) {
      const int mid = (c0 + e) >> 1;
      if (before[mid] <= n)
        c0 = mid;
      else
        e = mid;
    }
    const Split sp = splits[c0];
    const int t = (n - before[c0]) / B.group, h = n - before[c0] - t * B.group;  // token of the item, head of the group
    const int tile = t >= p.per_tile, r = (t - tile * p.per_tile) * B.group + h;
    auto piece = [&](int c) { return piece_state<D>(p.part, c0 + c, c == 0 && sp.first, tile, r); };
    // the pieces in their order, 32 at a time: a lane reads one's maximum and sum, while
    // the outputs of the first few are on their way
    constexpr int W = D / 32, AHEAD = 4;
    using Part = typename std::conditional<W == 4, float4, float2>::type;
    float x[W] = {}, l = 0.0f, m = -INFINITY;
    for (int i0 = 0; i0 < sp.pieces; i0 += 32) {
      const int here = min(32, sp.pieces - i0);
      float2 ml = make_float2(-INFINITY, 0.0f);
      if (lane < here) ml = __ldcg(reinterpret_cast<const float2*>(piece(i0 + lane) + D));
      auto output = [&](int i) { return __ldcg(reinterpret_cast<const Part*>(piece(i0 + i)) + lane); };
      Part y[AHEAD];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i)
        if (i < here) y[i] = output(i);
      float top = ml.x;
#pragma unroll
      for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
      top = fmaxf(top, m);
      const float old = m == -INFINITY ? 0.0f : cs::ex2_approx(m - top);
      const float weight = ml.x == -INFINITY ? 0.0f : cs::ex2_approx(ml.x - top);
      m = top;
      float sum = ml.y * weight;
#pragma unroll
      for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
      l = fmaf(l, old, sum);
#pragma unroll
      for (int w = 0; w < W; ++w) x[w] *= old;
      auto add = [&](int i, const Part& z) {
        const float f = __shfl_sync(0xFFFFFFFFu, weight, i);
#pragma unroll
        for (int w = 0; w < W; ++w) x[w] = fmaf(reinterpret_cast<const float*>(&z)[w], f, x[w]);
      };
#pragma unroll
      for (int i = 0; i < AHEAD; ++i)
        if (i < here) add(i, y[i]);
#pragma unroll 4
      for (int i = AHEAD; i < here; ++i) add(i, output(i));
    }
    const long long tok = sp.token + t, row = tok * B.heads + sp.kvh * B.group + h;
    if (!p.c.flat && p.flat_o) {  // join the prefix's output
      const float z = p.flat_lse[row], top = fmaxf(m, z);
      const float own = m == -INFINITY ? 0.0f : cs::ex2_approx(m - top), fold = z == -INFINITY ? 0.0f : cs::ex2_approx(z - top);
#pragma unroll
      for (int w = 0; w < W; ++w) x[w] = x[w] * own + p.flat_o[row * D + lane * W + w] * fold;
      l = l * own + fold;
      m = top;
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    if (p.c.flat) {
#pragma unroll
      for (int w = 0; w < W; ++w) p.flat_o[row * D + lane * W + w] = x[w] * inv;
    } else {
      uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<T*>(p.out) + tok * p.out_stride +
                                                  (sp.kvh * B.group + h) * D) + lane * (W / 2);
#pragma unroll
      for (int w = 0; w < W; w += 2) dst[w / 2] = Pair<T>::put(x[w] * inv, x[w + 1] * inv);
    }
    if (lane == 0) put_lse(p, row, m, l);
    float probe = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) probe = fmaf(x[w], 0.0f, probe);
    if (!p.c.flat && __any_sync(0xFFFFFFFFu, probe != 0.0f) && isfinite(l)) {
      __syncwarp();
      mend_row<T, D>(p, static_cast<int>(tok), sp.kvh * B.group + h);
    }
  }
  if (!mend) return;
  const long long all = static_cast<long long>(B.tokens) * B.heads;
  for (long long n = static_cast<long long>(blockIdx.x) * (JOIN_THREADS / 32) + warp; n < all;
       n += gridDim.x * (JOIN_THREADS / 32)) {
    if (p.mend[n] == 0) continue;
    __syncwarp();
    mend_row<T, D>(p, static_cast<int>(n / B.heads), static_cast<int>(n % B.heads));
    if (lane == 0) p.mend[n] = 0;
  }
  __syncthreads();
  if (tid == 0 && atomicAdd(&B.ctrl[CTRL_MENDED], 1u) == gridDim.x - 1) {  // every block has read the flag
    B.ctrl[CTRL_MENDED] = 0;
    B.ctrl[CTRL_MEND] = 0;
  }
}

// WINDOW: whether keys may be hidden behind a row's window (without, what deals with it is
// not in the code of the inner loops)
template <typename T, int D, bool WINDOW>
__global__ void __launch_bounds__(ATTN_THREADS, 1) cs_kv_attn_kernel(const __grid_constant__ AttnP p) {
  using Sh = AttnShape<D>;
  using Ctl = AttnCtl<Sh::SLOTS>;
  static_assert(sizeof(Ctl) <= CTL, "control block");
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* qbuf = smem;
  uint8_t* ring = smem + 2 * Sh::TILE;
  Ctl* sc = reinterpret_cast<Ctl*>(ring + Sh::SLOTS * Sh::TILE);
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int i = 0; i < Sh::SLOTS; ++i) {
      cs::mbar_init(&sc->full[i], 1);
      cs::mbar_init(&sc->empty[i], 2);  // both MMA warps
    }
    for (int w = 0; w < 2; ++w) {
      cs::mbar_init(&sc->q_full[w], 1);
      cs::mbar_init(&sc->q_empty[w], w == 0 ? 2 : 1);
      cs::mbar_init(&sc->s_full[w], 1);
      for (int h = 0; h < 2; ++h) cs::mbar_init(&sc->p_full[w][h], 4);  // the warps of its warpgroup
      cs::mbar_init(&sc->o_full[w], 1);
      cs::mbar_init(&sc->v_ready[w], 1);
    }
    cs::mbar_init(&sc->other_full, 128);
    cs::mbar_init(&sc->other_empty, 128);
    cs::mbar_init(&sc->drained, 2);
    sc->abort = sc->turn = sc->loads = sc->q_loads[0] = sc->q_loads[1] = 0;
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
  if (threadIdx.x == 0) p.splits[blockIdx.x].pieces = 0;
  find_range<ATTN_THREADS>(p.b, p.c, &sc->range, sc->scratch);
  constexpr int bf16 = sizeof(T) == 2 && !std::is_same<T, __half>::value;
  if (warp < 8) {
    regs_inc<SOFTMAX_REGS>();
    // (a softmax that gave up may have stores to tensor memory on their way)
    if (!softmax_role<T, D, WINDOW>(p, sc, ring, warp >> 2)) cs::tc_wait_st();
  } else {
    regs_dec<OTHER_REGS>();
    if (warp == 8) load_role<D>(p, sc, qbuf, ring);
    if (warp == 9 || warp == 10) mma_role<D, WINDOW>(p, sc, qbuf, ring, bf16, warp - 9);
  }
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
