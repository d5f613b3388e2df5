// Attention over the paged cache for few rows per key head (single tokens, or a few):
// at most 16 (token, query head) rows of a sequence read each key, so the keys' and
// values' bytes bound it, and for short contexts the latency.
//
// An item is the rows of one sequence and key head, a tile 64 keys: 16 for each of a
// CTA's warps, which has them copied (one TMA box for K, one for V) for itself, so that no
// barrier of the CTA lies on the way.  The order of the contracted dimensions of a product is
// free as long as both operands agree on it, so each lane's part of the m16n8k16
// fragments is 16 consecutive bytes: of K, of the key that is its column; of V, of
// its four keys.  Each warp has its own running maximum and sum; they are joined
// in shared memory at the end, and the pieces of an item by the last of its CTAs to
// store one (in their order, so that the result does not depend on which that is).
// mma.sync, because 16 rows would leave 7/8 of a tcgen05 tile of 128 empty; its rate is no
// bound here.
//
// 64 single tokens over 300 to 32000 keys, 64 / 8 heads of 128 (4.26 GB of keys and values):
// 664 to 692 us on several cards, 6.2 to 6.4 TB/s, 0.91 to 0.95 of a plain copy's measured 6.8;
// DRAM bounds it.  (The tensor-core kernel, whose rows are nearly all empty here, measured 662
// us when it still took this case: over long contexts either is at the memory's rate.  What
// this kernel is for is the rest: one user's token 31.6 us with that kernel, 135 under the
// window.)  128 single tokens under a window of 1024: 93 us, 5.7 TB/s; one user's token over
// 978 keys, 12 heads: 8.9 us, launch, lookups, a tile's latency and the joining one after
// another.  With 16 rows the joins count: 8 sequences of up to 4 tokens over up to 2000 keys
// take 26 us where single tokens take 16 (38 with one dimension a thread; reading all
// of a thread's rows at once needs 540 bytes of spills, and everything is slower).
// Fetching a segment's first tiles while the one before is joined was slower (decode over
// long contexts 690 -> 703 us, one user's 9.3 -> 10.1): it needs registers
// that the inner loop has not got, and three CTAs an SM cover for each other already.
#pragma once
#include <climits>

#include "cs_kv_attn.cuh"

namespace cskv {

constexpr int ROWS = 16;         // rows of an item
constexpr int ROWS_SHIFT = 6;     // keys of a tile: 64
constexpr int ROWS_WARPS = (1 << ROWS_SHIFT) / 16;  // 16 keys each
constexpr int ROWS_THREADS = 32 * ROWS_WARPS;
constexpr int ROWS_CTAS = 12 / ROWS_WARPS;  // per SM: 12 warps (168 registers a thread) with up to 16 KB in flight each

template <typename T>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  if constexpr (std::is_same<T, __half>::value)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <int D>
struct alignas(1024) RowsShared {
  static constexpr int STAGES = D == 128 ? 2 : 4;  // tiles on their way
  union {
    // [warp][stage][K, V][8-key group][64-dimension half][key][16-byte piece, at its index ^ key]
    uint4 kv[ROWS_WARPS][STAGES][2][2][D / 64][8][8];
    float o[ROWS_WARPS][ROWS][D + 4];        // each warp's output
    float sum[ROWS][D + 4];                  // of a part of an item's pieces: output, maximum, sum
  };
  Range range;
  unsigned long long scratch[ROWS_THREADS / 32];
  int last;
  volatile int abort;  // a wait ran out
  uint64_t full[ROWS_WARPS][STAGES][2];  // [warp][stage][K, V]
  float2 ml[ROWS_WARPS][ROWS];  // each warp's maximum and sum of a row
  uint4 q[ROWS][D / 8 + 1];
};

// How many copies of K (which 0) or V (1) a warp has issued into a stage when it waits for K
// (or, at_values, V) of its tile number `done`, `left` tiles before its segment's end: ST tiles
// are on their way, and K of the next one as soon as K of this one is read.
template <int ST>
CS_KV_BOTH uint32_t rows_issued(int which, int stage, bool at_values, uint32_t done, int left) {
  const uint32_t n = done + kv_min(left, ST) + (which == 0 && at_values && left > ST);
  return (n - stage + ST - 1) / ST;
}

template <typename T, int D>
__global__ void __launch_bounds__(ROWS_THREADS, ROWS_CTAS) cs_kv_rows_kernel(const __grid_constant__ AttnP p) {
  extern __shared__ __align__(1024) uint8_t rows_smem[];
  RowsShared<D>& sm =
      *reinterpret_cast<RowsShared<D>*>((reinterpret_cast<uintptr_t>(rows_smem) + 1023) & ~uintptr_t(1023));
  constexpr int ST = RowsShared<D>::STAGES;
  if (threadIdx.x == 0) {
    for (int i = 0; i < ROWS_WARPS * ST * 2; ++i) cs::mbar_init(&sm.full[0][0][0] + i, 1);
    sm.abort = 0;
    cs::fence_mbar_init();
    cs::prefetch_tmap(&p.k);
    cs::prefetch_tmap(&p.v);
  }
  // After a prefix's phase, all but the folding in of its result goes on beside the end of
  // that phase: whatever came before it was complete when it let this grid start, and
  // pieces and counters are other ones.  Every thread waits before it ends.
  const bool late = !p.c.flat && p.flat_o;
  if (!late) cs::grid_dep_wait();
  cs::grid_dep_launch_dependents();
  const Batch& B = p.b;
  find_range<ROWS_THREADS>(B, p.c, &sm.range, sm.scratch);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gq = lane >> 2, jq = lane & 3;
  constexpr int KB = D / 32, VB = D / 64;  // 16-byte pieces of a key per lane, of each of its four values
  uint32_t done = 0;  // tiles that this warp has read
  // a copy of this warp; one that never comes (an error) is waited for with a limit, and
  // then all warps give up
  auto arrived = [&](int which, uint32_t n) { return wait_warp(&sm.full[warp][n % ST][which], n / ST & 1u, &sm); };
  Walk walk(p.c, sm.range);
  Seg g;
  while (walk.next(B, p.c, g)) {
    const int first = g.item * p.c.per_item;  // the item's first token
    const int rows = min(p.c.per_item, g.s.n - first) * B.group;
    const int* table = p.c.flat ? p.pages : B.table + static_cast<long long>(g.b) * B.table_cols;
    cs::fence_proxy_async_shared();
    __syncthreads();  // shared memory of the segment before is read
    constexpr int QN = ROWS * (D / 8) / ROWS_THREADS;  // 16-byte pieces of the queries per thread
    uint4 qv[QN];
#pragma unroll
    for (int i = 0; i < QN; ++i) {
      const int x = tid + i * ROWS_THREADS, r = x / (D / 8), c = x % (D / 8);
      qv[i] = make_uint4(0, 0, 0, 0);
      if (r < rows) {
        const int t = r / B.group;
        qv[i] = *(reinterpret_cast<const uint4*>(static_cast<const T*>(p.q_raw) + (g.s.t0 + first + t) * p.q_stride +
                                                 (g.kvh * B.group + r - t * B.group) * D) + c);
      }
    }
    // keys [.., end) and from lo on, or below the sinks, are seen by rows gq and gq + 8
    int end[2], lo[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int r = gq + 8 * x, pos = g.s.m - g.s.n + first + r / B.group;
      end[x] = r >= rows ? 0 : p.c.flat ? g.s.m : pos + 1;
      lo[x] = p.c.window > 0 ? max(0, pos + 1 - p.c.window) : 0;
    }
    auto seen = [&](int key) { return key < g.hi && (key >= g.lo || key < p.c.sinks); };  // by some row
    // this warp's page of tile k, -1 if none of its keys is seen
    auto table_of = [&](int k) {
      if (k >= g.k1) return -1;
      const int j0 = g.key0(p.c, k) + warp * 16;
      if (j0 >= g.hi || (j0 + 16 <= g.lo && j0 >= p.c.sinks)) return -1;
      const int page = __ldg(table + (j0 >> B.page_shift));
      return page < 0 ? INT_MAX : page;
    };
    auto checked = [&](int page) {
      if (page < B.num_pages) return page;
      record(B.ctrl, ERR_INVALID, WHAT_PAGE, p.c.flat ? 0xFFFFFFFFu : static_cast<uint32_t>(g.b));
      return -1;
    };
    auto load = [&](int which, int k, int page, uint32_t n) {  // n: the warp's tile
      if (k >= g.k1 || lane != 0) return;
      uint64_t* bar = &sm.full[warp][n % ST][which];
      if (page < 0) {  // nothing to read
        cs::mbar_arrive(bar);
        return;
      }
      const int group = ((g.key0(p.c, k) + warp * 16) & (B.page_size - 1)) >> 3;
      const int c4 = p.head_groups ? (page * B.kv_heads + g.kvh) * p.head_groups + group : page * (B.page_size >> 3) + group;
      cs::mbar_arrive_expect_tx(bar, 16 * D * 2);
      tma_5d(&sm.kv[warp][n % ST][which], which ? &p.v : &p.k, 0, 0, 0, p.head_groups ? 0 : g.kvh, c4, bar);
    };
    int ahead[ST + 1];
#pragma unroll
    for (int i = 0; i <= ST; ++i) ahead[i] = table_of(g.k0 + i);
#pragma unroll
    for (int i = 0; i < ST; ++i) {
      const int page = checked(ahead[i]);
      load(0, g.k0 + i, page, done + i);
      load(1, g.k0 + i, page, done + i);
    }
    int next = ahead[ST];
    float o[VB][8][4];
#pragma unroll
    for (int h = 0; h < VB; ++h)
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[h][i][c] = 0.0f;
    float m_ref[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < QN; ++i) {
      const int x = tid + i * ROWS_THREADS;
      sm.q[x / (D / 8)][x % (D / 8)] = qv[i];
    }
    __syncthreads();  // the queries are there
    int k = g.k0;
    bool at_values = false;
#pragma unroll 1
    for (; k < g.k1; ++k) {
      const int j0 = g.key0(p.c, k) + warp * 16;
      const int page = checked(next);  // of tile k + ST
      next = table_of(k + ST + 1);
      const int stage = done % ST;
      if (!arrived(0, done)) break;
      float s[2][4] = {};
#pragma unroll
      for (int i = 0; i < KB; ++i) {
        const uint4 qa = sm.q[gq][4 * i + jq], qb = sm.q[gq + 8][4 * i + jq];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const uint4 kr = sm.kv[warp][stage][0][b][i >> 1][gq][(4 * (i & 1) + jq) ^ gq];
          mma16816<T>(s[b], qa.x, qb.x, qa.y, qb.y, kr.x, kr.y);
          mma16816<T>(s[b], qa.z, qb.z, qa.w, qb.w, kr.z, kr.w);
        }
      }
      __syncwarp();
      load(0, k + ST, page, done + ST);
      bool raise = false;
      float f[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float mx = -INFINITY;
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int key = j0 + 8 * b + 2 * jq + e;
            float& y = s[b][2 * x + e];
            y = key < end[x] && (key >= lo[x] || key < p.c.sinks) ? y * p.scale_log2 : -INFINITY;
            mx = fmaxf(mx, y);
          }
        mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
        // the reference is raised only when it is exceeded by more than 2^8
        const bool up = mx > m_ref[x] + RAISE_LOG2 || (m_ref[x] == -INFINITY && mx > -INFINITY);
        f[x] = up ? cs::ex2_approx(m_ref[x] - mx) : 1.0f;
        if (up) m_ref[x] = mx;
        raise |= up;
      }
      if (__any_sync(0xFFFFFFFFu, raise)) {
#pragma unroll
        for (int h = 0; h < VB; ++h)
#pragma unroll
          for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) o[h][i][c] *= f[c >> 1];
        l[0] *= f[0];
        l[1] *= f[1];
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float sub = m_ref[x] == -INFINITY ? 0.0f : m_ref[x];
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            s[b][2 * x + e] = cs::ex2_approx(s[b][2 * x + e] - sub);
            l[x] += s[b][2 * x + e];
          }
      }
      const uint32_t a0 = Pair<T>::put(s[0][0], s[0][1]), a1 = Pair<T>::put(s[0][2], s[0][3]);
      const uint32_t a2 = Pair<T>::put(s[1][0], s[1][1]), a3 = Pair<T>::put(s[1][2], s[1][3]);
      if (!arrived(1, done)) {
        at_values = true;
        break;
      }
      // values of keys that no row sees may be anything: zeros instead
      const bool part = j0 + 16 > g.hi || (j0 < g.lo && j0 + 16 > p.c.sinks);
#pragma unroll
      for (int h = 0; h < VB; ++h) {
        uint32_t v0[4], v1[4], v2[4], v3[4];
        *reinterpret_cast<uint4*>(v0) = sm.kv[warp][stage][1][0][h][2 * jq][gq ^ 2 * jq];
        *reinterpret_cast<uint4*>(v1) = sm.kv[warp][stage][1][0][h][2 * jq + 1][gq ^ (2 * jq + 1)];
        *reinterpret_cast<uint4*>(v2) = sm.kv[warp][stage][1][1][h][2 * jq][gq ^ 2 * jq];
        *reinterpret_cast<uint4*>(v3) = sm.kv[warp][stage][1][1][h][2 * jq + 1][gq ^ (2 * jq + 1)];
        if (part) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (!seen(j0 + 2 * jq)) v0[e] = 0;
            if (!seen(j0 + 2 * jq + 1)) v1[e] = 0;
            if (!seen(j0 + 2 * jq + 8)) v2[e] = 0;
            if (!seen(j0 + 2 * jq + 9)) v3[e] = 0;
          }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {  // column n of this MMA is dimension 8 n + i of the half
          const uint32_t pick = i & 1 ? 0x7632u : 0x5410u;
          mma16816<T>(o[h][i], a0, a1, a2, a3, __byte_perm(v0[i >> 1], v1[i >> 1], pick),
                      __byte_perm(v2[i >> 1], v3[i >> 1], pick));
        }
      }
      __syncwarp();
      load(1, k + ST, page, done + ST);
      ++done;
    }
    if (__builtin_expect(k < g.k1, 0) && lane == 0) {  // gave up: the copies on their way come to rest, with a limit
      int tries = 0;
#pragma unroll 1
      for (int i = 0; i < 2 * ST; ++i) {
        const uint32_t n = rows_issued<ST>(i & 1, i >> 1, at_values, done, g.k1 - k);
        while (n > 0 && !cs::mbar_try_wait(&sm.full[warp][i >> 1][i & 1], (n - 1) & 1u) && ++tries < SETTLE_TRIES) {
        }
      }
    }
    __syncthreads();  // every warp is done with its operands' memory
    if (sm.abort) {  // a warp can set it before this barrier or behind the next one only
      if (tid == 0) record(B.ctrl, ERR_WATCHDOG, WHAT_WAIT, blockIdx.x);
      break;
    }
    // the warps' states to shared memory
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      l[x] += __shfl_xor_sync(0xFFFFFFFFu, l[x], 1);
      l[x] += __shfl_xor_sync(0xFFFFFFFFu, l[x], 2);
      const int r = gq + 8 * x;
      if (r < rows) {
        if (jq == 0) sm.ml[warp][r] = make_float2(m_ref[x], l[x]);
#pragma unroll
        for (int h = 0; h < VB; ++h)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float4* to = reinterpret_cast<float4*>(&sm.o[warp][r][8 * (2 * jq + e + 8 * h)]);
            to[0] = make_float4(o[h][0][2 * x + e], o[h][1][2 * x + e], o[h][2][2 * x + e], o[h][3][2 * x + e]);
            to[1] = make_float4(o[h][4][2 * x + e], o[h][5][2 * x + e], o[h][6][2 * x + e], o[h][7][2 * x + e]);
          }
      }
    }
    __syncthreads();
    auto state = [&](unsigned cta, int which, int r) { return p.part + ((static_cast<size_t>(cta) * 2 + which) * ROWS + r) * (D + 4); };
    // dimensions 4 c .. 4 c + 3 of row r from their state
    auto finish = [&](int r, int c, float4 x, float m, float l) {
      const int t = r / B.group;
      const long long row = static_cast<long long>(g.s.t0 + first + t) * B.heads + g.kvh * B.group + r - t * B.group;
      float4* const pre = p.flat_o ? reinterpret_cast<float4*>(p.flat_o + row * D) + c : nullptr;
      if (!p.c.flat && pre) {  // join the prefix's output
        const float z = p.flat_lse[row], top = fmaxf(m, z);
        const float own = m == -INFINITY ? 0.0f : cs::ex2_approx(m - top), fold = z == -INFINITY ? 0.0f : cs::ex2_approx(z - top);
        const float4 y = *pre;
        x = make_float4(x.x * own + y.x * fold, x.y * own + y.y * fold, x.z * own + y.z * fold, x.w * own + y.w * fold);
        l = l * own + fold;
        m = top;
      }
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
      const float4 y = l == 0.0f ? make_float4(0.0f, 0.0f, 0.0f, 0.0f) : make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv);
      const float probe = fmaf(x.x, 0.0f, fmaf(x.y, 0.0f, fmaf(x.z, 0.0f, x.w * 0.0f)));  // NaN if one is not finite
      if (probe != 0.0f && isfinite(l) && g.s.n > 1) mark(p, row);  // several tokens: keys hidden from one only
      if (c == 0) put_lse(p, row, m, l);
      if (p.c.flat) {
        *pre = y;
      } else {
        uint2* out = reinterpret_cast<uint2*>(static_cast<T*>(p.out) + (g.s.t0 + first + t) * p.out_stride +
                                              (g.kvh * B.group + r - t * B.group) * D) + c;
        *out = make_uint2(Pair<T>::put(y.x, y.y), Pair<T>::put(y.z, y.w));
      }
    };
    auto add = [](float4& x, const float4& y, float f) {
      x.x = fmaf(y.x, f, x.x), x.y = fmaf(y.y, f, x.y), x.z = fmaf(y.z, f, x.z), x.w = fmaf(y.w, f, x.w);
    };
    constexpr int QUADS = D / 4;
    const bool whole = g.whole();
    if (late && whole) cs::grid_dep_wait();
    for (int i = tid; i < rows * QUADS; i += ROWS_THREADS) {
      const int r = i / QUADS, c = i % QUADS;
      float m = -INFINITY, sum = 0.0f;
      float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int w = 0; w < ROWS_WARPS; ++w) m = fmaxf(m, sm.ml[w][r].x);
#pragma unroll
      for (int w = 0; w < ROWS_WARPS; ++w) {
        const float2 ml = sm.ml[w][r];
        const float f = ml.x == -INFINITY ? 0.0f : cs::ex2_approx(ml.x - m);
        sum = fmaf(ml.y, f, sum);
        add(x, *reinterpret_cast<const float4*>(&sm.o[w][r][4 * c]), f);
      }
      if (whole) {
        finish(r, c, x, m, sum);
      } else {
        float* to = state(blockIdx.x, sm.range.x0 < g.x, r);
        reinterpret_cast<float4*>(to)[c] = x;
        if (c == 0) *reinterpret_cast<float2*>(to + D) = make_float2(m, sum);
      }
    }
    if (whole) continue;
    const unsigned me = blockIdx.x, quota = static_cast<unsigned>(min(sm.range.quota, 0x80000000ull));
    const unsigned long long end_x = g.x + g.tiles - 1;
    const unsigned c0 = sm.range.x0 > g.x ? me - (static_cast<unsigned>(sm.range.x0 - g.x) + quota - 1) / quota : me;
    const unsigned c1 = end_x >= sm.range.x1 ? me + static_cast<unsigned>(end_x - sm.range.x1) / quota + 1 : me;
    __syncthreads();  // all stores come before the one arrival at gpu scope
    if (tid == 0) {
      uint32_t* ctr = p.arrivals + c0;
      const uint32_t old = cs::atom_add_acq_rel_gpu(ctr, 1u);
      sm.last = old == c1 - c0;
      if (old == c1 - c0) *ctr = 0u;  // for the next call
    }
    __syncthreads();
    if (!sm.last) continue;
    if (late) cs::grid_dep_wait();
    // the last to arrive joins the pieces in their order
    const int pieces = static_cast<int>(c1 - c0) + 1;
    auto piece = [&](int i, int r) { return state(c0 + i, sm.range.quota * (c0 + i) < g.x, r); };
    // a warp (64 dimensions: half of one) sums a row over all pieces, or with few rows over a
    // part of them, a lane four dimensions; every lane knows the weights of 32 (16) pieces at a time
    constexpr int LANES = QUADS, UNITS = ROWS_THREADS / LANES, AHEAD = 3;  // a fourth is spilled, in the inner loop too
    static_assert(UNITS <= ROWS, "sums");
    const unsigned group = LANES == 32 ? 0xFFFFFFFFu : 0xFFFFu << (lane & 16);
    const int gl = lane % LANES;
    const int parts = rows >= UNITS ? 1 : UNITS / rows, per = (pieces + parts - 1) / parts;
    for (int u = tid / LANES; u < rows * parts; u += UNITS) {
      const int r = u % rows, part = u / rows, to = min(pieces, (part + 1) * per);
      float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      float sum = 0.0f, top = -INFINITY;
      for (int i0 = part * per; i0 < to; i0 += LANES) {
        const int here = min(LANES, to - i0);
        auto output = [&](int i) { return __ldcg(reinterpret_cast<const float4*>(piece(i0 + i, r)) + gl); };
        float2 ml = make_float2(-INFINITY, 0.0f);
        if (gl < here) ml = __ldcg(reinterpret_cast<const float2*>(piece(i0 + gl, r) + D));
        float4 y[AHEAD];  // on their way with the maxima and sums
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
          if (i < here) y[i] = output(i);
        float m = ml.x;
#pragma unroll
        for (int v = LANES / 2; v; v >>= 1) m = fmaxf(m, __shfl_xor_sync(group, m, v));
        m = fmaxf(m, top);
        const float old = top == -INFINITY ? 0.0f : cs::ex2_approx(top - m);
        const float weight = ml.x == -INFINITY ? 0.0f : cs::ex2_approx(ml.x - m);
        top = m;
        float l = ml.y * weight;
#pragma unroll
        for (int v = LANES / 2; v; v >>= 1) l += __shfl_xor_sync(group, l, v);
        sum = fmaf(sum, old, l);
        x.x *= old, x.y *= old, x.z *= old, x.w *= old;
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
          const float f = __shfl_sync(group, weight, i, LANES);
          if (i < here) add(x, y[i], f);
        }
#pragma unroll 4
        for (int i = AHEAD; i < here; ++i) add(x, output(i), __shfl_sync(group, weight, i, LANES));
      }
      reinterpret_cast<float4*>(sm.sum[u])[gl] = x;
      if (gl == 0) *reinterpret_cast<float2*>(&sm.sum[u][D]) = make_float2(top, sum);
    }
    __syncthreads();
    for (int i = tid; i < rows * QUADS; i += ROWS_THREADS) {
      const int r = i / QUADS, c = i % QUADS;
      float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      float l = 0.0f, top = -INFINITY;
      for (int part = 0; part < parts; ++part) top = fmaxf(top, sm.sum[part * rows + r][D]);
      for (int part = 0; part < parts; ++part) {
        const float m = sm.sum[part * rows + r][D], f = m == -INFINITY ? 0.0f : cs::ex2_approx(m - top);
        add(y, *reinterpret_cast<const float4*>(&sm.sum[part * rows + r][4 * c]), f);
        l = fmaf(sm.sum[part * rows + r][D + 1], f, l);
      }
      finish(r, c, y, top, l);
    }
  }
  if (late) cs::grid_dep_wait();
}

}  // namespace cskv
