// Attention over a paged cache in 4 bits for few rows per key head (single tokens, or a few):
// at most 16 (token, query head) rows of a sequence read each key.
//
// Items, tiles and joins are those of cs_kv_rows.cuh.  What differs: a key and its value are
// 2 x (head_dim / 2 + head_dim / 32) bytes, so that making operands of codes costs
// more than bringing them, and the products are turned round, S^T = K Q^T and O^T = V^T P^T:
// the cache is the operand of 16 rows, the queries' 8 columns are all that single tokens need,
// and each code is made an operand once for 8 (16) rows.
//
// Operands.  The order of the contracted dimensions is free as long as both operands agree on it.
// A lane (g, t) of S^T's first operand has 32 (16) consecutive dimensions of two keys, under one
// scale each; of V^T's it has 16 (8) dimensions of four keys: two keys' words, taken apart in
// 16-bit halves and put together by dimension, make pairs along the keys.  P^T is the second operand of O^T:
// an 8 x 8 transposition of S^T's accumulators (movmatrix).  The scores' operands are f16, whatever the
// cache's type is: a code is then a value after a mask and a multiply-add (FourScaled), values times 2^-7 are f16 numbers
// for every scale, and queries of bf16 are put to f16's range row by row.  The weights and V are of the cache's type:
// beside a key that takes nearly all the weight and whose value is about 0 (an attention sink) the others are the
// output, and f16 has no bits for weights below 2^-25 of the largest.  (With f16 for both types 64 sequences of 16000 keys
// took 239 us, now 244; 16000 keys 18 nats below one of value 0 on one SM lost those of that key's warp, 8 % of the output.)
//
// Row r of S^T's 8-row half is key r / 2 (r even) or 7 - r / 2 (r odd) of 8: with it all reads
// of the codes from shared memory are free of bank conflicts.
//
// Bound.  Instructions and their latency together: 338 (f16 318) for 16 keys of 128 dimensions and a warp, about half of them
// to make operands of codes, at 2.3 of 4 a cycle; no unit is full (the pipe of shifts, masks and byte selections is busy in 47 %
// of the cycles, DRAM in 53 %), and 12 warps an SM leave waits uncovered.
// 62 single tokens over 300 to 32000 keys, 64 / 8 heads of 128 (1.13 GB): 247 us, 4.6 TB/s, 0.68 of a plain copy's
// measured 6.8; the 16-bit cache (4.26 GB) takes 664 to 692.  32 x 4 tokens over 8000 keys, 32 / 8 heads of 128: 112 us (f16
// 107), over 16 bits 191.  128 tokens under a window of 1024, 40 / 8 heads of 64:
// 38.2 us, of which the start of a launch, its division and its last joins are about 13.  One user's token over 978
// keys, 12 heads: 9.1 us, the latency of its steps, as over the 16-bit cache; over 16000 keys, 8 heads: 25.5.
// Slower or no faster: the next keys' scores before the softmax of these (267 us for 64 sequences of 16000 keys where it
// took 243), leaving out runs that no row sees (251), items' first copies sent off while the item before is stored (81
// and 81 us for 256000 keys), runs one by one in half the code (84), right shifts as products' upper halves (96),
// prefetches of whole lines, five CTAs an SM (98), two with 16 columns (118 and 114).
#pragma once
#include <cfloat>

#include "cs_kv_rows.cuh"

namespace cskv {

// CTAs of four warps per SM.  Three leave a thread 168 registers, four 128, into which 8 columns just fit; at 128 dimensions
// independent work is worth more than warps (64 sequences of 16000 keys 247 us with three, 261 with four), at 64 it
// is not (182 and 171).  With 16 columns at 128 dimensions three CTAs spill 70 to 120 bytes a thread, and are
// faster than two without spills (114 and 118).
template <int D, int NT>
constexpr int ROWS4_CTAS = D == 64 && NT == 1 ? 4 : 3;

constexpr int ROWS4_SHIFT = 7;  // keys of a tile: 128, two runs of 16 for each warp, 64 apart

// A row's reference lies 2^7 below a score of its own, so its weights are at most 2^15: as far from f16's end as that
// goes, and 2^7 more of what f16 has at its other end.
constexpr float WEIGHT_LOG2 = 7.0f;
// Beyond +-2^20 a reference in 32 bits is off by more than a sixteenth, and the multiply-add, which rounds once, would show it
// in the weights: there scores are taken off one another before the factor.
constexpr float FAR_LOG2 = 1048576.0f;

template <int D>
struct Stage4 {  // a warp's keys of a tile: codes of K and V, their scales
  uint8_t codes[2][32][D / 2];
  uint8_t scales[2][32][D / GROUP4];
};

template <int D>
struct alignas(16) Rows4Shared {
  static constexpr int STAGES = D == 128 ? 3 : 6;  // 9 to 11 KB on their way for each warp
  union {
    Stage4<D> ring[ROWS_WARPS][STAGES];
    float o[ROWS_WARPS][ROWS][D + 4];  // each warp's output
    float piece[6 * ROWS][D + 4];      // rows of pieces of an item on their way: outputs, maxima, sums
  };
  Range range;
  unsigned long long scratch[ROWS_THREADS / 32];
  int last;
  float2 ml[ROWS_WARPS][ROWS];  // each warp's maximum and sum of a row
};

// 16 bytes to shared memory, zeros where nothing is to be read.
__device__ __forceinline__ void copy16(void* dst, const void* src, bool read) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(cs::smem_u32(dst)), "l"(src), "r"(read ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// 8 x 8 transposition of 16-bit values
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Joins the pieces of an item in their order: outputs go by way of shared memory, four (two) at a time while eight
// (four) more are on their way, and the lanes of a row know the weights of 32 (16) pieces at a time, so that a
// piece costs a read and four multiply-adds.  (With loads into registers, few at a time because the loop over the
// keys spills what more of them would need, and a running maximum, 63 pieces of 8 rows took over 20 us.)
template <typename T, int D, int NT>
__device__ __forceinline__ void join4(const AttnP& p, const Seg& g, int first, int rows, const Pieces& of, Rows4Shared<D>& sm) {
  constexpr int QUADS = D / 4, MINE = NT * 8 * QUADS / ROWS_THREADS;  // QUADS lanes for a row, MINE rows for a lane
  constexpr int BATCH = 4 / NT, SLOTS = 3 * BATCH;
  const int tid = threadIdx.x, lane = tid & 31, gl = lane % QUADS, r0 = tid / QUADS;
  const unsigned group = QUADS == 32 ? 0xFFFFFFFFu : 0xFFFFu << (lane & 16);
  auto piece = [&](int i, int r) {
    const unsigned cta = of.first + i;
    return rows_state<D>(p, cta, sm.range.quota * (cta - sm.range.cta) < g.x, r);
  };
  auto load = [&](int i) {  // a batch from piece i on: a lane copies what it reads
#pragma unroll 1
    for (int j = i; j < min(i + BATCH, of.count); ++j)
#pragma unroll
      for (int n = 0; n < MINE; ++n) {
        const int r = r0 + n * (ROWS_THREADS / QUADS);
        if (r < rows) copy16(&sm.piece[j % SLOTS * 8 * NT + r][4 * gl], piece(j, r) + 4 * gl, true);
      }
    copies_commit();
  };
  float4 x[MINE];
  float m[MINE], l[MINE], weight[MINE];
#pragma unroll
  for (int n = 0; n < MINE; ++n) x[n] = make_float4(0.0f, 0.0f, 0.0f, 0.0f), m[n] = -INFINITY, l[n] = 0.0f;
  load(0);
  load(BATCH);
#pragma unroll 1
  for (int i = 0; i < of.count; i += BATCH) {
    if (i % QUADS == 0) {  // the weights of the next pieces
#pragma unroll
      for (int n = 0; n < MINE; ++n) {
        const int r = r0 + n * (ROWS_THREADS / QUADS);
        float2 ml = make_float2(-INFINITY, 0.0f);
        if (r < rows && i + gl < of.count) ml = __ldcg(reinterpret_cast<const float2*>(piece(i + gl, r) + D));
        float top = ml.x;
#pragma unroll
        for (int v = QUADS / 2; v; v >>= 1) top = fmaxf(top, __shfl_xor_sync(group, top, v));
        top = fmaxf(top, m[n]);
        const float old = m[n] == -INFINITY ? 0.0f : cs::ex2_approx(m[n] - top);
        weight[n] = ml.x == -INFINITY ? 0.0f : cs::ex2_approx(ml.x - top);
        m[n] = top;
        float sum = ml.y * weight[n];
#pragma unroll
        for (int v = QUADS / 2; v; v >>= 1) sum += __shfl_xor_sync(group, sum, v);
        l[n] = fmaf(l[n], old, sum);
        x[n].x *= old, x[n].y *= old, x[n].z *= old, x[n].w *= old;
      }
    }
    load(i + 2 * BATCH);
    copies_wait<2>();  // this lane's own copies: no barrier
#pragma unroll
    for (int j = 0; j < BATCH; ++j)
#pragma unroll
      for (int n = 0; n < MINE; ++n) {
        const int r = r0 + n * (ROWS_THREADS / QUADS);
        const float f = __shfl_sync(group, weight[n], (i + j) % QUADS, QUADS);
        if (r < rows && i + j < of.count)
          add_weighted(x[n], *reinterpret_cast<const float4*>(&sm.piece[(i + j) % SLOTS * 8 * NT + r][4 * gl]), f);
      }
  }
  copies_wait<0>();
#pragma unroll
  for (int n = 0; n < MINE; ++n) {
    const int r = r0 + n * (ROWS_THREADS / QUADS);
    if (r < rows) rows_finish<T, D>(p, g, first, r, gl, x[n], m[n], l[n]);
  }
}

// NT: groups of 8 rows
template <typename T, int D, int NT, bool BY_HEAD>
__global__ void __launch_bounds__(ROWS_THREADS, ROWS4_CTAS<D, NT>) cs_kv4_rows_kernel(const __grid_constant__ AttnP p) {
  extern __shared__ __align__(1024) uint8_t rows_smem[];
  Rows4Shared<D>& sm = *reinterpret_cast<Rows4Shared<D>*>(rows_smem);
  constexpr int ST = Rows4Shared<D>::STAGES;
  constexpr int KW = D / 32, VW = D / 64;   // 32-bit words of a key per lane, of each of its four values
  constexpr int XS = NT == 1 ? 2 : 1;       // runs of 16 keys whose scores are computed together (16 rows: registers)
  const bool late = !p.c.flat && p.flat_o;  // as in cs_kv_rows_kernel
  if (!late) cs::grid_dep_wait();
  cs::grid_dep_launch_dependents();
  const Batch& B = p.b;
  find_range<ROWS_THREADS, BY_HEAD>(B, p.c, &sm.range, sm.scratch);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gq = lane >> 2, jq = lane & 3;
  const int key0 = gq & 1 ? 7 - (gq >> 1) : gq >> 1;  // this lane's key of K, the other is 8 behind
  const int key1 = jq, key2 = 7 - jq;                 // its keys of V, two more are 8 behind
  Stage4<D>* const ring = sm.ring[warp];
  // 16-byte piece `c` of key j lies at c ^ turn(j) in its row of 64 bytes (32 bytes: where it is)
  auto turn = [](int j) { return D == 128 ? j & 2 : 0; };
  // What a lane copies: of one of the warp's two runs of 16 keys a piece of every STEP-th key, and maybe 16
  // bytes of scales (which lie side by side).
  constexpr int PIECES = D / GROUP4, STEP = 16 / PIECES;
  const int run = lane >> 4, piece = lane & (PIECES - 1), first_key = (lane & 15) / PIECES;
  const uint32_t slot_bytes = static_cast<uint32_t>(B.slot_stride >> 1), page_bytes = static_cast<uint32_t>(B.page_stride >> 1);
  const uint32_t page_scales = B.kv_heads * B.page_size * PIECES;
  const bool has_scales = (lane & 15) < 2 * PIECES, of_v = (lane & 15) >= PIECES;
  WalkOf<BY_HEAD> walk(p.c, sm.range);
  Seg g;
  while (walk.next(B, p.c, g)) {
    const int first = g.item * p.c.per_item;  // the item's first token
    const int tokens = min(p.c.per_item, g.s.n - first), rows = tokens * B.group;
    const int* table = p.c.flat ? p.pages : B.table + static_cast<long long>(g.b) * B.table_cols;
    const int base = g.s.m - g.s.n + first;  // position of its first token
    const int mine = warp * 16 + run * 64;   // this lane's run of a tile
    const int skip = (g.lo >> ROWS4_SHIFT) - g.sinks;  // tiles between the sinks' and the window's
    auto tile_at = [&](int k) { return (k < g.sinks ? k : k + skip) << ROWS4_SHIFT; };  // Seg::key0
    // the page of this lane's run of tile k, -1 if none of its keys is seen
    auto table_of = [&](int k) {
      const int j = tile_at(k) + mine;
      if (k >= g.k1 || j >= g.hi || (j + 16 <= g.lo && j >= p.c.sinks)) return -1;
      const int page = __ldg(table + (j >> B.page_shift));
      return page < 0 ? INT_MAX : page;
    };
    auto checked = [&](int page) {
      if (page < B.num_pages) return page;
      record(B.ctrl, ERR_INVALID, WHAT_PAGE, p.c.flat ? 0xFFFFFFFFu : static_cast<uint32_t>(g.b));
      return -1;
    };
    // this lane's part of the codes of K, and V's offset from it; of the scales, K's or V's
    const uint8_t* const codes = static_cast<const uint8_t*>(p.k_raw) + (g.kvh * B.head_stride >> 1) + first_key * slot_bytes + piece * 16;
    const long long to_v = static_cast<const uint8_t*>(p.v_raw) - static_cast<const uint8_t*>(p.k_raw);
    const uint8_t* const scales = (of_v ? p.v_scales : p.k_scales) + g.kvh * (B.page_size * PIECES) + piece * 16;
    auto load = [&](int k, int page, Stage4<D>& to) {
      if (k < g.k1) {
        const bool read = page >= 0;
        const uint32_t from = read ? page : 0, slot = (tile_at(k) + mine) & (B.page_size - 1);
        const uint8_t* at = codes + static_cast<uint64_t>(from) * page_bytes + slot * slot_bytes;
        uint8_t* into = &to.codes[0][run * 16 + first_key][(piece ^ turn(first_key)) * 16];
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {  // (STEP is a multiple of 4, so the piece is turned alike)
          copy16(into + i * STEP * (D / 2), at, read);
          copy16(into + i * STEP * (D / 2) + sizeof(to.codes[0]), at + to_v, read);
          at += STEP * slot_bytes;
        }
        if (has_scales)
          copy16(&to.scales[of_v][run * 16][0] + piece * 16,
                 scales + static_cast<uint64_t>(from) * page_scales + slot * PIECES, read);
      }
      copies_commit();
    };
    int ahead[ST];
#pragma unroll
    for (int i = 0; i < ST; ++i) ahead[i] = table_of(g.k0 + i);
    __syncthreads();  // shared memory of the segment before is read
#pragma unroll
    for (int i = 0; i < ST - 1; ++i) load(g.k0 + i, checked(ahead[i]), ring[i]);
    int next = ahead[ST - 1];
    // the queries, in the order of a key's words, in f16: rows of bf16 times a power of two that puts their largest
    // value to 2^14 .. 2^15 (what is lost below 2^-25 is 2^-39 of it); `unit` undoes both operands' factors
    uint32_t q[NT][KW][4];
    float unit[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int r = 8 * n + gq, t = r / B.group;
      const uint4* from = reinterpret_cast<const uint4*>(static_cast<const T*>(p.q_raw) + (g.s.t0 + first + t) * p.q_stride +
                                                         (g.kvh * B.group + r - t * B.group) * D) + jq * KW;
#pragma unroll
      for (int w = 0; w < KW; ++w) *reinterpret_cast<uint4*>(q[n][w]) = r < rows ? from[w] : make_uint4(0, 0, 0, 0);
      float f = 1.0f;
      if constexpr (!std::is_same<T, __half>::value) {
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 4 * KW; ++i) {
          const uint32_t lo = q[n][i / 4][i % 4] << 16 & 0x7F800000u, hi = q[n][i / 4][i % 4] & 0x7F800000u;  // exponents
          top = max(top, max(lo == 0x7F800000u ? 0u : lo, hi == 0x7F800000u ? 0u : hi));
        }
        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
        const int shift = min(max(14 - (static_cast<int>(top >> 23) - 127), -112), 126);
        const float by = __uint_as_float(static_cast<uint32_t>(127 + shift) << 23);
        f = __uint_as_float(static_cast<uint32_t>(127 - shift) << 23);
#pragma unroll
        for (int i = 0; i < 4 * KW; ++i) {
          const float2 v = Pair<T>::get(q[n][i / 4][i % 4]);
          q[n][i / 4][i % 4] = Pair<__half>::put(v.x * by, v.y * by);
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e)
        // (neither infinite nor, for a row of zeros and a small scale, 0: hidden scores are -infinity before it)
        unit[n][e] = fmaxf(fminf(__shfl_sync(0xFFFFFFFFu, f, 4 * (2 * jq + e)) / FOUR_UNIT * p.scale_log2, FLT_MAX), FLT_MIN);
    }
    // keys below all_end and from all_lo on are seen by every row
    const int all_end = p.c.flat ? g.s.m : base + 1, all_lo = p.c.window > 0 ? max(0, base + tokens - p.c.window) : 0;
    // is key j seen by row 8 n + 2 jq + e?  (Rows behind the last see none.)
    auto seen_by = [&](int n, int e, int j) {
      const int r = 8 * n + 2 * jq + e, pos = base + r / B.group;
      const int end = r >= rows ? 0 : p.c.flat ? g.s.m : pos + 1;
      return j < end && (p.c.window <= 0 || j > pos - p.c.window || j < p.c.sinks);
    };
    float o[NT][4 * VW][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4 * VW; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[n][i][c] = 0.0f;
    float m_ref[NT][2], l[NT][2];  // of a row: the reference (of scores times unit) and the sum
    using Values = OperandsOf<T>;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) m_ref[n][e] = -INFINITY, l[n][e] = 0.0f;
    int at = 0;  // the stage of tile k
#pragma unroll 1
    for (int k = g.k0; k < g.k1; ++k) {
      copies_wait<ST - 2>();
      __syncwarp();  // every lane's copies are there, and the stage before is read
      load(k + ST - 1, checked(next), ring[at == 0 ? ST - 1 : at - 1]);
      next = table_of(k + ST);
      const Stage4<D>& st = ring[at];
      at = at == ST - 1 ? 0 : at + 1;
      const int tile0 = tile_at(k) + warp * 16;
      // some key is hidden from some row
      const bool mask = !(tile0 + 80 <= all_end && (tile0 >= all_lo || tile0 + 80 <= p.c.sinks));
#pragma unroll 1
      for (int x0 = 0; x0 < 2; x0 += XS) {
        // the scales of this lane's keys, two of K and two pairs of V, and whether one of the warp's is big
        uint32_t sk[XS], sv[XS][2], most = 0;
#pragma unroll
        for (int x = 0; x < XS; ++x) {
          const uint8_t* of_k = st.scales[0][(x0 + x) * 16 + key0] + (D == 128 ? jq : jq >> 1);
          const uint32_t k0 = of_k[0], k1 = of_k[8 * PIECES];
          uint32_t v[4];
#pragma unroll
          for (int y = 0; y < 4; ++y)
            v[y] = st.scales[1][(x0 + x) * 16 + (y & 1 ? key2 : key1) + 8 * (y >> 1)][D == 128 ? gq >> 1 : gq >> 2];
          if (__builtin_expect(mask, 0)) {  // a scale of a key that no row sees may be anything
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const int key = tile0 + (x0 + x) * 64 + (y & 1 ? key2 : key1) + 8 * (y >> 1);
              if (!(key < g.hi && (key >= g.lo || key < p.c.sinks))) v[y] = 0;
            }
          }
          const uint32_t v01 = v[1] * 0x10000u + v[0], v23 = v[3] * 0x10000u + v[2];
          sk[x] = k1 * 0x10000u + k0;
          sv[x][0] = v01 * 0x80u;
          sv[x][1] = v23 * 0x80u;
          most = __vmaxu2(most, sk[x]);
          if (Values::HAS_BIG) most = __vmaxu2(most, __vmaxu2(v01, v23));
        }
        const bool big = (most + (0x100u - FourScaled::BIG_BYTE) * 0x10001u & 0x01000100u) != 0;
        auto keys = [&](auto is_big) {
          constexpr bool BIG = decltype(is_big)::value;
          float s[XS][NT][4] = {};
#pragma unroll
          for (int x = 0; x < XS; ++x) {
            uint32_t ka[KW], kb[KW];
            const int j = (x0 + x) * 16 + key0;
            const uint8_t* row = st.codes[0][j] + (D == 128 ? (jq ^ turn(key0)) * 16 : jq * 8);
            if constexpr (D == 128) {
              *reinterpret_cast<uint4*>(ka) = *reinterpret_cast<const uint4*>(row);
              *reinterpret_cast<uint4*>(kb) = *reinterpret_cast<const uint4*>(row + 8 * (D / 2));
            } else {
              *reinterpret_cast<uint2*>(ka) = *reinterpret_cast<const uint2*>(row);
              *reinterpret_cast<uint2*>(kb) = *reinterpret_cast<const uint2*>(row + 8 * (D / 2));
            }
            const FourScaled fa(scale_pair(sk[x] & 0xFFu)), fb(scale_pair(sk[x] >> 16));
#pragma unroll
            for (int w = 0; w < KW; ++w) {
              uint32_t a[4], b[4];
              fa.pairs<BIG>(ka[w], a);
              fb.pairs<BIG>(kb[w], b);
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                mma16816<__half>(s[x][n], a[0], b[0], a[1], b[1], q[n][w][0], q[n][w][1]);
                mma16816<__half>(s[x][n], a[2], b[2], a[3], b[3], q[n][w][2], q[n][w][3]);
              }
            }
          }
          if (__builtin_expect(mask, 0)) {
#pragma unroll
            for (int x = 0; x < XS; ++x)
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int c = 0; c < 4; ++c)
                  if (!seen_by(n, c & 1, tile0 + (x0 + x) * 64 + key0 + 8 * (c >> 1))) s[x][n][c] = -INFINITY;
          }
          bool raise = false;
          float top[NT][2];
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              top[n][e] = fmaxf(s[0][n][e], s[0][n][2 + e]);
              if (XS == 2) top[n][e] = max3(top[n][e], s[XS - 1][n][e], s[XS - 1][n][2 + e]);
              // raised only when it is exceeded by more than 2^8 (from -infinity by anything but that)
              raise |= fmaf(top[n][e], unit[n][e], -m_ref[n][e]) > RAISE_LOG2 + WEIGHT_LOG2 || fabsf(m_ref[n][e]) > FAR_LOG2;
            }
          float sub[NT][2];
          if (__any_sync(0xFFFFFFFFu, raise)) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float t = top[n][e];
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) t = fmaxf(t, __shfl_xor_sync(0xFFFFFFFFu, t, d));
                const float m = fmaf(t, unit[n][e], -WEIGHT_LOG2);
                // (scores that overflow: -infinity raises nothing, as a hidden key; a reference of infinity makes the row NaN
                // when the warps' states are joined)
                if (m - m_ref[n][e] > RAISE_LOG2) {
                  const float f = cs::ex2_approx(m_ref[n][e] - m);
                  m_ref[n][e] = m;
                  l[n][e] *= f;
#pragma unroll
                  for (int i = 0; i < 4 * VW; ++i) o[n][i][e] *= f, o[n][i][2 + e] *= f;
                }
                sub[n][e] = m_ref[n][e] == -INFINITY ? 0.0f : -m_ref[n][e];
                if (fabsf(m) > FAR_LOG2 && fabsf(m) < INFINITY) {  // differences before the factor
                  sub[n][e] = m - m_ref[n][e] + WEIGHT_LOG2;
#pragma unroll
                  for (int x = 0; x < XS; ++x) s[x][n][e] -= t, s[x][n][2 + e] -= t;
                }
              }
          } else {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int e = 0; e < 2; ++e) sub[n][e] = -m_ref[n][e];
          }
          uint32_t pt[XS][NT][2];
#pragma unroll
          for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
              for (int x = 0; x < XS; ++x) {
                s[x][n][e] = cs::ex2_approx(fmaf(s[x][n][e], unit[n][e], sub[n][e]));
                s[x][n][2 + e] = cs::ex2_approx(fmaf(s[x][n][2 + e], unit[n][e], sub[n][e]));
                l[n][e] += s[x][n][e] + s[x][n][2 + e];
              }
            }
#pragma unroll
            for (int x = 0; x < XS; ++x) {
              pt[x][n][0] = transposed(Pair<T>::put(s[x][n][0], s[x][n][1]));
              pt[x][n][1] = transposed(Pair<T>::put(s[x][n][2], s[x][n][3]));
            }
          }
#pragma unroll
          for (int x = 0; x < XS; ++x) {
            // V: words of keys key1, key2, key1 + 8 and key2 + 8 of the run
            uint32_t v[4][VW];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const int of = y & 1 ? key2 : key1, j = (x0 + x) * 16 + of + 8 * (y >> 1);
              const uint8_t* row = st.codes[1][j] + (D == 128 ? (((gq >> 1) ^ turn(of)) * 16 + (gq & 1) * 8) : gq * 4);
              if constexpr (D == 128)
                *reinterpret_cast<uint2*>(v[y]) = *reinterpret_cast<const uint2*>(row);
              else
                v[y][0] = *reinterpret_cast<const uint32_t*>(row);
            }
            const Values fa(sv[x][0]), fb(sv[x][1]);
#pragma unroll
            for (int w = 0; w < VW; ++w) {
              uint32_t a0[4], a1[4], a2[4], a3[4];  // even and odd dimensions of keys key1, key2; of those 8 behind
              fa.template pairs<BIG>(__byte_perm(v[0][w], v[1][w], 0x5410), a0);
              fa.template pairs<BIG>(__byte_perm(v[0][w], v[1][w], 0x7632), a1);
              fb.template pairs<BIG>(__byte_perm(v[2][w], v[3][w], 0x5410), a2);
              fb.template pairs<BIG>(__byte_perm(v[2][w], v[3][w], 0x7632), a3);
#pragma unroll
              for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int n = 0; n < NT; ++n) mma16816<T>(o[n][4 * w + i], a0[i], a1[i], a2[i], a3[i], pt[x][n][0], pt[x][n][1]);
            }
          }
        };
        if (__builtin_expect(__any_sync(0xFFFFFFFFu, big), 0))
          keys(std::true_type());
        else
          keys(std::false_type());
      }
    }
    copies_wait<0>();
    __syncthreads();  // every warp is done with the ring's memory
    // the warps' states to shared memory: this lane has 8 VW dimensions of rows 8 n + 2 jq and 8 n + 2 jq + 1
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 8 * n + 2 * jq + e;
        float sum = l[n][e];
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
        if (r < rows) {
          if (gq == 0) sm.ml[warp][r] = make_float2(m_ref[n][e], sum);
          float4* to = reinterpret_cast<float4*>(&sm.o[warp][r][8 * VW * gq]);
#pragma unroll
          for (int i = 0; i < 4 * VW; i += 2)
            to[i / 2] = make_float4(o[n][i][e] / FOUR_UNIT, o[n][i][2 + e] / FOUR_UNIT, o[n][i + 1][e] / FOUR_UNIT,
                                    o[n][i + 1][2 + e] / FOUR_UNIT);
        }
      }
    __syncthreads();
    const Pieces of = rows_store<T, D>(p, g, first, rows, late, sm.o, sm.ml, sm.range, sm.last);
    if (of.count > 0) join4<T, D, NT>(p, g, first, rows, of, sm);
  }
  if (late) cs::grid_dep_wait();
}

}  // namespace cskv
