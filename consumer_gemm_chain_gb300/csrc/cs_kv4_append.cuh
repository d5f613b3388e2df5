// Writing new tokens' keys and values to a paged cache in 4 bits, and reading them back
// (include/cs_kv4.h).
#pragma once
#include "cs_kv4_codes.cuh"

namespace cskv {

struct Four4P {
  Batch b;
  const uint4* qkv;
  uint4* q_out;
  uint8_t *k_codes, *v_codes, *k_scales, *v_scales;
  uint4 *k_out, *v_out;  // of the reading
  const float4* rope;
  const int* positions;
  long long qkv_stride, q_stride, k_stride, v_stride;  // in 16-byte chunks
  int rope_rows, rotary_dim, half, head_chunks;        // half: HALF pairing; head_chunks = head_dim / 8
  int warps_shift;                                     // 1 << warps_shift warps have a token
  int units, q_units;                                  // of a token (an append's units are its keys' and values')
  int head_shift;                                      // head_chunks = 1 << head_shift
  int wide;                                            // outputs' rows start on 32-byte boundaries
};

constexpr int FOUR_THREADS = 256;

// Where a token's slot lies: its element offset in the codes (-1: the token is left out), its row of scales of head 0,
// and its row of the rotation table.
struct Place {
  long long codes, scales;
  int angle;
};

// One warp, all lanes.
template <bool ROTATE>
__device__ __forceinline__ Place find_place(const Four4P& p, int t) {
  const Batch& B = p.b;
  const int b = sequence_of(B, t);
  int t0, n, m;
  Place out{-1, 0, 0};
  const bool fits = sequence(B, b, t0, n, m);  // (every lane the same loads)
  const int pos = m - n + t - t0;
  if (!fits || t < t0 || t >= t0 + n || pos < 0) return out;
  if (ROTATE) out.angle = p.positions ? __ldg(p.positions + t) : pos;
  const int page = __ldg(B.table + static_cast<long long>(b) * B.table_cols + (pos >> B.page_shift)), slot = pos & (B.page_size - 1);
  if (page < 0 || page >= B.num_pages) {
    if ((threadIdx.x & 31) == 0) record(B.ctrl, ERR_INVALID, WHAT_PAGE, static_cast<uint32_t>(b));
  } else if (ROTATE && p.rotary_dim > 0 && (out.angle < 0 || out.angle >= p.rope_rows)) {
    if ((threadIdx.x & 31) == 0) record(B.ctrl, ERR_INVALID, WHAT_POSITION, static_cast<uint32_t>(t));
  } else {
    out.codes = page * B.page_stride + slot * B.slot_stride;
    out.scales = scale_row(B, page, slot, 0);
  }
  return out;
}

// The rotation: (a, b) -> (a cos - b sin, b cos + a sin), each product and each sum rounded to 32 bits (no
// multiply-add: what is kept does not depend on how it is compiled), the result to the dtype.
template <typename T>
struct Turn {
  static __device__ __forceinline__ float minus(float a, float c, float b, float s) {  // a c - b s
    return __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  }
  static __device__ __forceinline__ float plus(float a, float c, float b, float s) {  // a c + b s
    return __fadd_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  }
  // Pairs of neighbouring values: one chunk by four angles.
  static __device__ __forceinline__ void adjacent(uint32_t* x, const float4& c, const float4& s) {
    const float co[4] = {c.x, c.y, c.z, c.w}, si[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 a = Pair<T>::get(x[e]);
      x[e] = Pair<T>::put(minus(a.x, co[e], a.y, si[e]), plus(a.y, co[e], a.x, si[e]));
    }
  }
};

// c = x / s rounded to the nearest, ties to even, as the float 1.5 2^23 + 8 + c.  inv is 1 / s rounded, so x inv may
// miss a tie by a part in 2^23; a quotient that is no tie is at least 2^-13 away from one (x has at most 11
// significant bits, s has 4), so rounding to steps of 2^-16 first puts it right: a sum of 192 does.
__device__ __forceinline__ float rounded(float x, float inv) { return __fadd_rn(__fmaf_rn(x, inv, 192.0f), 12582728.0f); }
constexpr uint32_t ROUNDED_ZERO = 0x4B400000;  // 1.5 2^23

// The word of 8 values under one scale; `clamp`: quotients may be beyond +-7.5.
__device__ __forceinline__ uint32_t code_word(const float (&y)[8], float inv, bool clamp) {
  uint32_t word = 0, rest = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    float r = rounded(y[e], inv);
    if (clamp) r = fminf(fmaxf(r, 12582920.0f - 7.0f), 12582920.0f + 7.0f);
    const uint32_t at = 1u << (4 * (e >> 1) + 16 * (e & 1));
    word += __float_as_uint(r) * at;  // the exponents' bits are taken off together
    rest += ROUNDED_ZERO * at;
  }
  return word - rest;
}

// Appends: the rotated Q to its rows, the 4-bit form of the rotated K and of V to the cache.  Queries go 16 values a thread,
// both halves of a pair (so that they can be rotated in place); keys and values 8 a lane, with the other half of a pair from
// the lane that holds it and a group's maximum from its four lanes.  A warp has a token (or part of one) and looks its
// place up for itself: lookups by some warps of a block for all its tokens, behind a barrier, were slower (82.8 and 77.6 us).
// Bound by instructions and DRAM alike: 19743 tokens of 32 + 2 x 8 heads of 128 (435 MB): 77.6 us, 5.6 TB/s, 0.83 of a
// plain copy's measured 6.8.  (16000 of them, 66 us: 2.8 of 4 instructions a cycle, the busiest pipe 48 %, DRAM 60 %; warps
// wait for loads most.  A sixth block an SM makes it 12 bytes of spills a thread.)  (The 16-bit cache's append, which moves 495 MB and
// makes nothing of them, takes 74.)  247 single tokens of 40 + 2 x 8 heads of 64: 3.2 us, one token alone 3.1, launch and lookups.
template <typename T>
__global__ void __launch_bounds__(FOUR_THREADS, 6) cs_kv4_append_kernel(const __grid_constant__ Four4P p) {
  cs::grid_dep_wait();
  cs::grid_dep_launch_dependents();
  const Batch& B = p.b;
  const int turned = p.rotary_dim >> 4;    // chunks that hold one half of the pairs
  const int lane = threadIdx.x & 31, warp = blockIdx.x * (FOUR_THREADS / 32) + (threadIdx.x >> 5);
  const int t = warp >> p.warps_shift, part = warp & ((1 << p.warps_shift) - 1), step = 32 << p.warps_shift;
  if (t >= B.tokens) return;
  const uint4* const row = p.qkv + t * p.qkv_stride;
  // keys and values: chunk c of head h (V's behind K's), this lane's of the warp's 32 from i0 on
  int h, c;
  uint4 x4;
  auto fetch = [&](int i0) {
    if (i0 >= p.units) return;
    const int i = min(i0 + lane, p.units - 1);  // (lanes behind the end go along)
    h = i >> p.head_shift;
    c = i & (p.head_chunks - 1);
    x4 = row[B.heads * p.head_chunks + i];
  };
  fetch(part * 32);
  const Place place = find_place<true>(p, t);
  if (place.codes < 0) return;
  const float4* const angles = p.rope + static_cast<long long>(place.angle) * (p.rotary_dim >> 2);
  for (int i0 = part * 32; i0 < p.units;) {
    uint32_t* x = reinterpret_cast<uint32_t*>(&x4);
    const bool live = i0 + lane < p.units;
    const bool key = h < B.kv_heads, rotate = key && c < 2 * turned;
    if (p.half && turned > 0) {
      const bool upper = c >= turned;
      const int j = upper ? c - turned : c, from = rotate ? lane - c + (upper ? j : c + turned) : lane;
      uint32_t y[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = __shfl_sync(0xFFFFFFFFu, x[e], from);
      if (rotate) {
        const float4 ca = __ldg(angles + 2 * j), cb = __ldg(angles + 2 * j + 1);
        const float4 sa = __ldg(angles + 2 * turned + 2 * j), sb = __ldg(angles + 2 * turned + 2 * j + 1);
        const float co[8] = {ca.x, ca.y, ca.z, ca.w, cb.x, cb.y, cb.z, cb.w};
        const float si[8] = {sa.x, sa.y, sa.z, sa.w, sb.x, sb.y, sb.z, sb.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 a = Pair<T>::get(x[e]), b = Pair<T>::get(y[e]);
          const float u = upper ? b.x : -b.x, w = upper ? b.y : -b.y;  // (a sign changes no rounding)
          x[e] = Pair<T>::put(Turn<T>::plus(a.x, co[2 * e], u, si[2 * e]), Turn<T>::plus(a.y, co[2 * e + 1], w, si[2 * e + 1]));
        }
      }
    } else if (rotate) {
      Turn<T>::adjacent(x, __ldg(angles + c), __ldg(angles + 2 * turned + c));
    }
    // the greatest magnitude of the group, as bits: what is not finite is greater than what is
    uint32_t top = __vmaxu2(__vmaxu2(x[0] & 0x7FFF7FFFu, x[1] & 0x7FFF7FFFu), __vmaxu2(x[2] & 0x7FFF7FFFu, x[3] & 0x7FFF7FFFu));
    top = __vmaxu2(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
    top = __vmaxu2(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
    if (live) {
      const int kh = key ? h : h - B.kv_heads;
      const float amax = Pair<T>::get(max(top & 0xFFFFu, top >> 16)).x;
      const bool finite = isfinite(amax);
      const uint32_t byte = finite ? scale_byte(__fdiv_rn(amax, 7.0f)) : SCALE_NAN;
      uint32_t word = 0x88888888u;  // zeros
      if (finite && byte != 0) {
        float y[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 v = Pair<T>::get(x[e]);
          y[2 * e] = v.x, y[2 * e + 1] = v.y;
        }
        const float inv = __frcp_rn(scale_value(byte));
        // (a scale of 4 significant bits is off by a sixteenth at most, and amax / s below 7.5)
        word = byte < 8 || byte == SCALE_MOST ? code_word(y, inv, true) : code_word(y, inv, false);
      }
      *reinterpret_cast<uint32_t*>((key ? p.k_codes : p.v_codes) + (place.codes + kh * B.head_stride) / 2 + 4 * c) = word;
      if ((c & 3) == 0) {
        const long long at = place.scales + static_cast<long long>(kh) * B.page_size;
        (key ? p.k_scales : p.v_scales)[at * (p.head_chunks >> 2) + (c >> 2)] = static_cast<uint8_t>(byte);
      }
    }
    i0 += step;
    fetch(i0);
  }
  // queries: two chunks of a head, those that are rotated together, or neighbours
  uint4* const q_row = p.q_out + t * p.q_stride;
  uint4 a4, b4;
  int c0, c1;
  auto fetch_q = [&](int i) {
    if (i >= p.q_units) return;
    h = i >> (p.head_shift - 1);
    c = i & ((p.head_chunks >> 1) - 1);
    const bool apart = p.half && c < turned;
    c0 = h * p.head_chunks + (apart ? c : 2 * c), c1 = c0 + (apart ? turned : 1);
    a4 = row[c0], b4 = row[c1];
  };
  fetch_q(part * 32 + lane);
  for (int i = part * 32 + lane; i < p.q_units;) {
    uint32_t *x = reinterpret_cast<uint32_t*>(&a4), *y = reinterpret_cast<uint32_t*>(&b4);
    if (c < turned) {
      // 8 cosines, 8 sines: HALF rotates (x[e], y[e]), ADJACENT neighbouring values
      const float4 ca = __ldg(angles + 2 * c), cb = __ldg(angles + 2 * c + 1);
      const float4 sa = __ldg(angles + 2 * turned + 2 * c), sb = __ldg(angles + 2 * turned + 2 * c + 1);
      if (p.half) {
        const float co[8] = {ca.x, ca.y, ca.z, ca.w, cb.x, cb.y, cb.z, cb.w};
        const float si[8] = {sa.x, sa.y, sa.z, sa.w, sb.x, sb.y, sb.z, sb.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 a = Pair<T>::get(x[e]), b = Pair<T>::get(y[e]);
          const int u = 2 * e, w = 2 * e + 1;
          x[e] = Pair<T>::put(Turn<T>::minus(a.x, co[u], b.x, si[u]), Turn<T>::minus(a.y, co[w], b.y, si[w]));
          y[e] = Pair<T>::put(Turn<T>::plus(b.x, co[u], a.x, si[u]), Turn<T>::plus(b.y, co[w], a.y, si[w]));
        }
      } else {
        Turn<T>::adjacent(x, ca, sa);
        Turn<T>::adjacent(y, cb, sb);
      }
    }
    q_row[c0] = a4;
    q_row[c1] = b4;
    i += step;
    fetch_q(i);
  }
}

// Reads back the keys and values of the batch's new tokens.  A unit is 16 values: 8 bytes of codes and a scale;
// a thread has two of them on their way at a time.  Bound by DRAM, which takes the values: 69710 tokens of 8 heads of 128
// (361 MB): 56.2 us, 6.4 TB/s, 0.95 of a plain copy.  One, two and four units at a time: 57.4, 56.2 and 58.2 us; 977 tokens
// of 12 heads 3.1, 3.3 and 3.5.
template <typename T>
__global__ void __launch_bounds__(FOUR_THREADS, 6) cs_kv4_read_kernel(const __grid_constant__ Four4P p) {
  constexpr int AHEAD = 2;
  cs::grid_dep_wait();
  cs::grid_dep_launch_dependents();
  const Batch& B = p.b;
  const int lane = threadIdx.x & 31, warp = blockIdx.x * (FOUR_THREADS / 32) + (threadIdx.x >> 5);
  const int t = warp >> p.warps_shift, part = warp & ((1 << p.warps_shift) - 1), step = 32 << p.warps_shift;
  if (t >= B.tokens) return;
  const Place place = find_place<false>(p, t);
  if (place.codes < 0) return;
  const int total = p.units, per_head = p.head_chunks >> 1;  // units of a head
  for (int i0 = part * 32 + lane; i0 < total; i0 += AHEAD * step) {
    uint2 w[AHEAD];
    uint32_t byte[AHEAD];
    uint4* to[AHEAD];
#pragma unroll
    for (int n = 0; n < AHEAD; ++n) {
      const int i = i0 + n * step;
      if (i >= total) break;
      const int h = i >> (p.head_shift - 1), j = i & (per_head - 1);
      const bool key = p.k_out && h < B.kv_heads;  // without k_out all units are V's
      const int kh = p.k_out && !key ? h - B.kv_heads : h;
      w[n] = __ldg(reinterpret_cast<const uint2*>((key ? p.k_codes : p.v_codes) + (place.codes + kh * B.head_stride) / 2 + 8 * j));
      const long long at = place.scales + static_cast<long long>(kh) * B.page_size;
      byte[n] = __ldg((key ? p.k_scales : p.v_scales) + at * (p.head_chunks >> 2) + (j >> 1));
      to[n] = (key ? p.k_out + t * p.k_stride : p.v_out + t * p.v_stride) + kh * p.head_chunks + 2 * j;
    }
#pragma unroll
    for (int n = 0; n < AHEAD; ++n) {
      if (i0 + n * step >= total) break;
      const Four<T> four(scale_pair(byte[n]));
      uint32_t x[8];
      four.pairs(w[n].x, x[0], x[1], x[2], x[3]);
      four.pairs(w[n].y, x[4], x[5], x[6], x[7]);
      if (p.wide) {
        st32(to[n], x);
      } else {
        to[n][0] = make_uint4(x[0], x[1], x[2], x[3]);
        to[n][1] = make_uint4(x[4], x[5], x[6], x[7]);
      }
    }
  }
}

}  // namespace cskv
