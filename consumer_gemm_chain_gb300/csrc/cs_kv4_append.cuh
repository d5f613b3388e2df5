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
  int tokens_per_block;
  // units per token, and ceil(2^32 / units): i / units is the upper half of the product while i units < 2^32
  uint32_t units, per_unit, q_units, per_q_unit;  // (an append's units are its keys' and values')
  int head_shift;                                      // head_chunks = 1 << head_shift
  int wide;                                            // outputs' rows start on 32-byte boundaries
};

constexpr int FOUR_THREADS = 256;
constexpr int FOUR_MAX_TOKENS = 32;  // per block

// Where the tokens of a block lie: the element offset of a token's slot in the codes (-1: left out), and its
// row of scales of head 0.
struct Places {
  long long codes[FOUR_MAX_TOKENS], scales[FOUR_MAX_TOKENS];
  int angle[FOUR_MAX_TOKENS];  // its row of the rotation table
};

// Looked up by a warp each; then a barrier.
template <bool ROTATE>
__device__ __forceinline__ void find_places(const Four4P& p, int first, int count, Places& out) {
  const Batch& B = p.b;
  for (int w = threadIdx.x >> 5; w < count; w += FOUR_THREADS / 32) {
    const int t = first + w, b = sequence_of(B, t);
    if ((threadIdx.x & 31) != 0) continue;
    int t0, n, m, row = 0;
    long long at = -1, scales = 0;
    if (sequence(B, b, t0, n, m) && t >= t0 && t < t0 + n && m - n + t - t0 >= 0) {
      const int pos = m - n + t - t0, slot = pos & (B.page_size - 1);
      if (ROTATE) row = p.positions ? __ldg(p.positions + t) : pos;
      const int page = __ldg(B.table + static_cast<long long>(b) * B.table_cols + (pos >> B.page_shift));
      if (page < 0 || page >= B.num_pages) {
        record(B.ctrl, ERR_INVALID, WHAT_PAGE, static_cast<uint32_t>(b));
      } else if (ROTATE && p.rotary_dim > 0 && (row < 0 || row >= p.rope_rows)) {
        record(B.ctrl, ERR_INVALID, WHAT_POSITION, static_cast<uint32_t>(t));
      } else {
        at = page * B.page_stride + slot * B.slot_stride;
        scales = scale_row(B, page, slot, 0);
      }
    }
    out.codes[w] = at;
    out.scales[w] = scales;
    if (ROTATE) out.angle[w] = row;
  }
}

// Appends: (a, b) -> (a cos - b sin, b cos + a sin) for every rotated pair of Q and K, each product and each sum
// rounded to 32 bits (no multiply-add: what is kept does not depend on how it is compiled) and the result to the dtype;
// then the 4-bit form of K and V.  Queries go 16 values a thread, both halves of a pair (so that they can be
// rotated in place); keys and values 8 a lane, with the other half of a pair from the lane
// that holds it and a group's maximum from its four lanes.
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

template <typename T>
__global__ void __launch_bounds__(FOUR_THREADS, 6) cs_kv4_append_kernel(const __grid_constant__ Four4P p) {
  __shared__ Places places;
  cs::grid_dep_wait();
  cs::grid_dep_launch_dependents();
  const Batch& B = p.b;
  const int first = blockIdx.x * p.tokens_per_block;
  const int count = min(p.tokens_per_block, B.tokens - first);
  const int turned = p.rotary_dim >> 4;    // chunks that hold one half of the pairs
  const int lane = threadIdx.x & 31;
  // keys and values: chunk c of head h (V's behind K's), this lane's of the warp's 32 from i0 on
  const int kv_total = count * p.units;
  int k, h, c;
  uint4 x4;
  auto fetch = [&](int i0) {
    if (i0 >= kv_total) return;
    const int i = min(i0 + lane, kv_total - 1);  // (lanes behind the end go along)
    k = __umulhi(i, p.per_unit);
    const int in = i - k * p.units;
    h = in >> p.head_shift;
    c = in & (p.head_chunks - 1);
    x4 = p.qkv[(first + k) * p.qkv_stride + (B.heads + h) * p.head_chunks + c];
  };
  fetch(threadIdx.x - lane);
  find_places<true>(p, first, count, places);
  __syncthreads();
  for (int i0 = threadIdx.x - lane; i0 < kv_total;) {
    uint32_t* x = reinterpret_cast<uint32_t*>(&x4);
    const long long at = i0 + lane < kv_total ? places.codes[k] : -1;
    const bool key = h < B.kv_heads, rotate = key && c < 2 * turned;
    const float4* angles = p.rope + static_cast<long long>(places.angle[k]) * (p.rotary_dim >> 2);
    if (p.half && turned > 0) {
      const bool upper = c >= turned;
      const int j = upper ? c - turned : c, from = rotate ? lane - c + (upper ? j : c + turned) : lane;
      uint32_t y[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = __shfl_sync(0xFFFFFFFFu, x[e], from);
      if (rotate && at >= 0) {
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
    } else if (rotate && at >= 0) {
      Turn<T>::adjacent(x, __ldg(angles + c), __ldg(angles + 2 * turned + c));
    }
    // the greatest magnitude of the group, as bits: what is not finite is greater than what is
    uint32_t top = __vmaxu2(__vmaxu2(x[0] & 0x7FFF7FFFu, x[1] & 0x7FFF7FFFu), __vmaxu2(x[2] & 0x7FFF7FFFu, x[3] & 0x7FFF7FFFu));
    top = __vmaxu2(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
    top = __vmaxu2(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
    if (at >= 0) {
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
      *reinterpret_cast<uint32_t*>((key ? p.k_codes : p.v_codes) + (at + kh * B.head_stride) / 2 + 4 * c) = word;
      if ((c & 3) == 0) {
        const long long row = places.scales[k] + static_cast<long long>(kh) * B.page_size;
        (key ? p.k_scales : p.v_scales)[row * (p.head_chunks >> 2) + (c >> 2)] = static_cast<uint8_t>(byte);
      }
    }
    i0 += FOUR_THREADS;
    fetch(i0);
  }
  // queries: two chunks of a head, those that are rotated together, or neighbours
  const int q_total = count * p.q_units;
  uint4 a4, b4;
  int c0, c1;
  auto fetch_q = [&](int i) {
    if (i >= q_total) return;
    k = __umulhi(i, p.per_q_unit);
    const int in = i - k * p.q_units;
    h = in >> (p.head_shift - 1);
    c = in & ((p.head_chunks >> 1) - 1);
    const bool apart = p.half && c < turned;
    c0 = apart ? c : 2 * c, c1 = apart ? c + turned : 2 * c + 1;
    const uint4* src = p.qkv + (first + k) * p.qkv_stride + h * p.head_chunks;
    a4 = src[c0], b4 = src[c1];
  };
  fetch_q(threadIdx.x);
  for (int i = threadIdx.x; i < q_total;) {
    if (places.codes[k] >= 0) {
      uint32_t *x = reinterpret_cast<uint32_t*>(&a4), *y = reinterpret_cast<uint32_t*>(&b4);
      if (c < turned) {
        // 8 cosines, 8 sines: HALF rotates (x[e], y[e]), ADJACENT neighbouring values
        const float4* angles = p.rope + static_cast<long long>(places.angle[k]) * (p.rotary_dim >> 2);
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
      uint4* dst = p.q_out + (first + k) * p.q_stride + h * p.head_chunks;
      dst[c0] = a4;
      dst[c1] = b4;
    }
    i += FOUR_THREADS;
    fetch_q(i);
  }
}

// Reads back the keys and values of the batch's new tokens.  A unit is 16 values: 8 bytes of codes and a scale;
// a thread has some of them on their way at a time.
template <typename T>
__global__ void __launch_bounds__(FOUR_THREADS, 5) cs_kv4_read_kernel(const __grid_constant__ Four4P p) {
  constexpr int AHEAD = 4;
  __shared__ Places places;
  cs::grid_dep_wait();
  cs::grid_dep_launch_dependents();
  const Batch& B = p.b;
  const int first = blockIdx.x * p.tokens_per_block;
  const int count = min(p.tokens_per_block, B.tokens - first), total = count * p.units;
  const int per_head = p.head_chunks >> 1;  // units of a head
  find_places<false>(p, first, count, places);
  __syncthreads();
  for (int i0 = threadIdx.x; i0 < total; i0 += AHEAD * FOUR_THREADS) {
    uint2 w[AHEAD];
    uint32_t byte[AHEAD];
    uint4* to[AHEAD];
#pragma unroll
    for (int n = 0; n < AHEAD; ++n) {
      const int i = i0 + n * FOUR_THREADS;
      to[n] = nullptr;
      if (i >= total) continue;
      const int k = __umulhi(i, p.per_unit), in = i - k * p.units;
      const int h = in >> (p.head_shift - 1), j = in & (per_head - 1);
      const bool key = p.k_out && h < B.kv_heads;  // without k_out all units are V's
      const int kh = p.k_out && !key ? h - B.kv_heads : h;
      const long long at = places.codes[k];
      if (at < 0) continue;
      w[n] = __ldg(reinterpret_cast<const uint2*>((key ? p.k_codes : p.v_codes) + (at + kh * B.head_stride) / 2 + 8 * j));
      const long long row = places.scales[k] + static_cast<long long>(kh) * B.page_size;
      byte[n] = __ldg((key ? p.k_scales : p.v_scales) + row * (p.head_chunks >> 2) + (j >> 1));
      to[n] = (key ? p.k_out + (first + k) * p.k_stride : p.v_out + (first + k) * p.v_stride) + kh * p.head_chunks + 2 * j;
    }
#pragma unroll
    for (int n = 0; n < AHEAD; ++n) {
      if (!to[n]) continue;
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
