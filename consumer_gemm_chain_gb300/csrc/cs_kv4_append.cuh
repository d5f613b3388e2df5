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
  int tokens_per_block, units;                         // units per token
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

// c + 8 for c = x / s rounded to the nearest, ties to even, within -7 .. 7.  inv is 1 / s rounded, so x inv may miss
// a tie by a part in 2^23; a quotient that is no tie is at least 2^-13 away from one (x has at most 11 significant
// bits, s has 4), so rounding to steps of 2^-16 first puts it right: a sum with 192 does, and one with 1.5 2^23 + 8 rounds.
__device__ __forceinline__ uint32_t code_of(float x, float inv) {
  const float y = __fsub_rn(__fadd_rn(__fmul_rn(x, inv), 192.0f), 192.0f);
  return __float_as_uint(__fadd_rn(fminf(fmaxf(y, -7.0f), 7.0f), 12582920.0f)) & 15u;
}

template <typename T>
__global__ void __launch_bounds__(FOUR_THREADS, 5) cs_kv4_append_kernel(const __grid_constant__ Four4P p) {
  __shared__ Places places;
  cs::grid_dep_wait();
  cs::grid_dep_launch_dependents();
  const Batch& B = p.b;
  const int first = blockIdx.x * p.tokens_per_block;
  const int count = min(p.tokens_per_block, B.tokens - first);
  const int turned = p.rotary_dim >> 4;    // chunks that hold one half of the pairs
  const int lane = threadIdx.x & 31;
  // keys and values: chunk c of head h (V's behind K's), this lane's of the warp's 32 from i0 on
  const int kv_units = 2 * B.kv_heads * p.head_chunks, kv_total = count * kv_units;
  int k, h, c;
  uint4 x4;
  auto fetch = [&](int i0) {
    if (i0 >= kv_total) return;
    const int i = min(i0 + lane, kv_total - 1);  // (lanes behind the end go along)
    k = i / kv_units;
    h = (i - k * kv_units) / p.head_chunks;
    c = i - k * kv_units - h * p.head_chunks;
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
    // the greatest magnitude of the group (as bits: what is not finite is greater than what is)
    float y[8];
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 v = Pair<T>::get(x[e]);
      y[2 * e] = v.x, y[2 * e + 1] = v.y;
      top = max(top, max(__float_as_uint(fabsf(v.x)), __float_as_uint(fabsf(v.y))));
    }
    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
    if (at >= 0) {
      const int kh = key ? h : h - B.kv_heads;
      const bool finite = top < 0x7F800000u;
      const uint32_t byte = finite ? scale_byte(__fdiv_rn(__uint_as_float(top), 7.0f)) : SCALE_NAN;
      uint32_t word = 0x88888888u;  // zeros
      if (finite && byte != 0) {
        const float inv = __frcp_rn(scale_value(byte));
        word = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) word |= code_of(y[e], inv) << (4 * (e >> 1) + 16 * (e & 1));
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
  const int per_head = p.head_chunks >> 1, q_units = B.heads * per_head;
  for (int i = threadIdx.x; i < count * q_units; i += FOUR_THREADS) {
    const int t = i / q_units, qh = (i - t * q_units) / per_head, j = i - t * q_units - qh * per_head;
    if (places.codes[t] < 0) continue;
    const bool rotate = j < turned, apart = p.half && rotate;
    const int c0 = apart ? j : 2 * j, c1 = apart ? j + turned : 2 * j + 1;
    const uint4* src = p.qkv + (first + t) * p.qkv_stride + qh * p.head_chunks;
    uint4 a4 = src[c0], b4 = src[c1];
    uint32_t *x = reinterpret_cast<uint32_t*>(&a4), *y = reinterpret_cast<uint32_t*>(&b4);
    if (rotate) {
      // 8 cosines, 8 sines: HALF rotates (x[e], y[e]), ADJACENT neighbouring values
      const float4* angles = p.rope + static_cast<long long>(places.angle[t]) * (p.rotary_dim >> 2);
      const float4 ca = __ldg(angles + 2 * j), cb = __ldg(angles + 2 * j + 1);
      const float4 sa = __ldg(angles + 2 * turned + 2 * j), sb = __ldg(angles + 2 * turned + 2 * j + 1);
      if (apart) {
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
    uint4* dst = p.q_out + (first + t) * p.q_stride + qh * p.head_chunks;
    dst[c0] = a4;
    dst[c1] = b4;
  }
}

// Reads back the keys and values of the batch's new tokens.  A unit is 16 values: 8 bytes of codes and a scale.
template <typename T>
__global__ void __launch_bounds__(FOUR_THREADS) cs_kv4_read_kernel(const __grid_constant__ Four4P p) {
  __shared__ Places places;
  cs::grid_dep_wait();
  cs::grid_dep_launch_dependents();
  const Batch& B = p.b;
  const int first = blockIdx.x * p.tokens_per_block;
  const int count = min(p.tokens_per_block, B.tokens - first), total = count * p.units;
  const int per_head = p.head_chunks >> 1;  // units of a head
  find_places<false>(p, first, count, places);
  __syncthreads();
  for (int i = threadIdx.x; i < total; i += FOUR_THREADS) {
    const int k = i / p.units, h = (i - k * p.units) / per_head, j = i - k * p.units - h * per_head;
    const bool key = p.k_out && h < B.kv_heads;  // without k_out all units are V's
    const int kh = p.k_out && !key ? h - B.kv_heads : h;
    const long long at = places.codes[k];
    if (at < 0) continue;
    const uint2 w = *reinterpret_cast<const uint2*>((key ? p.k_codes : p.v_codes) + (at + kh * B.head_stride) / 2 + 8 * j);
    const long long row = places.scales[k] + static_cast<long long>(kh) * B.page_size;
    const Four<T> four(scale_pair((key ? p.k_scales : p.v_scales)[row * (p.head_chunks >> 2) + (j >> 1)]));
    uint32_t x[4], y[4];
    four.pairs(w.x, x);
    four.pairs(w.y, y);
    uint4* to = key ? p.k_out + (first + k) * p.k_stride : p.v_out + (first + k) * p.v_stride;
    to += kh * p.head_chunks + 2 * j;
    to[0] = make_uint4(x[0], x[1], x[2], x[3]);
    to[1] = make_uint4(y[0], y[1], y[2], y[3]);
  }
}

}  // namespace cskv
