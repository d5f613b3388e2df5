// What the paged key/value cache operators (include/cs_kv.h) share, and the append kernel.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>
#include <type_traits>

#include "cs_ptx.cuh"

namespace cskv {

// What every kernel of a plan reads: the batch, the cache's geometry and the
// plan's error words.
struct Batch {
  const int* cu_q;
  const int* kv_lens;
  const int* table;
  int tokens, seqs, max_q, table_cols;
  int heads, kv_heads, group;  // group = heads / kv_heads
  int page_size, page_shift, num_pages;
  long long page_stride, slot_stride, head_stride;  // cache strides in elements
  uint32_t* ctrl;
};

// ctrl words: first device error (cs_status), what did not fit, and its index; whether rows
// are to be mended (cs_kv_join_kernel), and the blocks that are through with it
enum : int { CTRL_ERROR = 0, CTRL_WHAT = 1, CTRL_INDEX = 2, CTRL_MEND = 3, CTRL_MENDED = 4, CTRL_COUNTERS = 16 };
enum : uint32_t { WHAT_LENGTHS = 1, WHAT_PAGE = 2, WHAT_POSITION = 3, WHAT_WAIT = 4 };
constexpr uint32_t ERR_INVALID = 1, ERR_WATCHDOG = 6;  // cs_status values

__device__ __forceinline__ void record(uint32_t* ctrl, uint32_t code, uint32_t what, uint32_t index) {
  if (atomicCAS(&ctrl[CTRL_ERROR], 0u, code) == 0u) {
    ctrl[CTRL_WHAT] = what;
    ctrl[CTRL_INDEX] = index;
  }
}

// Rows [t0, t0 + n) and key count m of sequence b; false (and the device error)
// where they do not fit the call.
__device__ __forceinline__ bool sequence(const Batch& B, int b, int& t0, int& n, int& m) {
  t0 = __ldg(B.cu_q + b);
  const int t1 = __ldg(B.cu_q + b + 1);
  m = __ldg(B.kv_lens + b);
  n = t1 - t0;
  if (t0 >= 0 && t1 >= t0 && t1 <= B.tokens && n <= B.max_q && m >= 0 && m <= B.table_cols * B.page_size) return true;
  record(B.ctrl, ERR_INVALID, WHAT_LENGTHS, static_cast<uint32_t>(b));
  return false;
}

// One warp, all lanes: the last sequence whose first row is <= t (it holds row t unless t
// is padding); 32 trials at a time.
__device__ __forceinline__ int sequence_of(const Batch& B, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = B.seqs;  // cu_q[lo] <= t < cu_q[hi], where they are so at all
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, at = lo + lane * step;
    const unsigned le = __ballot_sync(0xFFFFFFFFu, at < hi && __ldg(B.cu_q + at) <= t) | 1u;
    lo += (31 - __clz(le)) * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

template <typename T>
struct Pair;  // two values of the storage type in a 32-bit word
template <>
struct Pair<__half> {
  static __device__ __forceinline__ float2 get(uint32_t w) { return __half22float2(*reinterpret_cast<__half2*>(&w)); }
  static __device__ __forceinline__ uint32_t put(float a, float b) {
    __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&h);
  }
};
template <>
struct Pair<__nv_bfloat16> {
  static __device__ __forceinline__ float2 get(uint32_t w) {
    return __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&w));
  }
  static __device__ __forceinline__ uint32_t put(float a, float b) {
    __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&h);
  }
};

// ---------------------------------------------------------------- append
// (a, b) -> (a cos - b sin, b cos + a sin) for the rotated pairs of Q and K, a copy
// for the rest.  A unit is 16 values of one head: the two 8-value chunks whose
// pairs lie across them (HALF) or two neighbouring chunks (ADJACENT, and what
// is not rotated).  One thread reads and writes both, so that the rotation
// may run in place.  Bound by DRAM: every value is read and written once, the
// rotation's row of a token comes from L1 for all heads but the first.
struct AppendP {
  Batch b;
  const uint4* qkv;
  uint4* q_out;
  uint4* k_cache;
  uint4* v_cache;
  const float4* rope;
  const int* positions;
  long long qkv_stride, q_stride;  // in 16-byte chunks
  int rope_rows, rotary_dim, half, head_chunks;  // half: HALF pairing; head_chunks = head_dim / 8
  int tokens_per_block, units;  // units per token
};

constexpr int APPEND_THREADS = 256;
constexpr int APPEND_MAX_TOKENS = 32;  // per block

// Appends: (a, b) -> (a cos - b sin, b cos + a sin) for every rotated pair of Q and K in fp32,
// rounded once; K and V to their pages.  Bound by its bytes: everything is read and written
// once, 16 bytes at a time, a rotation's pair in one thread (so that Q can be rotated in
// place).  A token's page takes a chain of three or four dependent reads, which the other
// blocks of the SM cover: 40 registers a thread make it six of them.  19743 tokens of
// 32 + 2 x 8 heads of 128 (495 MB): 74 us, 6.7 TB/s, 0.98 of a plain copy's measured 6.8;
// 253 single tokens of 64 + 2 x 8 heads: 4.2 us, where one token alone takes 2.4.
template <typename T>
__global__ void __launch_bounds__(APPEND_THREADS, 6) cs_kv_append_kernel(const __grid_constant__ AppendP p) {
  __shared__ long long place[APPEND_MAX_TOKENS];  // element offset of the token's slot in a cache, -1: left out
  __shared__ int angle[APPEND_MAX_TOKENS];        // its row of the rotation table
  cs::grid_dep_wait();
  cs::grid_dep_launch_dependents();
  const Batch& B = p.b;
  const int first = blockIdx.x * p.tokens_per_block;
  const int count = min(p.tokens_per_block, B.tokens - first);
  const int per_head = p.head_chunks >> 1;  // units of a head
  const int turned = p.rotary_dim >> 4;     // of them rotated
  const int heads = B.heads + B.kv_heads;   // heads that are rotated
  // a unit is two chunks of head h: those that are rotated together, or neighbours
  auto chunk = [&](int h, int j, int second) { return p.half && j < turned && h < heads ? j + second * turned : 2 * j + second; };
  int k, h, j;  // token, head, unit of the head
  uint4 x, y;
  auto fetch = [&](int i) {
    if (i >= count * p.units) return;
    k = i / p.units;
    h = (i - k * p.units) / per_head;
    j = i - k * p.units - h * per_head;
    const uint4* src = p.qkv + (first + k) * p.qkv_stride + h * p.head_chunks;
    x = src[chunk(h, j, 0)];
    y = src[chunk(h, j, 1)];
  };
  // the tokens' places, looked up by a warp each
  for (int w = threadIdx.x >> 5; w < count; w += APPEND_THREADS / 32) {
    const int t = first + w;
    const int b = sequence_of(B, t);
    int t0, n, m;
    long long at = -1;
    int row = 0;
    if ((threadIdx.x & 31) == 0 && sequence(B, b, t0, n, m) && t >= t0 && t < t0 + n && m - n + t - t0 >= 0) {
      const int pos = m - n + t - t0;
      row = p.positions ? __ldg(p.positions + t) : pos;
      const int page = __ldg(B.table + static_cast<long long>(b) * B.table_cols + (pos >> B.page_shift));
      if (page < 0 || page >= B.num_pages)
        record(B.ctrl, ERR_INVALID, WHAT_PAGE, static_cast<uint32_t>(b));
      else if (p.rotary_dim > 0 && (row < 0 || row >= p.rope_rows))
        record(B.ctrl, ERR_INVALID, WHAT_POSITION, static_cast<uint32_t>(t));
      else
        at = page * B.page_stride + (pos & (B.page_size - 1)) * B.slot_stride;
    }
    if ((threadIdx.x & 31) == 0) {
      place[w] = at;
      angle[w] = row;
    }
  }
  fetch(threadIdx.x);
  __syncthreads();
  for (int i = threadIdx.x; i < count * p.units;) {
    const long long at = place[k];
    const bool rotate = j < turned && h < heads;
    uint4* dst;
    if (h < B.heads) {
      dst = p.q_out + (first + k) * p.q_stride + h * p.head_chunks;
    } else {
      const bool key = h < heads;
      const int kh = h - B.heads - (key ? 0 : B.kv_heads);
      dst = (key ? p.k_cache : p.v_cache) + ((at + kh * B.head_stride) >> 3);
    }
    if (rotate && at >= 0) {
      const float4* row = p.rope + static_cast<long long>(angle[k]) * (p.rotary_dim >> 2);
      // 8 cosines, 8 sines: HALF rotates (x[e], y[e]), ADJACENT neighbouring values
      const float4 ca = __ldg(row + 2 * j), cb = __ldg(row + 2 * j + 1);
      const float4 sa = __ldg(row + 2 * turned + 2 * j), sb = __ldg(row + 2 * turned + 2 * j + 1);
      const float c[8] = {ca.x, ca.y, ca.z, ca.w, cb.x, cb.y, cb.z, cb.w};
      const float s[8] = {sa.x, sa.y, sa.z, sa.w, sb.x, sb.y, sb.z, sb.w};
      uint32_t* xw = reinterpret_cast<uint32_t*>(&x);
      uint32_t* yw = reinterpret_cast<uint32_t*>(&y);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 a = Pair<T>::get(xw[e]), b = Pair<T>::get(yw[e]);
        if (p.half) {
          xw[e] = Pair<T>::put(a.x * c[2 * e] - b.x * s[2 * e], a.y * c[2 * e + 1] - b.y * s[2 * e + 1]);
          yw[e] = Pair<T>::put(b.x * c[2 * e] + a.x * s[2 * e], b.y * c[2 * e + 1] + a.y * s[2 * e + 1]);
        } else {
          xw[e] = Pair<T>::put(a.x * c[e] - a.y * s[e], a.y * c[e] + a.x * s[e]);
          yw[e] = Pair<T>::put(b.x * c[e + 4] - b.y * s[e + 4], b.y * c[e + 4] + b.x * s[e + 4]);
        }
      }
    }
    if (at >= 0) {
      dst[chunk(h, j, 0)] = x;
      dst[chunk(h, j, 1)] = y;
    }
    i += APPEND_THREADS;
    fetch(i);
  }
}

}  // namespace cskv
