// Keys and values in 4 bits (include/cs_kv4.h): the format, and the instructions that make
// 16-bit operands of it.
//
// A group is 32 consecutive dimensions of one key (value) of one head: a scale s, an unsigned
// byte of 5 exponent and 3 mantissa bits (so a half has the byte at its bits 7 .. 14), and
// 4-bit codes c + 8 with c in -7 .. 7.  A value is s c: 4 and 3 significant bits make at most
// 7, which both 16-bit types hold, so what follows works with the values themselves and
// rounds nothing.  Of the 8 values in a 32-bit word, value 2 j lies at bit 4 j and value
// 2 j + 1 at bit 16 + 4 j: a mask then picks a pair in its 16-bit halves, in order.
//
// Code bits put under a constant exponent are a number without a conversion: the method of Kim, Henry, Fahim and
// Hassan Awadalla, "Who Says Elephants Can't Run: Bringing Large Scale MoE Models into Cloud Scale Production" (2022).
#pragma once
#include "cs_kv_append.cuh"

namespace cskv {

constexpr int GROUP4 = 32;            // dimensions of a scale
constexpr uint32_t SCALE_MOST = 0xF7;  // the largest finite scale, 61440
constexpr uint32_t SCALE_NAN = 0xFF;

// The row of a key's scales, [pages, kv_heads, page_size] (in units of head_dim / 32 bytes).
__device__ __forceinline__ long long scale_row(const Batch& B, int page, int slot, int kh) {
  return (static_cast<long long>(page) * B.kv_heads + kh) * B.page_size + slot;
}

__device__ __forceinline__ float scale_value(uint32_t byte) {
  return __half2float(__ushort_as_half(static_cast<unsigned short>(byte << 7)));
}

// The byte of the scale nearest to a finite x >= 0 (ties to the even byte), at most the largest.
__device__ __forceinline__ uint32_t scale_byte(float x) {
  if (x < 6.103515625e-05f) return __float2uint_rn(x * 131072.0f);  // below 2^-14: steps of 2^-17
  const uint32_t b = __float_as_uint(x);
  const uint32_t r = ((b + 0x7FFFFu + (b >> 20 & 1u)) >> 20) - ((127 - 15) << 3);
  return min(r, SCALE_MOST);
}

// Values 2 i, 2 i + 1 of a key's row of codes and scales.
__device__ __forceinline__ float2 four_pair(const uint8_t* codes, const uint8_t* scales, int i) {
  const uint32_t w = reinterpret_cast<const uint32_t*>(codes)[i >> 2] >> 4 * (i & 3);
  const float s = scale_value(scales[i >> 4]);
  return make_float2(s * (static_cast<int>(w & 15u) - 8), s * (static_cast<int>(w >> 16 & 15u) - 8));
}

// One scale twice, as halves (a product, because the pipe of shifts is the busy one).
__device__ __forceinline__ uint32_t scale_pair(uint32_t byte) { return byte * 0x00800080u; }

// (w & mask) | bits, in one instruction (the compiler makes two of it, with an immediate each).
__device__ __forceinline__ uint32_t masked(uint32_t w, uint32_t mask, uint32_t bits) {
  uint32_t x;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(x) : "r"(w), "r"(mask), "r"(bits));
  return x;
}

// Two scales, and what turns codes into values.
template <typename T>
struct Four;

// f16: code bits under the exponent of 1024 are 1024 + (c + 8), those of the next 4 bits 1024 + 16 (c + 8);
// c is exact, and so is s c.  (One multiply-add from there would need 1032 s, which overflows for s > 63.)
template <>
struct Four<__half> {
  __half2 s;
  // bits: the scales as halves (scale_pair)
  __device__ __forceinline__ explicit Four(uint32_t bits) { s = *reinterpret_cast<__half2*>(&bits); }
  static __device__ __forceinline__ __half2 low(uint32_t w) {
    const uint32_t x = masked(w, 0x000F000Fu, 0x64006400u), bias = 0x64086408u;  // 1032
    return __hsub2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&bias));
  }
  static __device__ __forceinline__ __half2 high(uint32_t w) {
    const uint32_t x = masked(w, 0x00F000F0u, 0x64006400u), by = 0x2C002C00u, bias = 0xD480D480u;  // 1/16, -72
    return __hfma2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&by),
                   *reinterpret_cast<const __half2*>(&bias));
  }
  // the four pairs of a word
  __device__ __forceinline__ void pairs(uint32_t w, uint32_t (&x)[4]) const {
    __half2* y = reinterpret_cast<__half2*>(x);
    y[0] = __hmul2(low(w), s);
    y[1] = __hmul2(high(w), s);
    y[2] = __hmul2(low(w >> 8), s);
    y[3] = __hmul2(high(w >> 8), s);
  }
  __device__ __forceinline__ void pairs(uint32_t w, uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) const {
    uint32_t x[4];
    pairs(w, x);
    a = x[0], b = x[1], c = x[2], d = x[3];
  }
};

// bf16: code bits under the exponent of 128 are 128 + (c + 8), and one multiply-add leaves s c: 136 s = 17 * 8 s
// has 8 significant bits at most, and nothing is near the type's limits.
template <>
struct Four<__nv_bfloat16> {
  __nv_bfloat162 s, off;
  __device__ __forceinline__ explicit Four(uint32_t bits) {
    s = __float22bfloat162_rn(__half22float2(*reinterpret_cast<__half2*>(&bits)));
    const uint32_t bias = 0xC308C308u;  // -136
    off = __hmul2(s, *reinterpret_cast<const __nv_bfloat162*>(&bias));
  }
  __device__ __forceinline__ void pairs(uint32_t w, uint32_t (&x)[4]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t y = masked(w >> 4 * i, 0x000F000Fu, 0x43004300u);
      *reinterpret_cast<__nv_bfloat162*>(&x[i]) = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&y), s, off);
    }
  }
  __device__ __forceinline__ void pairs(uint32_t w, uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) const {
    uint32_t x[4];
    pairs(w, x);
    a = x[0], b = x[1], c = x[2], d = x[3];
  }
};

// Operands of products in f16, of keys whatever the cache's type is: values times 2^-7, numbers of f16 for all scales (from
// 2^-24 on).  Code bits under the exponent of 1024 are 1024 + (c + 8), those of the next four 64 + (c + 8) under the
// exponent of 64, and one multiply-add makes either a value: 1032 s and 72 s have at most 11 significant
// bits.  Only where 1032 s overflows (BIG: bytes from 0xE0 on, values of some 55000) c is made first.
struct FourScaled {
  static constexpr uint32_t BIG_BYTE = 0xE0;
  static constexpr bool HAS_BIG = true;
  __half2 s, low, high;
  __device__ __forceinline__ explicit FourScaled(uint32_t bits) {
    const uint32_t unit = 0x20002000u, lo = 0xE408E408u, hi = 0xD480D480u;  // 2^-7, -1032, -72
    s = __hmul2(*reinterpret_cast<__half2*>(&bits), *reinterpret_cast<const __half2*>(&unit));
    low = __hmul2(s, *reinterpret_cast<const __half2*>(&lo));
    high = __hmul2(s, *reinterpret_cast<const __half2*>(&hi));
  }
  template <bool BIG>
  __device__ __forceinline__ uint32_t one(uint32_t w, uint32_t mask, uint32_t magic, uint32_t minus, __half2 off) const {
    const uint32_t x = masked(w, mask, magic);
    const __half2 h = *reinterpret_cast<const __half2*>(&x);
    const __half2 y = BIG ? __hmul2(__hadd2(h, *reinterpret_cast<const __half2*>(&minus)), s) : __hfma2(h, s, off);
    return *reinterpret_cast<const uint32_t*>(&y);
  }
  // the four pairs of a word
  template <bool BIG>
  __device__ __forceinline__ void pairs(uint32_t w, uint32_t (&x)[4]) const {
    const uint32_t v = w >> 8;
    x[0] = one<BIG>(w, 0x000F000Fu, 0x64006400u, 0xE408E408u, low);
    x[1] = one<BIG>(w, 0x00F000F0u, 0x54005400u, 0xD480D480u, high);
    x[2] = one<BIG>(v, 0x000F000Fu, 0x64006400u, 0xE408E408u, low);
    x[3] = one<BIG>(v, 0x00F000F0u, 0x54005400u, 0xD480D480u, high);
  }
};
constexpr float FOUR_UNIT = 0.0078125f;

// The same values as operands of products in bf16.  The f16 number 1024 + u has u in its lowest bits, and the same
// bits are 2^66 (128 + u) in bf16: one multiply-add makes it s c 2^-7, 136 s having 8 significant bits.  The second code of a
// byte is 64 + u in f16 after the mask, and a sum there (+ 960) puts it in place: the pipe of shifts is the busy one
// (with a shift for each of three codes 64 sequences of 16000 keys took 248 us, so 244).
struct FourScaledBf16 {
  static constexpr bool HAS_BIG = false;
  __nv_bfloat162 s, off;
  __device__ __forceinline__ explicit FourScaledBf16(uint32_t bits) {
    const uint32_t unit = 0x1B001B00u, bias = 0xE408E408u;  // 2^-73, -136 2^66
    const __nv_bfloat162 h = __float22bfloat162_rn(__half22float2(*reinterpret_cast<__half2*>(&bits)));
    s = __hmul2(h, *reinterpret_cast<const __nv_bfloat162*>(&unit));
    off = __hmul2(s, *reinterpret_cast<const __nv_bfloat162*>(&bias));
  }
  __device__ __forceinline__ uint32_t value(uint32_t x) const {
    const __nv_bfloat162 y = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x), s, off);
    return *reinterpret_cast<const uint32_t*>(&y);
  }
  __device__ __forceinline__ uint32_t high(uint32_t w) const {
    const uint32_t x = masked(w, 0x00F000F0u, 0x54005400u), up = 0x63806380u;  // 960
    const __half2 y = __hadd2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&up));
    return value(*reinterpret_cast<const uint32_t*>(&y));
  }
  // the four pairs of a word
  template <bool>
  __device__ __forceinline__ void pairs(uint32_t w, uint32_t (&x)[4]) const {
    const uint32_t v = w >> 8;
    x[0] = value(masked(w, 0x000F000Fu, 0x64006400u));
    x[1] = high(w);
    x[2] = value(masked(v, 0x000F000Fu, 0x64006400u));
    x[3] = high(v);
  }
};

template <typename T>
using OperandsOf = std::conditional_t<std::is_same<T, __half>::value, FourScaled, FourScaledBf16>;

}  // namespace cskv
