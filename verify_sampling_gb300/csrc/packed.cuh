// A paged cache in 4 bits: where a head's elements lie and how they are coded.
//
// A token's head is D / 32 groups of 32 elements; a group is 16 bytes (element j in nibble j,
// the low one of a byte first) and a scale byte b, s = 2^((b >> 3) - 20) (1 + (b & 7) / 8); an
// element is s (nibble - 8), nibble 1 .. 15.
//
// Scales of four significant bits make an element one of seven: exact in bf16, so that what
// a kernel multiplies is what the cache holds, and its code shifted left by 20 (4) bits and
// an added exponent are its bits in fp32 (bf16).  s is amax / 7 rounded to nearest, not up:
// |x / s| <= 7.44, so no element is off by more than s / 2 either way.
//
// Data are [pages, Hk, D / 32, P, 16]: a group of 8 tokens is 128 bytes side by side, a
// conflict-free 8 x 8 matrix of 16-bit words for ldmatrix, and a page's head one copy.
#pragma once

#include "common.cuh"
#include "tc.cuh"

namespace spec {
namespace q4 {

constexpr int kGroup = 32;
constexpr int kLeastExp = 107;  // fp32 exponent field of code 0

struct Cache {  // data and scales of keys and values
  const uint8_t *k, *v, *k_scale, *v_scale;
};

// Whether a page's bytes are below 2^31.
inline bool page_fits(int64_t page_size, int Hk, int D) { return page_size * Hk < ((int64_t)1 << 32) / D; }

// First byte of group 0 of a token's head (the next group is 16 P bytes on), and of its scales.
__host__ __device__ __forceinline__ int64_t data_at(int64_t page, int h, int tok, int Hk, int groups, int P) {
  return ((page * Hk + h) * groups * P + tok) * 16;
}
__host__ __device__ __forceinline__ int64_t scale_at(int64_t page, int h, int tok, int Hk, int groups, int P) {
  return ((page * Hk + h) * P + tok) * groups;
}

__device__ __forceinline__ float scale_of(uint32_t code) {
  return __uint_as_float((code << 20) + ((uint32_t)kLeastExp << 23));
}
// Code of a group's largest magnitude / 7, 255 for NaN (half a step is added to the bits: halves go up).
// The product with 1 / 7, whose nearest fp32 is 0.75 2^-24 too large, is rounded down: for a half
// way point h, 7 h is a number of 8 bits and its product (1 + 0.75 2^-24) h or h, and the number
// below 7 h is at least 4/7 of h's last place below after division, its product below h.  So
// this is the code of the rounded quotient, for every magnitude.
__device__ __forceinline__ uint32_t code_of(float amax) {
  const uint32_t bits = __float_as_uint(__fmul_rz(amax, 1.f / 7.f));  // (below 2^31, the sum of a NaN's not)
  return (uint32_t)min(max((int)((bits + (1u << 19)) >> 20) - 8 * kLeastExp, 0), 255);
}
__device__ __forceinline__ float reciprocal(float s) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  return r;
}
// N x / s to the nearest whole numbers, halves to even, for |x| < 7.5 s, as nibbles n + 8, the first
// lowest; `inv` is 1 / s within an ulp or two.
// The product with it may miss a half that the quotient meets exactly
// (16-bit values often do), so it is made a little small, and x - n s, which is exact, decides.
// The sum with 1.5 2^23 has the whole number in its low bits; what lies above them is the same for
// all and taken off the word at its end.
template <int N>
__device__ __forceinline__ uint32_t nibbles_of(const float (&x)[N], float s, float inv) {
  constexpr float kWhole = 12582912.f;
  constexpr uint32_t kWholeBits = 0x4B400000u, kOnes = 0x11111111u >> (32 - 4 * N);
  const int half = __float_as_int(0.5f * s);
  uint32_t w = 0;
  auto join = [&](float t, float rest) {
    const int odd = __float_as_int(t) & 1;
    w = w * 16u + __float_as_uint(t) + (__float_as_int(rest) + odd > half);  // (below 0: a negative int)
  };
  if constexpr (N == 1) {
    const float t = fmaf(x[0], inv, -0x1p-18f) + kWhole;
    join(t, fmaf(-(t - kWhole), s, x[0]));
  } else {
    const uint64_t inv2 = tc::pair(inv, inv), less = tc::pair(-s, -s);
#pragma unroll
    for (int e = N - 2; e >= 0; e -= 2) {
      const uint64_t x2 = tc::pair(x[e], x[e + 1]);
      const uint64_t t2 = tc::add2(tc::fma2(x2, inv2, tc::pair(-0x1p-18f, -0x1p-18f)), tc::pair(kWhole, kWhole));
      const float2 t = tc::halves(t2), rest = tc::halves(tc::fma2(tc::add2(t2, tc::pair(-kWhole, -kWhole)), less, x2));
      join(t.y, rest.y);
      join(t.x, rest.x);
    }
  }
  w += 8u * kOnes - kWholeBits * kOnes;
  return N == 8 ? w : w & (0xffffffffu >> (32 - 4 * N));
}

// ------------------------------------------------ elements in bf16 pairs --
__device__ __forceinline__ uint32_t fma_bf16(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
// Scales of a pair of elements in bf16, and -24 times them.
struct Scale {
  uint32_t s, z;
};
__device__ __forceinline__ Scale scale_bits(uint32_t bits) { return Scale{bits, fma_bf16(bits, 0xC1C0C1C0u, 0x80008000u)}; }  // -24 s - 0
constexpr uint32_t kScaleBits = ((uint32_t)kLeastExp << 7) * 0x10001u;
// From codes in the halves' low bytes, one code for both, and a code each.
__device__ __forceinline__ Scale scale_pair(uint32_t codes) { return scale_bits(codes * 16u + kScaleBits); }
__device__ __forceinline__ Scale scale_one(uint32_t code) { return scale_bits(code * 0x00100010u + kScaleBits); }
__device__ __forceinline__ Scale scale_two(uint32_t lo, uint32_t hi) { return scale_bits(hi * 0x00100000u + (lo * 16u + kScaleBits)); }
// (x & mask) | bits in one instruction, which two constants alone may become two.
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t mask, uint32_t bits) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(x), "r"(mask), "r"(bits));
  return r;
}
// Elements I and I + 4 of a word's 8 (its halves' I-th nibbles): n goes to bits 3-6 under the
// exponent of 16, which is 16 + n, and (16 + n) s - 24 s is exact, as 24 s and the result are
// numbers of six and seven bits.
template <int I>
__device__ __forceinline__ uint32_t element_pair(uint32_t w, const Scale& s) {
  const uint32_t n = I == 0 ? w * 8u : w >> (4 * I - 3);
  return fma_bf16(and_or(n, 0x00780078u, 0x41804180u), s.s, s.z);
}
// n - 8 of elements I and I + 4 in fp16 by the published conversion of small integers (Kim et al., "Who Says Elephants Can't
// Run", 2022): an integer's bits under the exponent whose unit they are, and the exponent taken off by one fma, as above in bf16
// with the scale in the same fma.  `high` is the word shifted right by 8: n lies in bits
// 0-3 under the exponent of 1024 (I even), which is 1024 + n, or in bits 4-7, 1024 + 16 n.
template <int I>
__device__ __forceinline__ uint32_t number_pair(uint32_t w, uint32_t high) {
  const uint32_t v = I < 2 ? w : high;
  uint32_t r;
  if (I % 2 == 0)
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(and_or(v, 0x000f000fu, 0x64006400u)), "r"(0x3C003C00u), "r"(0xE408E408u));  // x - 1032
  else
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(and_or(v, 0x00f000f0u, 0x64006400u)), "r"(0x2C002C00u), "r"(0xD480D480u));  // x / 16 - 72
  return r;
}

}  // namespace q4
}  // namespace spec
