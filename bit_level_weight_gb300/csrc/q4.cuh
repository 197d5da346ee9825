// q4.cuh - the record of a token's kv head in the 4-bit paged cache, and its
// codes as bf16.
//
// 144 bytes: 64 of key codes, 64 of value codes, 8 key scales, 8 value scales.
// 16 consecutive dimensions share a scale; a value is code * scale.
//   code   4 bits, two's complement (the append writes -7..7). Four bytes hold
//          eight dimensions: of dimensions 2i and 2i + 1 the first lies at bit
//          4i, the second at bit 16 + 4i, so that one shift and one mask leave a
//          pair in the two halves of a register
//   scale  8 bits eeeeemmm: 2^(e - 20) (1 + m / 8), no zero, no infinity, no NaN:
//          its bits shifted left by 4 and an offset are the bf16 number. The append writes
//          16..231 (2^-18..480)
// A product has 4 + 4 significant bits: exact in bf16. Zero bytes read as zeros, and
// no byte of a record stands for anything that is not finite.
//
// The codes are integers because of the way back: a pair becomes 136 + c with one
// logic instruction (bf16 counts in ones from 128 to 255) and one packed
// multiply-add takes it to c * s, (136 + c) * s - 136 * s, with nothing rounded
// (136 s = 17 * 8 s has at most 8 significant bits). Floating point codes of 4 bits
// take 11 instead of 7 integer instructions for 8 values, and are coarser for
// normally distributed ones (5.0 instead of 4.1 % of the group's largest value).
#pragma once
#include <cuda_fp16.h>

#include "common.cuh"

namespace cas {

constexpr int kRec = 144, kRecV = 64, kRecKs = 128, kRecVs = 136;
constexpr int kScaleLeast = 16, kScaleMost = 231;  // bytes that the append writes
constexpr uint32_t kScaleBias = 0x35803580u;  // 2^-20 in both halves

// Twice the scale byte `b` (0..255) as bf16.
__device__ __forceinline__ uint32_t q4_scale2(uint32_t b) { return b * 0x00100010u + kScaleBias; }
__device__ __forceinline__ uint32_t q4_fma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
// -136 s: what goes with s below.
__device__ __forceinline__ uint32_t q4_offset(uint32_t s2) { return q4_fma2(s2, 0xC308C308u, 0x80008000u); }
// The codes at bits 0..3 of both halves of w, times the halves of s2. A logic instruction
// takes one immediate: the second constant stays in a register, opaque to the compiler,
// which else makes it anew.
struct Q4Bf16 {
  uint32_t c;
  __device__ __forceinline__ Q4Bf16() { asm volatile("mov.u32 %0, 0x43084308;" : "=r"(c)); }
  __device__ __forceinline__ uint32_t pair(uint32_t w, uint32_t s2, uint32_t n2) const {
    uint32_t r;
    asm("lop3.b32 %0, %1, 0x000F000F, %2, 0x6A;" : "=r"(r) : "r"(w), "r"(c));  // (a & b) ^ c
    return q4_fma2(r, s2, n2);
  }
  // Eight dimensions in order.
  __device__ __forceinline__ uint4 word(uint32_t w, uint32_t s2, uint32_t n2) const {
    return make_uint4(pair(w, s2, n2), pair(w >> 4, s2, n2), pair(w >> 8, s2, n2), pair(w >> 12, s2, n2));
  }
};

// ---------------------------------------------------------------- as fp16
// fp16 counts in ones from 1024 to 2047, and in ones sixteen times as high in its bits from
// 64 to 127, so that the codes at bits 4..7 of a half need no shift: four pairs of a word
// take one shift instead of three.
//   bits 0..3:  (1032 + c) * s - 1032 s          bits 4..7:  (72 + c) * s - 72 s
// s is an eighth of the scale: for the scale bytes 16..231 that the append writes all
// of these are fp16 numbers and nothing is rounded.
// The second constants of both kinds in registers, as above.
struct Q4Const {
  uint32_t c0, c1;
  __device__ __forceinline__ Q4Const() {
    asm volatile("mov.u32 %0, 0x64086408;" : "=r"(c0));
    asm volatile("mov.u32 %0, 0x54805480;" : "=r"(c1));
  }
};
struct Q4Half : Q4Const {
  __half2 s, n0, n1;  // an eighth of the scales, -1032 and -72 times that
  __device__ __forceinline__ explicit Q4Half(const Q4Const& c) : Q4Const(c) {}
  // From scale bytes in the two halves.
  __device__ __forceinline__ void set(uint32_t bytes) {
    const __half2 s6 = as_half2(bytes * 0x80u + 0x04000400u);  // 2^6 scales
    s = __hmul2(s6, __float2half2_rn(0x1p-9f));
    n0 = __hmul2(s6, __float2half2_rn(-1032 * 0x1p-9f));
    n1 = __hmul2(s6, __float2half2_rn(-72 * 0x1p-9f));
  }
  static __device__ __forceinline__ __half2 as_half2(uint32_t v) { return *reinterpret_cast<__half2*>(&v); }
  static __device__ __forceinline__ uint32_t fma(uint32_t h, __half2 s, __half2 n) {
    const __half2 r = __hfma2(as_half2(h), s, n);
    return *reinterpret_cast<const uint32_t*>(&r);
  }
  // The codes at bits 0..3 (low) or 4..7 of both halves of w, as the numbers above.
  __device__ __forceinline__ uint32_t count(uint32_t w) const {
    uint32_t r;
    asm("lop3.b32 %0, %1, 0x000F000F, %2, 0x6A;" : "=r"(r) : "r"(w), "r"(c0));  // (a & b) ^ c
    return r;
  }
  __device__ __forceinline__ uint32_t count_high(uint32_t w) const {
    uint32_t r;
    asm("lop3.b32 %0, %1, 0x00F000F0, %2, 0x6A;" : "=r"(r) : "r"(w), "r"(c1));
    return r;
  }
  // Times the two scales; times the first, the second of them.
  __device__ __forceinline__ uint32_t low(uint32_t w) const { return fma(count(w), s, n0); }
  __device__ __forceinline__ uint32_t high(uint32_t w) const { return fma(count_high(w), s, n1); }
  template <int I>
  __device__ __forceinline__ uint32_t low_by(uint32_t w) const {
    return fma(count(w), I ? __high2half2(s) : __low2half2(s), I ? __high2half2(n0) : __low2half2(n0));
  }
  template <int I>
  __device__ __forceinline__ uint32_t high_by(uint32_t w) const {
    return fma(count_high(w), I ? __high2half2(s) : __low2half2(s), I ? __high2half2(n1) : __low2half2(n1));
  }
};

// ---------------------------------------------------------------- making codes
// Scale byte of 16 values, the largest of which is `top`: top / 7 rounded to four
// significant bits, to nearest even, within 2^-18..480 (an infinite one: 480).
__device__ __forceinline__ uint32_t q4_scale_byte(float top) {
  const uint32_t u = __float_as_uint(__fdiv_rn(top, 7.f));
  const int r = (int)((u + 0x7FFFFu + ((u >> 20) & 1u)) >> 20) - (107 << 3);
  return (uint32_t)min(max(r, kScaleLeast), kScaleMost);
}
__device__ __forceinline__ float q4_scale_value(uint32_t byte) { return __uint_as_float((byte + (107u << 3)) << 20); }
// x / s rounded to nearest even, -7..7 (a NaN counts as -inf). The division is a true one: quotients
// that lie in the middle of two codes are common where x is a bf16 number.
__device__ __forceinline__ uint32_t q4_code(float x, float s) {
  return (uint32_t)__float2int_rn(fminf(fmaxf(__fdiv_rn(x, s), -7.f), 7.f)) & 15u;
}
// Four bytes of eight dimensions.
__device__ __forceinline__ uint32_t q4_word(const float x[8], float s) {
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) w |= q4_code(x[i], s) << (4 * (i >> 1) + 16 * (i & 1));
  return w;
}

}  // namespace cas
