// Layout of the 4-bit KV cache and the arithmetic of its groups.
//
// A group is 16 consecutive dims of one token's key (or value) of one kv head:
// 16 e2m1 codes and one e4m3 scale; the value of a code is
// e2m1 * e4m3 * 2^exp, at most six significant bits, so it is exact in f16,
// bf16 and fp32 alike (range permitting).
//
// A record holds 16 consecutive slots of one kv head, 18 d bytes, and record
// (slot / 16, head) starts at ((slot / 16) * H_kv + head) * 18 d.  With
// P = max(1, d / 128) parts of D = d / P dims and C = D / 16:
//   K codes   [P][16 rows][D / 2]                     at 0
//   V codes   [P][2 halves][8 chunks][4][2][C]        at  8 d
//   K scales  [16 rows][d / 16]                       at 16 d
//   V scales  [P][2 halves][D / 16][4][2]             at 17 d
// where row = slot % 16 = 8 half + 2 pair + bit.  The order is that of the
// attention's matrix fragments: lane (g, t) = (lane / 4, lane % 4) of a warp
// finds the key dims it multiplies (the t-th D/4 of row g, and of row g + 8) and
// the values it multiplies (chunk g, D/8 dims, of rows 2t and 2t+1, and of
// 2t+8 and 2t+9) as one aligned vector each, and the 32 lanes' vectors are
// consecutive, so a shared-memory read of them has no bank conflict.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace upf {
namespace kv {

__host__ __device__ constexpr int record_bytes(int d) { return 18 * d; }
__host__ __device__ constexpr int part_dims(int d) { return d >= 128 ? 128 : d; }

// Byte offset inside a record of the codes of eight dims (half a group, 4 bytes):
// dims 8 oct .. 8 oct + 7 of row `row`.
__device__ __forceinline__ int k_codes(int d, int row, int oct) {
  const int D = part_dims(d), per = D / 8;
  return (oct / per) * (8 * D) + row * (D / 2) + (oct % per) * 4;
}

// Values: at D = 128 a chunk is two of these, at D = 64 one.
__device__ __forceinline__ int v_codes(int d, int row, int oct) {
  const int D = part_dims(d), C = D / 16, per = D / 8, in = oct % per;
  return 8 * d + (oct / per) * (8 * D) + (row >> 3) * (4 * D) + in * 4 / C * (8 * C) + (row & 7) * C + in * 4 % C;
}

__device__ __forceinline__ int k_scale(int d, int row, int grp) { return 16 * d + row * (d / 16) + grp; }

__device__ __forceinline__ int v_scale(int d, int row, int grp) {
  const int D = part_dims(d), per = D / 16;
  return 17 * d + (grp / per) * D + (row >> 3) * (D / 2) + (grp % per) * 8 + (row & 7);
}

// Two e4m3 bytes (low byte first) as f16x2.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t v) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(v));
  return r;
}

// The four bytes of `w` (eight e2m1 codes, low nibble first) as four f16x2.
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// Eight fp32 values as eight e2m1 codes, nearest even, saturating at 6.
__device__ __forceinline__ uint32_t f32_to_e2m1x8(const float* x) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return r;
}

__device__ __forceinline__ uint8_t f32_to_e4m3(float x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(x));
  return static_cast<uint8_t>(r & 0xFF);
}

__device__ __forceinline__ float2 half2_bits_to_float2(uint32_t h) {
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Bit patterns of |x| at and above this are infinite or NaN.
template <typename T>
constexpr uint32_t kFirstNonfinite = 0x7F80u;
template <>
constexpr uint32_t kFirstNonfinite<__half> = 0x7C00u;

__device__ __forceinline__ float2 pair_to_float2(uint32_t w, const __nv_bfloat16*) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ float2 pair_to_float2(uint32_t w, const __half*) { return half2_bits_to_float2(w); }

// Elementwise the larger magnitude (a NaN where there is one).
__device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t b, const __nv_bfloat16*) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a & 0x7FFF7FFFu), "r"(b & 0x7FFF7FFFu));
  return r;
}
__device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t b, const __half*) {
  uint32_t r;
  asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a & 0x7FFF7FFFu), "r"(b & 0x7FFF7FFFu));
  return r;
}

__device__ __forceinline__ uint32_t float2_to_pair(float a, float b, const __nv_bfloat16*) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t float2_to_pair(float a, float b, const __half*) {
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Quantise a group of 16 values (eight 32-bit words of two).  mul = 2^-exp.
//
// Every decision is the exact one, without a division.  The scale: amax * mul is
// exact (a power of two) and has at most 11 bits; a border between two e4m3
// numbers has at most five, so amax * mul / 6 is a border or differs from it by
// 2^-13 of itself or more.  The product with 1/6 is off by under 2^-22 of itself,
// and rounding it to 16 bits brings it onto a border where the exact quotient is
// one and leaves everything else on its own side.  The codes: x has at most 11 bits
// and s four, so x / s is either one of the ties 1/4, 3/4, 5/4, ... 5 exactly or at
// least 2^-13 away from it (for quotients up to 6.5).  x * (mul / s) is off by under
// 2^-18, and adding and taking away 768 rounds it to a multiple of 2^-14.
template <typename T>
__device__ __forceinline__ uint2 quantise16(const uint32_t (&w)[8], float mul, uint8_t* scale) {
  constexpr const T* kT = nullptr;
  const uint32_t m = max_abs2(max_abs2(max_abs2(w[0], w[1], kT), max_abs2(w[2], w[3], kT), kT),
                              max_abs2(max_abs2(w[4], w[5], kT), max_abs2(w[6], w[7], kT), kT), kT);
  const uint32_t top = max(m & 0x7FFFu, m >> 16 & 0x7FFFu);   // of the bit patterns: a NaN is above all
  if (top >= kFirstNonfinite<T>) {   // the whole group reads back as NaN
    *scale = 0x7F;
    return make_uint2(0u, 0u);
  }
  const float amax = pair_to_float2(top, kT).x;
  const float want = __uint_as_float((__float_as_uint(amax * mul * (1.f / 6.f)) + 0x80u) & 0xFFFFFF00u);
  const uint8_t sb = f32_to_e4m3(fminf(want, 448.f));
  const float s = half2_bits_to_float2(e4m3x2_to_f16x2(sb)).x;
  const float inv = sb ? __fdividef(mul, s) : 0.f;
  float x[16];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 v = pair_to_float2(w[i], kT);
    x[2 * i] = __fadd_rn(__fmaf_rn(v.x, inv, 768.f), -768.f);
    x[2 * i + 1] = __fadd_rn(__fmaf_rn(v.y, inv, 768.f), -768.f);
  }
  *scale = sb;
  return make_uint2(f32_to_e2m1x8(x), f32_to_e2m1x8(x + 8));
}

// Eight values in the output type: codes, scale byte, mul = 2^exp.
template <typename T>
__device__ __forceinline__ uint4 dequantise8(uint32_t codes, uint8_t scale, float mul) {
  const float s = half2_bits_to_float2(e4m3x2_to_f16x2(scale)).x * mul;
  uint32_t h[4], w[4];
  e2m1x8_to_f16(codes, h);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 v = half2_bits_to_float2(h[j]);
    w[j] = float2_to_pair(v.x * s, v.y * s, static_cast<const T*>(nullptr));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

}  // namespace kv
}  // namespace upf
