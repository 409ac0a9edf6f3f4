// The 8-bit key/value cache: layout, and the conversion between bf16 rows and
// 8-bit blocks.
//
// A block is 64 consecutive tokens of one KV head.  Its codes c (int8, or
// e4m3) and its scale s = 2^e stand for the values c s.  e is the least
// integer with amax <= LIM 2^e (LIM = 127 or 448), and at least -100, so
//     c = round(x / s), |c| <= LIM, |c s - x| <= s / 2 (int8).
// Powers of two, instead of s = amax / LIM, cost up to one bit of the codes
// and make both directions exact: x / s has no rounding of its own (so no
// ties decided by it), and c s is a bf16 number, so rows read back from the
// cache can be stored again without a second kind of rounding.  A block that
// holds an infinity or a NaN has the scale NaN (and codes 0): everything
// that reads it becomes NaN, as it would with the bf16 rows.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "kernels.h"

namespace fsvd {

// 16-byte load of data that is read once and may have been written by the
// kernel before this one on the stream (so not through the read-only path:
// this kernel can start before that one ends).
__device__ __forceinline__ uint4 ld_once(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
// Exponent field of a bf16 magnitude (bits without sign) -> the block
// exponent e.  amax = (1 + m / 128) 2^(E - 127):
//   int8: amax <= 127 2^e   <=>  e >= E - 133, or E - 132 when 1 + m/128 > 127/64
//   e4m3: amax <= 448 2^e   <=>  e >= E - 135, or E - 134 when 1 + m/128 > 448/256
// (a subnormal or zero amax has E = 0 and falls under the floor of -100).
template <bool E4M3>
__device__ __forceinline__ int kv8_exponent(uint32_t amax) {
  const int E = (int)(amax >> 7), m = (int)(amax & 127u);
  const int e = E4M3 ? E - 135 + (m > 96 ? 1 : 0) : E - 133 + (m > 126 ? 1 : 0);
  return e < -100 ? -100 : e;
}
__device__ __forceinline__ bool kv8_finite(uint32_t amax) { return amax < 0x7f80u; }
__device__ __forceinline__ float exp2i(int e) { return __int_as_float((e + 127) << 23); }
__device__ __forceinline__ float kv8_scale(int e, bool finite) {
  return finite ? exp2i(e) : __int_as_float(0x7fc00000);
}

// Largest magnitude (as bf16 bits) of the eight bf16 in u; non-finite ones
// compare above every finite one.
__device__ __forceinline__ uint32_t amax8(const uint4& u) {
  uint32_t m = __vmaxu2(__vmaxu2(u.x & 0x7fff7fffu, u.y & 0x7fff7fffu),
                        __vmaxu2(u.z & 0x7fff7fffu, u.w & 0x7fff7fffu));
  return max(m & 0xffffu, m >> 16);
}

// Four values x (already divided by the scale) -> four codes.
template <bool E4M3>
__device__ __forceinline__ uint32_t kv8_encode4(float a, float b, float c, float d) {
  if (E4M3) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
  }
  // |x| <= 127: adding 1.5 2^23 rounds to the nearest integer (ties to even)
  // and leaves its two's complement in the low byte
  constexpr float R = 12582912.f;
  const uint32_t ab = __byte_perm(__float_as_uint(a + R), __float_as_uint(b + R), 0x0040);
  const uint32_t cd = __byte_perm(__float_as_uint(c + R), __float_as_uint(d + R), 0x0040);
  return __byte_perm(ab, cd, 0x5410);
}
// Sixteen bf16 (two 16-byte vectors) -> sixteen codes; inv = 1 / scale, or 0
// for a block that is not finite.
template <bool E4M3>
__device__ __forceinline__ uint4 kv8_encode16(const uint4& a, const uint4& b, float inv, bool finite) {
  if (!finite) return make_uint4(0, 0, 0, 0);
  uint4 r;
  r.x = kv8_encode4<E4M3>(bf_lo(a.x) * inv, bf_hi(a.x) * inv, bf_lo(a.y) * inv, bf_hi(a.y) * inv);
  r.y = kv8_encode4<E4M3>(bf_lo(a.z) * inv, bf_hi(a.z) * inv, bf_lo(a.w) * inv, bf_hi(a.w) * inv);
  r.z = kv8_encode4<E4M3>(bf_lo(b.x) * inv, bf_hi(b.x) * inv, bf_lo(b.y) * inv, bf_hi(b.y) * inv);
  r.w = kv8_encode4<E4M3>(bf_lo(b.z) * inv, bf_hi(b.z) * inv, bf_lo(b.w) * inv, bf_hi(b.w) * inv);
  return r;
}

// Two e4m3 codes -> two half-precision numbers (exact).
__device__ __forceinline__ uint32_t e4m3x2_to_h2(uint16_t w) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(w));
  return r;
}
// Four codes in w -> (w.b0, w.b1) and (w.b2, w.b3) as half pairs, exactly.
// int8: the byte 0x64 above the byte v + 128 is the half 1024 + 128 + v.
template <bool E4M3>
__device__ __forceinline__ void kv8_decode4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if (E4M3) {
    lo = e4m3x2_to_h2((uint16_t)(w & 0xffffu));
    hi = e4m3x2_to_h2((uint16_t)(w >> 16));
  } else {
    const uint32_t u = w ^ 0x80808080u;
    const __half2 bias = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
    uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    __half2 x = __hsub2(*reinterpret_cast<__half2*>(&a), bias);
    __half2 y = __hsub2(*reinterpret_cast<__half2*>(&b), bias);
    lo = *reinterpret_cast<uint32_t*>(&x);
    hi = *reinterpret_cast<uint32_t*>(&y);
  }
}
// Sixteen codes -> eight half pairs (in order, exact).
template <bool E4M3>
__device__ __forceinline__ void kv8_decode16h(const uint4& c, __half2* h) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t lo, hi;
    kv8_decode4<E4M3>(w[i], lo, hi);
    h[2 * i] = *reinterpret_cast<__half2*>(&lo);
    h[2 * i + 1] = *reinterpret_cast<__half2*>(&hi);
  }
}
// Sixteen codes (as halves) of a block with exponent e + shift -> codes for
// the exponent e: code * 2^shift rounded to nearest, ties to even; at most
// the format's limit by the choice of e.  A shift below -20 rounds every code
// to zero, as -20 does.  In half precision the product is exact wherever the
// result is not zero, and adding 1.5 * 2^10 in the same instruction rounds it
// to an integer whose two's complement is the low byte (int8).  A code of 1
// passes the int8 limit at 7, one of 2^-9 the e4m3 limit at 18: larger shifts
// occur with zero codes alone, and those above 15, which half precision does
// not hold, go in two steps.
template <bool E4M3>
__device__ __forceinline__ uint4 kv8_rescale16(__half2* h, int shift) {
  shift = shift < -20 ? -20 : shift;
  if (shift > 15) {
    if (E4M3) {
      const __half2 f = __float2half2_rn(exp2i((shift > 24 ? 24 : shift) - 15));
#pragma unroll
      for (int i = 0; i < 8; ++i) h[i] = __hmul2(h[i], f);
    }
    shift = 15;
  }
  const __half2 f = __float2half2_rn(exp2i(shift));
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (E4M3) {
      const __half2 x = __hmul2(h[2 * i], f), y = __hmul2(h[2 * i + 1], f);
      uint16_t lo, hi;
      asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(lo) : "r"(*reinterpret_cast<const uint32_t*>(&x)));
      asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(hi) : "r"(*reinterpret_cast<const uint32_t*>(&y)));
      r[i] = (uint32_t)lo | ((uint32_t)hi << 16);
    } else {
      const __half2 c = __float2half2_rn(1536.f);
      const __half2 x = __hfma2(h[2 * i], f, c), y = __hfma2(h[2 * i + 1], f, c);
      r[i] = __byte_perm(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y), 0x6420);
    }
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}
// Sixteen codes times the scale -> sixteen bf16 (exact).
template <bool E4M3>
__device__ __forceinline__ void kv8_decode16(const uint4& c, float s, uint4& a, uint4& b) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
  uint32_t o[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t lo, hi;
    kv8_decode4<E4M3>(w[i], lo, hi);
    const float2 f = __half22float2(*reinterpret_cast<__half2*>(&lo));
    const float2 g = __half22float2(*reinterpret_cast<__half2*>(&hi));
    o[2 * i] = pack_bf2(f.x * s, f.y * s);
    o[2 * i + 1] = pack_bf2(g.x * s, g.y * s);
  }
  a = make_uint4(o[0], o[1], o[2], o[3]);
  b = make_uint4(o[4], o[5], o[6], o[7]);
}

}  // namespace fsvd
