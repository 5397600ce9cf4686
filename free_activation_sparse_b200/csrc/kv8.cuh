// Device helpers of the 8-bit paged key/value cache: the two byte formats, the power-of-two
// scales, and the places of a page.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "common.cuh"

namespace wina {
namespace kv8 {

constexpr int kMaxB = 8192;                  // requests of one call, at most
constexpr int kMaxPage = 128;                // places of a page, at most
constexpr int kScaleEMin = -120, kScaleEMax = 122;

// The smallest power of two s with amax <= qmax * s, from the bits of a finite amax >= 0:
// with amax = m 2^k, 1 <= m < 2, and qmax = mq 2^kq, s = 2^(k - kq + (m > mq)). Subnormal
// amax (k below -126) lands under the smallest exponent kept either way.
template <bool E4M3>
__device__ __forceinline__ float pow2_scale(uint32_t amax_bits) {
  constexpr uint32_t mq = E4M3 ? 0x600000u : 0x7E0000u;  // 448 = 1.75 2^8, 127 = 1.984375 2^6
  constexpr int kq = E4M3 ? 8 : 6;
  int e = (int)(amax_bits >> 23) - 127 - kq + ((amax_bits & 0x7FFFFFu) > mq ? 1 : 0);
  e = max(kScaleEMin, min(kScaleEMax, e));
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

// Four numbers, already divided by the scale, to four bytes: one rounding to nearest even.
template <bool E4M3>
__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) {
  if constexpr (E4M3) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
  } else {
    const uint32_t x = (uint32_t)max(-127, min(127, __float2int_rn(a))), y = (uint32_t)max(-127, min(127, __float2int_rn(b)));
    const uint32_t z = (uint32_t)max(-127, min(127, __float2int_rn(c))), w = (uint32_t)max(-127, min(127, __float2int_rn(d)));
    return __byte_perm(__byte_perm(x, y, 0x0040), __byte_perm(z, w, 0x0040), 0x5410);
  }
}

// The largest byte whose product with the scale s is finite, in all four places, where that is not
// every byte; else 0. (A number near float32's largest rounds up to a byte that stands for 2^128:
// 63.5 * 2^122 and above to 64 in int8, 248 * 2^120 and above to 256 in e4m3.)
template <bool E4M3>
__device__ __forceinline__ uint32_t byte_limit(float s) {
  if (!(s > 0x1p119f && s < INFINITY)) return 0u;
  const float top = __fdiv_rd(3.40282347e+38f, s);  // >= 1
  if (top >= (E4M3 ? 448.f : 127.f)) return 0u;
  const uint32_t b = E4M3 ? (__float_as_uint(top) >> 20) - (120u << 3) : (uint32_t)(int)top;
  return b * 0x01010101u;
}

// Four bytes, none of a larger magnitude than byte_limit's (not 0).
template <bool E4M3>
__device__ __forceinline__ uint32_t limit4(uint32_t w, uint32_t limit) {
  if constexpr (E4M3) return __vminu4(w & 0x7f7f7f7fu, limit) | (w & 0x80808080u);
  else return __vmaxs4(__vmins4(w, limit), __vneg4(limit));
}

// Holds down (limit4) the bytes of rows i, i + step, ... below n: eight at `at` of each, DH apart.
// Behind the stores of a page's rows (the new ones, and the older ones that were rounded again)
// rather than in them, where it would cost registers that every write pays for.
template <bool E4M3, int DH>
__device__ __forceinline__ void limit_rows(uint8_t* at, int i, int step, int n, uint32_t limit) {
#pragma unroll 1
  for (; i < n; i += step) {
    uint2* w = reinterpret_cast<uint2*>(at + i * DH);
    *w = make_uint2(limit4<E4M3>(w->x, limit), limit4<E4M3>(w->y, limit));
  }
}

// Four bytes to the numbers they hold (exact).
template <bool E4M3>
__device__ __forceinline__ void unpack4(uint32_t w, float (&f)[4]) {
  if constexpr (E4M3) {
    const __half2 lo = __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xffffu), __NV_E4M3));
    const __half2 hi = __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> 16), __NV_E4M3));
    const float2 a = __half22float2(lo), b = __half22float2(hi);
    f[0] = a.x;
    f[1] = a.y;
    f[2] = b.x;
    f[3] = b.y;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = (float)(int)(int8_t)(w >> (8 * i));
  }
}

// Eight consecutive elements of a bf16 or float32 row (16-byte aligned), widened.
template <bool BF16>
struct Row8 {
  uint4 w[BF16 ? 1 : 2];
  __device__ __forceinline__ void load(const void* p, int64_t at) {
    if constexpr (BF16) {
      w[0] = __ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p) + at));
    } else {
      const uint4* s = reinterpret_cast<const uint4*>(reinterpret_cast<const float*>(p) + at);
      w[0] = __ldg(s);
      w[1] = __ldg(s + 1);
    }
  }
  // a becomes the largest magnitude's bits: of bf16 rows, of the even and of the odd elements
  __device__ __forceinline__ void amax(uint32_t& a) const {
    const uint32_t* u = reinterpret_cast<const uint32_t*>(w);
#pragma unroll
    for (int i = 0; i < (BF16 ? 4 : 8); ++i) a = BF16 ? __vmaxu2(a, u[i] & 0x7fff7fffu) : max(a, u[i] & 0x7fffffffu);
  }
  __device__ __forceinline__ float get(int i) const {
    const uint32_t* u = reinterpret_cast<const uint32_t*>(w);
    if constexpr (BF16) return __uint_as_float((i & 1) ? (u[i >> 1] & 0xffff0000u) : (u[i >> 1] << 16));
    else return __uint_as_float(u[i]);
  }
};

}  // namespace kv8
}  // namespace wina
