// Shared by the kernels of the paged 8-bit KV cache: the conversions of its
// two formats and the host checks of its description.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "et_common.cuh"

namespace et {
namespace {

constexpr int kPageMin = 16, kPageMax = 256;  // tokens per page, multiples of 16
constexpr int kScaleExp = 48;                 // page scales are 2^e, -48 <= e <= 48

// two codes (low byte first) -> two fp16 values; exact in both formats
template <int FMT>
__device__ __forceinline__ uint32_t f8x2_to_f16x2(uint16_t c) {
  uint32_t r;
  if (FMT == ET_KV_E4M3) asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
  else asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(r) : "h"(c));
  return r;
}
// four codes -> two pairs of fp16 values
template <int FMT>
__device__ __forceinline__ void f8x4_to_f16(uint32_t w, uint32_t &lo, uint32_t &hi) {
  lo = f8x2_to_f16x2<FMT>((uint16_t)(w & 0xffffu));
  hi = f8x2_to_f16x2<FMT>((uint16_t)(w >> 16));
}
template <int FMT>
__device__ __forceinline__ void f8x4_to_f32(uint32_t w, float (&x)[4]) {
  uint32_t lo, hi;
  f8x4_to_f16<FMT>(w, lo, hi);
  const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&lo));
  const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
  x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
}
// two fp32 values -> two codes, round to nearest even, saturating, NaN kept
template <int FMT>
__device__ __forceinline__ uint32_t f32x2_to_f8x2(float lo, float hi) {
  uint16_t r;
  if (FMT == ET_KV_E4M3) asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// four, packed in order
template <int FMT>
__device__ __forceinline__ uint32_t f32x4_to_f8x4(float x0, float x1, float x2, float x3) {
  uint32_t r;
  if (FMT == ET_KV_E4M3)
    asm("{\n .reg .b16 l, h;\n cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n mov.b32 %0, {l, h};\n}"
        : "=r"(r) : "f"(x0), "f"(x1), "f"(x2), "f"(x3));
  else
    asm("{\n .reg .b16 l, h;\n cvt.rn.satfinite.e5m2x2.f32 l, %2, %1;\n cvt.rn.satfinite.e5m2x2.f32 h, %4, %3;\n mov.b32 %0, {l, h};\n}"
        : "=r"(r) : "f"(x0), "f"(x1), "f"(x2), "f"(x3));
  return r;
}

// smallest 2^e >= amax / MAX, MAX = 0.875 * 2^TOP: amax = m 2^x with m in
// [0.5, 1) needs x - TOP when m <= 0.875, one more otherwise; x and m from the
// bits of amax (a subnormal one is below the smallest scale whatever its x)
template <int FMT>
__device__ __forceinline__ int page_exponent(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  const int x = (int)(bits >> 23) - 126;
  const int e = x - (FMT == ET_KV_E4M3 ? 9 : 16) + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return max(-kScaleExp, min(kScaleExp, e));
}
// 2^e, e a normal number's exponent
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }
template <int FMT>
__device__ __forceinline__ float page_scale(float amax) {
  return power_of_two(page_exponent<FMT>(amax));
}

inline et_status paged_cache_status(const et_paged_cache *c) {
  if (!c) return ET_ERR_INVALID_ARG;
  if (c->Hkv < 1 || c->d < 1 || c->page_size < 1 || c->num_pages < 1 || c->num_pages >= (1ll << 31))
    return ET_ERR_INVALID_ARG;
  if (c->format != ET_KV_E4M3 && c->format != ET_KV_E5M2) return ET_ERR_INVALID_ARG;
  if (c->d != 64 && c->d != 128) return ET_ERR_UNSUPPORTED;
  if (c->page_size % 16 != 0 || c->page_size > kPageMax || c->Hkv > 16384) return ET_ERR_UNSUPPORTED;
  if (c->page_stride < (long long)c->Hkv * c->page_size * c->d || c->page_stride % 16 != 0 ||
      c->page_stride >= (1ll << 40) || c->num_pages > (1ll << 62) / c->page_stride)
    return ET_ERR_INVALID_ARG;
  if (!c->k_pages || !c->v_pages || !c->k_scale || !c->v_scale) return ET_ERR_INVALID_ARG;
  if (!et_aligned(c->k_pages, 16) || !et_aligned(c->v_pages, 16) || !et_aligned(c->k_scale, 4) ||
      !et_aligned(c->v_scale, 4))
    return ET_ERR_INVALID_ARG;
  return ET_OK;
}

}  // namespace
}  // namespace et
