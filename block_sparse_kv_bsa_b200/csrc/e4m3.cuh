// e4m3.cuh - conversions between e4m3 codes and wider types.
#pragma once

#include "common.cuh"

namespace bsa {

constexpr float kE4m3Max = 448.f;
constexpr float kAmaxFloor = 5.421010862427522e-20f;  // 2^-64

// Two floats to two codes (lo in the low byte): round to nearest even,
// values past +-448 (infinities too) to +-448, NaN to NaN.
__device__ __forceinline__ uint32_t pack_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint32_t pack_e5m2x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// The two codes of the low (high) half of w to f16 pairs, exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t w) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(w));
  return r;
}
__device__ __forceinline__ uint32_t e4m3_lo_f16x2(uint32_t w) {
  return e4m3x2_to_f16x2(static_cast<uint16_t>(w & 0xffffu));
}
__device__ __forceinline__ uint32_t e4m3_hi_f16x2(uint32_t w) {
  return e4m3x2_to_f16x2(static_cast<uint16_t>(w >> 16));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Smallest value scale, 2^-80.  A row's sum is held as the sum of weight / v with
// weights of up to 2^15, so 2^31 keys stay below 2^126.  The append writes no
// scale below 2^-64 / 448.
constexpr float kVScaleMin = 8.271806125530277e-25f;

// A block scale as read: one that is not finite and positive, or a value scale
// below its bound, is reported and counts as 1.
__device__ __forceinline__ float checked_scale(float s, float least, int32_t* d_err) {
  if (!(s > 0.f && s >= least && s <= 3.402823466e38f)) {
    report(d_err, BSA_DEV_BAD_SCALE);
    return 1.f;
  }
  return s;
}
__device__ __forceinline__ float checked_k_scale(float s, int32_t* d_err) {
  return checked_scale(s, 0.f, d_err);
}
__device__ __forceinline__ float checked_v_scale(float s, int32_t* d_err) {
  return checked_scale(s, kVScaleMin, d_err);
}

}  // namespace bsa
