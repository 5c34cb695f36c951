// ar_e4m3.h -- E4M3 block quantisation in registers, shared by the codec, the compressed ring and the norm kernels.
// A 128-element block lies in the 16 lanes of one DPP row of a wave, 8 elements per lane.
#pragma once

#include "ar_device.h"

namespace ar {

constexpr int kBlock = AR_FP8_BLOCK;  // 128
constexpr int kPerLane = 8;

// E4M3 conversions use gfx950's OCP-format instructions: v_cvt_pk_fp8_f32 (two fp32 -> two codes, round to
// nearest even) and v_cvt_pk_f32_fp8 (two codes -> two exact fp32). They are not saturating: |v| >= 464 and
// +-inf would become NaN codes. The encoder never sees such values: a block's values are multiplied by
// inv = RN(448 / amax) with |v| <= amax, so |v * inv| <= 448 (1 + 2^-23)^2 < 464, which rounds to at most 448;
// the fallbacks (inv = 1 only for amax < 448 / FLT_MAX, inv = 0 for an infinite amax) keep that true or give
// NaN, which stays NaN. Over every fp32 input below 464 in magnitude these instructions round exactly as
// nearest-even E4M3 with saturation does.
typedef float f32x2 __attribute__((ext_vector_type(2)));

// Round-trip four values through E4M3: returns value(code(v)), codes packed in *codes (byte k = value k).
__device__ __forceinline__ void e4m3_round4(const float* v, float* r, uint32_t* codes) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], w, true);
  const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8(w, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(w, true);
  r[0] = lo[0];
  r[1] = lo[1];
  r[2] = hi[0];
  r[3] = hi[1];
  *codes = static_cast<uint32_t>(w);
}

// A NaN value encodes as 0x7F whatever its sign (the hardware may set the sign bit).
__device__ __forceinline__ uint32_t canonical_nan_codes(uint32_t w) {
  uint32_t out = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint32_t b = (w >> (8 * k)) & 0xFFu;
    b = (b & 0x7Fu) == 0x7Fu ? 0x7Fu : b;
    out |= b << (8 * k);
  }
  return out;
}

// Max over the 16 lanes of a row of non-negative, non-NaN floats (their bit patterns order as integers).
__device__ __forceinline__ float row16_max(float v) {
  int x = __float_as_int(v);
  x = max(x, __builtin_amdgcn_update_dpp(0, x, 0xB1, 0xF, 0xF, false));   // quad_perm [1,0,3,2]
  x = max(x, __builtin_amdgcn_update_dpp(0, x, 0x4E, 0xF, 0xF, false));   // quad_perm [2,3,0,1]
  x = max(x, __builtin_amdgcn_update_dpp(0, x, 0x141, 0xF, 0xF, false));  // row_half_mirror
  x = max(x, __builtin_amdgcn_update_dpp(0, x, 0x140, 0xF, 0xF, false));  // row_mirror
  return __int_as_float(x);
}

struct BlockScale {
  float inv, scale;
};

// The largest magnitude of a lane's values. Elements past the end of the data are held as zeros, so they never raise it;
// a NaN never compares greater, so it never counts.
template <int N> __device__ __forceinline__ float lane_amax(const float* v) {
  float m = 0.0f;
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const float a = fabsf(v[k]);
    m = a > m ? a : m;
  }
  return m;
}
__device__ __forceinline__ BlockScale scale_for(float amax) {
  const float inv = 448.0f / amax, scale = amax / 448.0f;  // amax == 0 gives inv = inf: replaced below
  const bool unit = !(amax > 0.0f) || __builtin_isinf(inv);
  return BlockScale{unit ? 1.0f : inv, unit ? 1.0f : scale};
}
// Block scale. The 16 lanes that hold the block must all call it (DPP).
__device__ __forceinline__ BlockScale block_scale(const float (&v)[kPerLane]) {
  return scale_for(row16_max(lane_amax<kPerLane>(v)));
}

}  // namespace ar
