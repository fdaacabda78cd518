// FP8 (E4M3) blocks on the device: the scale of a block and the codes of its values (gfx950).
//
// A block of 128 (k of a row) or 128 x 128 values shares one fp32 scale. With a the largest |x|,
//   S = max(fl32(a / 448), 2^-126),   code = E4M3 nearest to fl32(x / S), ties to the even code,
// with the sign bit of x; a block that holds a NaN or an infinity gets S = NaN and codes 0.
// |x / S| is below 448 (1 + 2^-22), which rounds to 448: nothing saturates.
#pragma once

#include "aq_device.h"

namespace aq {
namespace fp8 {

constexpr int kBlock = 128;

// the bits of |x| order as |x| does, and put infinity and NaN above everything else
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// S of a block from the bits of its largest |x|
__device__ __forceinline__ float scale_of(uint32_t amax) {
  return amax >= 0x7F800000u ? __uint_as_float(0x7FC00000u) : fmaxf(__uint_as_float(amax) / 448.0f, 0x1p-126f);
}

// Quotients by one block's scale. fl32(x / S) is an IEEE division; with r = fl32(1 / S), q = fl32(x r) and
// fl32(q + r (x - q S)) by two fused operations is the same number (Markstein) as long as x - q S, above
// 2^-34 S where the code is not zero, is not cut off: S >= 2^-90. Smaller scales divide.
struct Quotient {
  float s, r;
  __device__ __forceinline__ explicit Quotient(float scale) : s(scale), r(1.0f / scale) {}
  __device__ __forceinline__ bool fast() const { return s >= 0x1p-90f; }
  __device__ __forceinline__ float operator()(float x) const {
    const float q = x * r;
    return __builtin_copysignf(__builtin_fmaf(__builtin_fmaf(-q, s, x), r, q), x);   // (-0 would become 0)
  }
};

// four codes, the first in the low byte (v_cvt_pk_fp8_f32: nearest, ties to even, subnormals kept)
__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) {
  int w = 0;
  w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, w, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}

// the codes of 4 N values of a block with scale s (NaN: all zero)
template <int N>
__device__ __forceinline__ void codes_of(const float (&x)[4 * N], float s, uint32_t (&out)[N]) {
  const Quotient by(s);
  if (by.fast()) {
#pragma unroll
    for (int i = 0; i < N; ++i) out[i] = pack4(by(x[4 * i]), by(x[4 * i + 1]), by(x[4 * i + 2]), by(x[4 * i + 3]));
  } else if (s < 0x1p-90f) {
    for (int i = 0; i < N; ++i) out[i] = pack4(x[4 * i] / s, x[4 * i + 1] / s, x[4 * i + 2] / s, x[4 * i + 3] / s);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) out[i] = 0;
  }
}

// max over the 16 lanes of a row, by DPP
__device__ __forceinline__ uint32_t row_umax(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false));    // quad_perm [1, 0, 3, 2]
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false));    // quad_perm [2, 3, 0, 1]
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x124, 0xF, 0xF, false));   // row_ror:4
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x128, 0xF, 0xF, false));   // row_ror:8
  return v;
}

// silu(g) u; silu(g) is g times the reciprocal of 1 + 2^(-g log2 e).  The exponent's rounding moves the power by some
// |g| 2^-23 of itself, exp2, sum and reciprocal add a few 2^-24: far below the 2^-4 of the rounding to E4M3 that
// follows.  From g = -87.34 down the reciprocal is below 2^-126 and becomes 0.
__device__ __forceinline__ float gated(float g, float u) {
  return g * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -1.44269504f)) * u;
}

// eight consecutive values of a row
template <bool BF16>
struct Eight {
  u32x4 v[BF16 ? 1 : 2];
  __device__ __forceinline__ void load(const void* X, int64_t e) {
    const u32x4* p = reinterpret_cast<const u32x4*>(static_cast<const uint8_t*>(X) + e * (BF16 ? 2 : 4));
    v[0] = p[0];
    if constexpr (!BF16) v[1] = p[1];
  }
  __device__ __forceinline__ void clear() {
    v[0] = u32x4{0, 0, 0, 0};
    if constexpr (!BF16) v[1] = v[0];
  }
  __device__ __forceinline__ void values(float (&x)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (BF16) x[i] = i & 1 ? bf16_hi(v[0][i >> 1]) : bf16_lo(v[0][i >> 1]);
      else x[i] = __uint_as_float(v[i >> 2][i & 3]);
    }
  }
  __device__ __forceinline__ uint32_t amax() const {
    float x[8];
    values(x);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, abs_bits(x[i]));
    return m;
  }
};

}  // namespace fp8
}  // namespace aq
