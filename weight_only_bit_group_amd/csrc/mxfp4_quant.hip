// MXFP4 quantiser and read-back (gfx950).
//
// Format: 32 consecutive k of a row share one E8M0 byte s (the factor 2^(s - 127); 255 is
// NaN); each element is an E2M1 code (magnitudes 0, .5, 1, 1.5, 2, 3, 4, 6).  With a the
// largest |x| of the block,
//   e = max(floor(log2 a) - 2, -127)   (-127 for an all-zero block),  s = e + 127,
//   code = nearest E2M1 of x 2^-e, ties to the even code, at most 6,
// the sign bit set only on non-zero magnitudes; a block that holds a NaN or an infinity
// gets s = 255 and codes 0.  floor(log2 a) is the exponent field of a, so s is that field
// minus 2 and nothing is divided: every step is exact but the one rounding to E2M1.
//
// Both kernels move bytes: 2 or 4 per element in and 17/32 out (the read-back the other
// way round), so what counts is 16-byte accesses, several in flight per lane.  A lane
// takes 8 consecutive elements (one 16-byte load of bf16, two of fp32); four lanes hold a
// block and share its maximum by two DPP quad permutations on the bit patterns (unsigned
// order of |x|'s bits is its order, and puts NaN above everything).
// v_cvt_scalef32_pk_fp4_{f32,bf16} divides by the block's factor (only the exponent field
// of its scale operand counts, so the field 0 is 2^-127), rounds to nearest even and
// saturates: its codes equal the formula for every bf16 value at scales from 2^-127 to
// 2^125.
#include "aq_device.h"
#include "aq_kernels.h"

namespace aq {

namespace {

constexpr int kMxThreads = 256;
constexpr int kMxUnits = 4;   // 8-element units per thread, all loaded before the first is used

// max over the quad of lanes (l & ~3) .. + 3
__device__ __forceinline__ uint32_t quad_umax(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false));   // quad_perm [1, 0, 3, 2]
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false));   // quad_perm [2, 3, 0, 1]
  return v;
}

// E8M0 byte of a block from the bits of its largest |x| as fp32
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax) {
  const uint32_t e = amax >> 23;
  return e == 255u ? 255u : e < 2u ? 0u : e - 2u;
}

// the sign bit of zero magnitudes cleared ((m + 7) & 8 is 8 exactly for m = 1 .. 7), and
// all codes of a block without a finite maximum
__device__ __forceinline__ uint32_t mx_clean(uint32_t w, uint32_t s) {
  const uint32_t m = w & 0x77777777u;
  return s == 255u ? 0u : m | (w & 0x88888888u & (m + 0x77777777u));
}

template <bool BF16>
struct MxIn;
template <>
struct MxIn<true> {
  u32x4 v;
  __device__ __forceinline__ void load(const void* X, int64_t e) {
    v = *reinterpret_cast<const u32x4*>(reinterpret_cast<const uint16_t*>(X) + e);
  }
  __device__ __forceinline__ uint32_t amax() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max(m, max((v[i] << 16) & 0x7FFF0000u, v[i] & 0x7FFF0000u));
    return m;
  }
  __device__ __forceinline__ uint32_t codes(float scale) const {
    // (copies: a bit cast of a vector's element would take the vector's first bytes)
    const uint32_t p0 = v[0], p1 = v[1], p2 = v[2], p3 = v[3];
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2, p0), scale, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2, p1), scale, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2, p2), scale, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2, p3), scale, 3);
  }
};
template <>
struct MxIn<false> {
  f32x4 v[2];
  __device__ __forceinline__ void load(const void* X, int64_t e) {
    const f32x4* p = reinterpret_cast<const f32x4*>(reinterpret_cast<const float*>(X) + e);
    v[0] = p[0];
    v[1] = p[1];
  }
  __device__ __forceinline__ uint32_t amax() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i >> 2][i & 3]) & 0x7FFFFFFFu);
    return m;
  }
  __device__ __forceinline__ uint32_t codes(float scale) const {
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0][0], v[0][1], scale, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0][2], v[0][3], scale, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[1][0], v[1][1], scale, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[1][2], v[1][3], scale, 3);
  }
};

// units of 8 elements, K / 8 per row; a quad of consecutive units is one block, and the
// unit count is a multiple of four, so a quad is inside or outside as a whole
template <bool BF16>
__global__ __launch_bounds__(kMxThreads) void mxfp4_quantize_kernel(const void* __restrict__ X, int64_t units,
                                                                      int64_t ldx, int upr,
                                                                      uint8_t* __restrict__ codes,
                                                                      uint8_t* __restrict__ scales) {
  const int64_t u0 = (int64_t)blockIdx.x * (kMxThreads * kMxUnits) + threadIdx.x;
  const bool dense = ldx == (int64_t)upr * 8;
  MxIn<BF16> in[kMxUnits];
#pragma unroll
  for (int i = 0; i < kMxUnits; ++i) {
    const int64_t u = u0 + i * kMxThreads;
    if (u < units) {
      int64_t e = u * 8;
      if (!dense) {
        const int64_t row = u / upr;
        e = row * ldx + (u - row * upr) * 8;
      }
      in[i].load(X, e);
    }
  }
#pragma unroll
  for (int i = 0; i < kMxUnits; ++i) {
    const int64_t u = u0 + i * kMxThreads;
    if (u < units) {
      const uint32_t s = mx_scale_byte(quad_umax(in[i].amax()));
      const uint32_t w = mx_clean(in[i].codes(__uint_as_float(s << 23)), s);
      *reinterpret_cast<uint32_t*>(codes + u * 4) = w;
      if ((threadIdx.x & 3) == 0) scales[u >> 2] = (uint8_t)s;
    }
  }
}

template <bool BF16>
__global__ __launch_bounds__(kMxThreads) void mxfp4_dequantize_kernel(const uint8_t* __restrict__ codes,
                                                                        const uint8_t* __restrict__ scales,
                                                                        int64_t units, void* __restrict__ Y) {
  const int64_t u0 = (int64_t)blockIdx.x * (kMxThreads * kMxUnits) + threadIdx.x;
  uint32_t w[kMxUnits], s[kMxUnits];
#pragma unroll
  for (int i = 0; i < kMxUnits; ++i) {
    const int64_t u = u0 + i * kMxThreads;
    if (u < units) {
      w[i] = *reinterpret_cast<const uint32_t*>(codes + u * 4);
      s[i] = scales[u >> 2];
    }
  }
#pragma unroll
  for (int i = 0; i < kMxUnits; ++i) {
    const int64_t u = u0 + i * kMxThreads;
    if (u < units) {
      // exact in both types: two significant bits, the factor no smaller than 2^-127
      const float f = __uint_as_float(s[i] << 23);
      if constexpr (BF16) {
        const u32x4 o = {__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[i], f, 0)),
                         __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[i], f, 1)),
                         __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[i], f, 2)),
                         __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[i], f, 3))};
        *reinterpret_cast<u32x4*>(reinterpret_cast<uint16_t*>(Y) + u * 8) = o;
      } else {
        const auto a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i], f, 0);
        const auto b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i], f, 1);
        const auto c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i], f, 2);
        const auto d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i], f, 3);
        f32x4* p = reinterpret_cast<f32x4*>(reinterpret_cast<float*>(Y) + u * 8);
        p[0] = f32x4{a[0], a[1], b[0], b[1]};
        p[1] = f32x4{c[0], c[1], d[0], d[1]};
      }
    }
  }
}

unsigned mx_grid(int64_t units) {
  return (unsigned)((units + kMxThreads * kMxUnits - 1) / (kMxThreads * kMxUnits));
}

}  // namespace

hipError_t launch_mxfp4_quantize(const void* X, bool x_bf16, int64_t M, int64_t K, int64_t ldx, uint8_t* codes,
                                 uint8_t* scales, hipStream_t stream) {
  const int64_t units = M * (K / 8);
  const dim3 grid(mx_grid(units)), block(kMxThreads);
  if (x_bf16)
    hipLaunchKernelGGL((mxfp4_quantize_kernel<true>), grid, block, 0, stream, X, units, ldx, (int)(K / 8), codes, scales);
  else
    hipLaunchKernelGGL((mxfp4_quantize_kernel<false>), grid, block, 0, stream, X, units, ldx, (int)(K / 8), codes, scales);
  return hipGetLastError();
}

hipError_t launch_mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t M, int64_t K, void* Y,
                                   bool y_bf16, hipStream_t stream) {
  const int64_t units = M * (K / 8);
  const dim3 grid(mx_grid(units)), block(kMxThreads);
  if (y_bf16)
    hipLaunchKernelGGL((mxfp4_dequantize_kernel<true>), grid, block, 0, stream, codes, scales, units, Y);
  else
    hipLaunchKernelGGL((mxfp4_dequantize_kernel<false>), grid, block, 0, stream, codes, scales, units, Y);
  return hipGetLastError();
}

}  // namespace aq
