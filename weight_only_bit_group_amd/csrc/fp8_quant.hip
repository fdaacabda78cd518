// FP8 quantiser and read-back (gfx950); the format's mathematics is in fp8_device.h.
//
// All of these move bytes: 2 or 4 per value in and 1 + 4 / 128 out (1 + 4 / 16384 for 128 x 128 blocks), the
// read-back the other way round, so every access is 8 or 16 bytes a lane and several are in flight.
//   Rows: 16 lanes hold a block of 128 k, 8 values each, and share its maximum by four DPP steps. Lanes past a
// row's end hold zeros and store nothing, so the last block may have any whole number of lanes.
//   128 x 128 blocks: one workgroup holds a block in registers, 64 values a thread, so that it is read once.
#include "aq_kernels.h"
#include "fp8_device.h"

namespace aq {

namespace {

using namespace fp8;

constexpr int kThreads = 256;
constexpr int kGroups = kThreads / 16;   // blocks of 128 k that a workgroup takes at once

// ITEMS blocks a thread, all loaded before the first is used
template <bool BF16, int ITEMS>
__global__ __launch_bounds__(kThreads) void fp8_quantize_rows_kernel(const void* __restrict__ X, uint32_t items, int K,
                                                                     int64_t ldx, int nkb, uint8_t* __restrict__ codes,
                                                                     float* __restrict__ scales) {
  const int unit = threadIdx.x & 15;
  const uint32_t first = blockIdx.x * (kGroups * ITEMS) + (threadIdx.x >> 4);
  Eight<BF16> in[ITEMS];
  int64_t to[ITEMS];   // the code of the unit's first value, or -1 past a row's end
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const uint32_t item = first + i * kGroups;
    in[i].clear();
    to[i] = -1;
    if (item < items) {
      const uint32_t row = item / (uint32_t)nkb;
      const int k = (int)(item - row * nkb) * kBlock + unit * 8;
      if (k < K) {
        in[i].load(X, row * ldx + k);
        to[i] = (int64_t)row * K + k;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const uint32_t item = first + i * kGroups;
    const float s = scale_of(row_umax(in[i].amax()));
    if (to[i] >= 0) {
      float x[8];
      in[i].values(x);
      uint32_t w[2];
      codes_of<2>(x, s, w);
      *reinterpret_cast<uint64_t*>(codes + to[i]) = w[0] | ((uint64_t)w[1] << 32);
      if (unit == 0) scales[item] = s;
    }
  }
}

// one 128 x 128 block of one of E matrices a workgroup: 16 rows of 16 units at a time
template <bool BF16>
__global__ __launch_bounds__(kThreads) void fp8_quantize_blocks_kernel(const void* __restrict__ X, int N, int K, int64_t ldx,
                                                                       int nnb, int nkb, uint8_t* __restrict__ codes,
                                                                       float* __restrict__ scales) {
  __shared__ uint32_t part[kThreads / 64];
  const uint32_t at = blockIdx.x / (uint32_t)nkb, kb = blockIdx.x - at * nkb;
  const uint32_t e = at / (uint32_t)nnb, nb = at - e * nnb;
  const int k = (int)kb * kBlock + (threadIdx.x & 15) * 8;
  const int n0 = (int)nb * kBlock + (threadIdx.x >> 4);
  const int64_t row0 = (int64_t)e * N + n0;
  Eight<BF16> in[8];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (k < K && n0 + 16 * i < N) in[i].load(X, (row0 + 16 * i) * ldx + k);
    else in[i].clear();
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, in[i].amax());
  m = row_umax(m);
  m = max(m, (uint32_t)__shfl_xor((int)m, 16, 64));
  m = max(m, (uint32_t)__shfl_xor((int)m, 32, 64));
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
  __syncthreads();
  const float s = scale_of(max(max(part[0], part[1]), max(part[2], part[3])));
  if (threadIdx.x == 0) scales[blockIdx.x] = s;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (k < K && n0 + 16 * i < N) {
      float x[8];
      in[i].values(x);
      uint32_t w[2];
      codes_of<2>(x, s, w);
      *reinterpret_cast<uint64_t*>(codes + (row0 + 16 * i) * K + k) = w[0] | ((uint64_t)w[1] << 32);
    }
  }
}

// fl32(value * S), exact but for that rounding, then to bf16 where asked; the same lanes as the rows' quantiser
template <bool BF16, int ITEMS>
__global__ __launch_bounds__(kThreads) void fp8_dequantize_kernel(const uint8_t* __restrict__ codes,
                                                                  const float* __restrict__ scales, uint32_t items, int K,
                                                                  uint32_t N, bool blocks, int nnb, int nkb,
                                                                  void* __restrict__ Y) {
  const int unit = threadIdx.x & 15;
  const uint32_t first = blockIdx.x * (kGroups * ITEMS) + (threadIdx.x >> 4);
  u32x2 w[ITEMS];
  float s[ITEMS];
  int64_t to[ITEMS];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const uint32_t item = first + i * kGroups;
    to[i] = -1;
    if (item < items) {
      const uint32_t row = item / (uint32_t)nkb, kb = item - row * nkb;
      const int k = (int)kb * kBlock + unit * 8;
      if (k < K) {
        int64_t at = item;
        if (blocks) {
          const uint32_t e = row / N;
          at = ((int64_t)e * nnb + (row - e * N) / kBlock) * nkb + kb;
        }
        to[i] = (int64_t)row * K + k;
        w[i] = *reinterpret_cast<const u32x2*>(codes + to[i]);
        s[i] = scales[at];
      }
    }
  }
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    if (to[i] < 0) continue;
    float v[8];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i][j], false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i][j], true);
      v[4 * j] = lo[0] * s[i];
      v[4 * j + 1] = lo[1] * s[i];
      v[4 * j + 2] = hi[0] * s[i];
      v[4 * j + 3] = hi[1] * s[i];
    }
    if constexpr (BF16) {
      u32x4 o;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bf16x2 p = {(__bf16)v[2 * j], (__bf16)v[2 * j + 1]};
        o[j] = __builtin_bit_cast(uint32_t, p);
      }
      *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(Y) + to[i]) = o;
    } else {
      f32x4* p = reinterpret_cast<f32x4*>(static_cast<float*>(Y) + to[i]);
      p[0] = f32x4{v[0], v[1], v[2], v[3]};
      p[1] = f32x4{v[4], v[5], v[6], v[7]};
    }
  }
}

// Four blocks a thread where that still leaves every compute unit several workgroups.
constexpr int kMany = 4;
bool many_items(uint32_t items) { return items >= (uint32_t)(kGroups * kMany * 8 * device_cu_count()); }
dim3 items_grid(uint32_t items, bool many) {
  const uint32_t per = kGroups * (many ? kMany : 1);
  return dim3((items + per - 1) / per);
}

}  // namespace

hipError_t launch_fp8_quantize(const void* X, bool x_bf16, int64_t E, int64_t N, int64_t K, int64_t ldx, bool blocks,
                               uint8_t* codes, float* scales, hipStream_t stream) {
  const int nkb = (int)((K + kBlock - 1) / kBlock);
  if (blocks) {
    const int nnb = (int)((N + kBlock - 1) / kBlock);
    const dim3 grid((unsigned)(E * nnb * nkb));
    auto* kernel = x_bf16 ? fp8_quantize_blocks_kernel<true> : fp8_quantize_blocks_kernel<false>;
    hipLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, stream, X, (int)N, (int)K, ldx, nnb, nkb, codes, scales);
    return hipGetLastError();
  }
  const uint32_t items = (uint32_t)(E * N * nkb);
  const bool many = many_items(items);
  auto* kernel = x_bf16 ? many ? fp8_quantize_rows_kernel<true, kMany> : fp8_quantize_rows_kernel<true, 1>
                        : many ? fp8_quantize_rows_kernel<false, kMany> : fp8_quantize_rows_kernel<false, 1>;
  hipLaunchKernelGGL(kernel, items_grid(items, many), dim3(kThreads), 0, stream, X, items, (int)K, ldx, nkb, codes, scales);
  return hipGetLastError();
}

hipError_t launch_fp8_dequantize(const uint8_t* codes, const float* scales, int64_t E, int64_t N, int64_t K, bool blocks,
                                 void* Y, bool y_bf16, hipStream_t stream) {
  const int nkb = (int)((K + kBlock - 1) / kBlock), nnb = (int)((N + kBlock - 1) / kBlock);
  const uint32_t items = (uint32_t)(E * N * nkb);
  const bool many = many_items(items);
  auto* kernel = y_bf16 ? many ? fp8_dequantize_kernel<true, kMany> : fp8_dequantize_kernel<true, 1>
                        : many ? fp8_dequantize_kernel<false, kMany> : fp8_dequantize_kernel<false, 1>;
  hipLaunchKernelGGL(kernel, items_grid(items, many), dim3(kThreads), 0, stream, codes, scales, items, (int)K, (uint32_t)N,
                     blocks, nnb, nkb, Y);
  return hipGetLastError();
}

}  // namespace aq
