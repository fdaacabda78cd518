// A router's choices grouped by expert, the gated activation between the experts' two products, and the weighted
// sum over a token's choices (gfx950).
#include <hip/hip_runtime.h>

#include "aq_kernels.h"
#include "fp8_device.h"

namespace aq {

namespace {

// ---- choices grouped by expert --------------------------------------------------------------
// A stable counting sort: choice i goes to offsets[ids[i]] + (choices before it with the same expert).  Every wave of a
// workgroup takes a run of neighbouring choices, counts its experts in LDS counters of its own, and after the
// counters' sums over waves (and workgroups) have become starts places its choices 64 at a time: lanes with the same
// expert find one another by a ballot for each bit of the index, so the order needs no atomics.  (The counting uses
// LDS atomics; sums of integers do not depend on their order.)
//   Up to kSingle choices take one workgroup and launch; more take three launches: counts of every kChunk choices,
// their prefix sums, the placing.  The choices of 16 tokens, 8 each, take 4.1 us, of 512 7.0, of 2048 15.7 (64 experts)
// in one launch; of 2049 tokens 12.6, of 4096 12.4, of 16384 (128 experts) 15, of 65536 (256) 26, of 2^20 256 in three
// (graph-replayed; the host has two launches more).
constexpr int kChunk = 4096;
constexpr int64_t kSingle = 16384;

int group_waves(int E) { return E <= 512 ? 16 : 8; }   // their counters stay below 40 KiB of LDS

__device__ __forceinline__ int id_at(const int32_t* ids, int64_t i, int64_t end, int E) {
  const int id = i < end ? ids[i] : -1;
  return id >= 0 && id < E ? id : -1;
}

// counts of this wave's run [lo, hi) in cnt[0 .. E - 1] (zeroed)
__device__ __forceinline__ void count_run(const int32_t* ids, int64_t lo, int64_t hi, int E, uint32_t* cnt) {
  for (int64_t i = lo + (threadIdx.x & 63); i < hi; i += 64) {
    const int id = id_at(ids, i, hi, E);
    if (id >= 0) atomicAdd(&cnt[id], 1u);
  }
}

// places 64 choices from i0 on, id the lane's (or -1); cnt holds the next free place of each expert
__device__ __forceinline__ void place_64(int64_t i, int64_t end, int id, int bits, int top, uint32_t* cnt, int32_t* rows,
                                         int32_t* slots) {
  const int lane = threadIdx.x & 63;
  const uint64_t below = ((uint64_t)1 << lane) - 1;
  uint64_t same = __ballot(id >= 0);
  for (int b = 0; b < bits; ++b) {
    const bool one = id >> b & 1;
    const uint64_t m = __ballot(one);
    same &= one ? m : ~m;
  }
  int slot = -1;
  wave_order();   // (the counters that the caller, or the 64 before, wrote)
  if (id >= 0) {
    const uint32_t at = cnt[id];   // (one load of all lanes, ahead of the store that depends on it)
    slot = (int)(at + __popcll(same & below));
    if ((same & ~below) == ((uint64_t)1 << lane)) cnt[id] = slot + 1;   // the last of its equals
    rows[slot] = (int)((uint32_t)i / (uint32_t)top);
  }
  if (i < end) slots[i] = slot;
}

// this wave's run
__device__ __forceinline__ void place_run(const int32_t* ids, int64_t lo, int64_t hi, int E, int bits, int top, uint32_t* cnt,
                                          int32_t* rows, int32_t* slots) {
  for (int64_t i0 = lo; i0 < hi; i0 += 64) {
    const int64_t i = i0 + (threadIdx.x & 63);
    place_64(i, hi, id_at(ids, i, hi, E), bits, top, cnt, rows, slots);
  }
}

// exclusive prefix sums over the workgroup of one value a thread, and their total
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* part, uint32_t& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  uint32_t incl = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t u = __shfl_up(incl, d, 64);
    if (lane >= d) incl += u;
  }
  __syncthreads();
  if (lane == 63) part[wave] = incl;
  __syncthreads();
  uint32_t before = 0;
  total = 0;
  for (int w = 0; w < waves; ++w) {
    if (w < wave) before += part[w];
    total += part[w];
  }
  return before + incl - v;
}

// starts [E] of the experts from this workgroup's totals; offsets [E + 1] as well
__device__ __forceinline__ void starts_of(int E, uint32_t* start, uint32_t* part, int32_t* offsets) {
  uint32_t base = 0, total = 0;
  for (int e0 = 0; e0 < E; e0 += blockDim.x) {
    const int e = e0 + threadIdx.x;
    const uint32_t before = base + block_scan(e < E ? start[e] : 0, part, total);
    if (e < E) {
      start[e] = before;
      offsets[e] = (int)before;
    }
    base += total;
  }
  if (threadIdx.x == 0) offsets[E] = (int)base;
}

// Each wave's run, at most PER choices a lane, stays in registers between the counting and the placing (loaded twice:
// 25 us for 16384 choices of 64 experts, so 15).
template <int PER>
__device__ __forceinline__ void group_single(const int32_t* ids, int C, int E, int bits, int top, int32_t* offsets,
                                             int32_t* rows, int32_t* slots, uint32_t* lds, uint32_t* part) {
  // lds: counters [waves][E], starts [E]
  const int waves = blockDim.x >> 6, wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  uint32_t* start = lds + waves * E;
  uint32_t* cnt = lds + wave * E;
  const int run = (C + waves - 1) / waves, lo = min(wave * run, C), hi = min(lo + run, C);
  int id[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) id[j] = id_at(ids, lo + 64 * j + lane, hi, E);
  for (int i = threadIdx.x; i < waves * E; i += blockDim.x) lds[i] = 0;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < PER; ++j)
    if (id[j] >= 0) atomicAdd(&cnt[id[j]], 1u);
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    uint32_t sum = 0;
    for (int w = 0; w < waves; ++w) {
      const uint32_t c = lds[w * E + e];
      lds[w * E + e] = sum;
      sum += c;
    }
    start[e] = sum;
  }
  __syncthreads();
  starts_of(E, start, part, offsets);
  __syncthreads();
  for (int e = lane; e < E; e += 64) cnt[e] += start[e];
#pragma unroll
  for (int j = 0; j < PER; ++j)
    if (lo + 64 * j < hi) place_64(lo + 64 * j + lane, hi, id[j], bits, top, cnt, rows, slots);
}

template <int PER>
__global__ __launch_bounds__(1024) void group_single_kernel(const int32_t* __restrict__ ids, int C, int E, int bits, int top,
                                                           int32_t* __restrict__ offsets, int32_t* __restrict__ rows,
                                                           int32_t* __restrict__ slots) {
  extern __shared__ uint32_t lds[];
  __shared__ uint32_t part[16];
  group_single<PER>(ids, C, E, bits, top, offsets, rows, slots, lds, part);
}

// The same by the first workgroup, the rounding of the tokens' rows to FP8 (16 lanes a block of 128) by the others: one
// launch for two small ones.  16 tokens of 2048 and 128 choices: 5.0 us, one after the other 4.6 + 4.6, and the experts'
// layer around them 94.9 and 97.2 (both in turn on the same inputs); 2048 tokens and 16384 choices 16.8, and 16.2 + 5.0.
template <int PER, bool BF16>
__global__ __launch_bounds__(1024) void group_quantize_kernel(const int32_t* __restrict__ ids, int C, int E, int bits, int top,
                                                             int32_t* __restrict__ offsets, int32_t* __restrict__ rows,
                                                             int32_t* __restrict__ slots, const void* __restrict__ X,
                                                             uint32_t items, int K, int64_t ldx, int nkb,
                                                             uint8_t* __restrict__ codes, float* __restrict__ scales) {
  extern __shared__ uint32_t lds[];
  __shared__ uint32_t part[16];
  if (blockIdx.x == 0) {
    group_single<PER>(ids, C, E, bits, top, offsets, rows, slots, lds, part);
    return;
  }
  const uint32_t item = (blockIdx.x - 1) * (blockDim.x >> 4) + (threadIdx.x >> 4);
  const uint32_t row = item / (uint32_t)nkb;
  const int k = (int)(item - row * nkb) * fp8::kBlock + (threadIdx.x & 15) * 8;
  const bool mine = item < items && k < K;
  fp8::Eight<BF16> in;
  in.clear();
  if (mine) in.load(X, row * ldx + k);
  const float s = fp8::scale_of(fp8::row_umax(in.amax()));
  if (mine) {
    float x[8];
    in.values(x);
    uint32_t w[2];
    fp8::codes_of<2>(x, s, w);
    *reinterpret_cast<uint64_t*>(codes + (int64_t)row * K + k) = w[0] | ((uint64_t)w[1] << 32);
    if ((threadIdx.x & 15) == 0) scales[item] = s;
  }
}

// chunk b's counts of every expert: counts[b E + e]
__global__ __launch_bounds__(1024) void group_count_kernel(const int32_t* __restrict__ ids, int64_t C, int E,
                                                          uint32_t* __restrict__ counts) {
  extern __shared__ uint32_t lds[];
  for (int e = threadIdx.x; e < E; e += blockDim.x) lds[e] = 0;
  __syncthreads();
  const int64_t c0 = (int64_t)blockIdx.x * kChunk, end = min(c0 + kChunk, C);
  const int run = kChunk / (int)(blockDim.x >> 6);
  const int64_t lo = min(c0 + (int64_t)(threadIdx.x >> 6) * run, end);
  count_run(ids, lo, min(lo + run, end), E, lds);
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += blockDim.x) counts[(int64_t)blockIdx.x * E + e] = lds[e];
}

// counts of all chunks become starts: of expert e in chunk b
__global__ __launch_bounds__(1024) void group_starts_kernel(int chunks, int E, uint32_t* __restrict__ counts,
                                                           int32_t* __restrict__ offsets) {
  extern __shared__ uint32_t start[];
  __shared__ uint32_t part[16];
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    uint32_t sum = 0;
#pragma unroll 8
    for (int b = 0; b < chunks; ++b) sum += counts[(int64_t)b * E + e];
    start[e] = sum;
  }
  __syncthreads();
  starts_of(E, start, part, offsets);
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    uint32_t at = start[e];
#pragma unroll 8
    for (int b = 0; b < chunks; ++b) {
      const uint32_t c = counts[(int64_t)b * E + e];
      counts[(int64_t)b * E + e] = at;
      at += c;
    }
  }
}

__global__ __launch_bounds__(1024) void group_place_kernel(const int32_t* __restrict__ ids, int64_t C, int E, int bits, int top,
                                                          const uint32_t* __restrict__ starts, int32_t* __restrict__ rows,
                                                          int32_t* __restrict__ slots) {
  extern __shared__ uint32_t lds[];   // counters [waves][E]
  const int waves = blockDim.x >> 6, wave = threadIdx.x >> 6;
  for (int i = threadIdx.x; i < waves * E; i += blockDim.x) lds[i] = 0;
  __syncthreads();
  const int64_t c0 = (int64_t)blockIdx.x * kChunk, end = min(c0 + kChunk, C);
  const int run = kChunk / waves;
  const int64_t lo = min(c0 + (int64_t)wave * run, end), hi = min(lo + run, end);
  count_run(ids, lo, hi, E, lds + wave * E);
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    uint32_t sum = starts[(int64_t)blockIdx.x * E + e];
    for (int w = 0; w < waves; ++w) {
      const uint32_t c = lds[w * E + e];
      lds[w * E + e] = sum;
      sum += c;
    }
  }
  __syncthreads();
  place_run(ids, lo, hi, E, bits, top, lds + wave * E, rows, slots);
}

// ---- gated activation, rounded to FP8 -------------------------------------------------------
// h = silu(g) u of rows [g | u], in blocks of 128 as the quantiser's rows: 16 lanes a block, 8 values each.  Moves
// bytes: 8 or 4 in, 1 + 4 / 128 out.
constexpr int kThreads = 256;
constexpr int kGroups = kThreads / 16;

template <bool BF16>
__global__ __launch_bounds__(kThreads) void swiglu_quantize_kernel(const void* __restrict__ H, uint32_t items, int I, int nkb,
                                                                   const int32_t* __restrict__ end, uint8_t* __restrict__ codes,
                                                                   float* __restrict__ scales) {
  using namespace fp8;
  const int unit = threadIdx.x & 15;
  const uint32_t item = blockIdx.x * kGroups + (threadIdx.x >> 4);
  const uint32_t row = item / (uint32_t)nkb;
  const int k = (int)(item - row * nkb) * kBlock + unit * 8;
  const bool mine = item < items && k < I && (end == nullptr || (int)row < *end);
  float x[8];
  uint32_t m = 0;
  if (mine) {
    Eight<BF16> g, u;
    g.load(H, (int64_t)row * 2 * I + k);
    u.load(H, (int64_t)row * 2 * I + I + k);
    float gv[8], uv[8];
    g.values(gv);
    u.values(uv);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] = gated(gv[i], uv[i]);
      m = max(m, abs_bits(x[i]));
    }
  }
  const float s = scale_of(row_umax(m));
  if (mine) {
    uint32_t w[2];
    codes_of<2>(x, s, w);
    *reinterpret_cast<uint64_t*>(codes + (int64_t)row * I + k) = w[0] | ((uint64_t)w[1] << 32);
    if (unit == 0) scales[item] = s;
  }
}

// ---- the sum over a token's choices ---------------------------------------------------------
// out[t] = sum_j weights[t, j] Y[slots[t, j]] in the order of j, fp32; a slot outside 0 .. R - 1 adds nothing (its
// weight and row are not looked at).  Eight columns a thread; moves bytes: 8 choices of 2048 tokens, 2048 columns of fp32
// to bf16, 143 MB, 22 us; 4096 tokens of 4096 columns, 570 MB, 110.
template <bool Y16, bool O16>
__global__ __launch_bounds__(kThreads) void combine_kernel(const void* __restrict__ Y, int64_t R, int K8,
                                                           const int32_t* __restrict__ slots, const float* __restrict__ weights,
                                                           int64_t T, int top, void* __restrict__ out) {
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int64_t t = i / K8;
  if (t >= T) return;
  const int64_t col = (i - t * K8) * 8;
  float acc[8] = {};
#pragma unroll 4
  for (int j = 0; j < top; ++j) {
    const int slot = slots[t * top + j];
    const bool in = slot >= 0 && slot < R;
    const float w = weights[t * top + j];
    fp8::Eight<Y16> y;
    y.load(Y, (in ? slot : 0) * (int64_t)K8 * 8 + col);
    float v[8];
    y.values(v);
#pragma unroll
    for (int c = 0; c < 8; ++c) acc[c] = in ? __builtin_fmaf(w, v[c], acc[c]) : acc[c];
  }
  if constexpr (O16) {
    u32x4 o;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const bf16x2 p = {(__bf16)acc[2 * c], (__bf16)acc[2 * c + 1]};
      o[c] = __builtin_bit_cast(uint32_t, p);
    }
    *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(out) + t * K8 * 8 + col) = o;
  } else {
    f32x4* p = reinterpret_cast<f32x4*>(static_cast<float*>(out) + t * K8 * 8 + col);
    p[0] = f32x4{acc[0], acc[1], acc[2], acc[3]};
    p[1] = f32x4{acc[4], acc[5], acc[6], acc[7]};
  }
}

// dweights[t, j] = sum_k dout[t, k] Y[slots[t, j], k] (0 for a slot outside); one wave a choice, fp32.  Moves bytes: 23.5
// and 101 us at the sizes above.
template <bool Y16, bool O16>
__global__ __launch_bounds__(kThreads) void combine_backward_kernel(const void* __restrict__ Y, int64_t R, int K8,
                                                                    const int32_t* __restrict__ slots, int64_t C, int top,
                                                                    const void* __restrict__ dout,
                                                                    float* __restrict__ dweights) {
  const int64_t c = (int64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6);
  if (c >= C) return;
  const int lane = threadIdx.x & 63;
  const int slot = slots[c];
  float acc = 0.0f;
  if (slot >= 0 && slot < R) {
    const int64_t t = c / top;
    for (int k = lane; k < K8; k += 64) {
      fp8::Eight<Y16> y;
      fp8::Eight<O16> d;
      y.load(Y, ((int64_t)slot * K8 + k) * 8);
      d.load(dout, (t * K8 + k) * 8);
      float yv[8], dv[8];
      y.values(yv);
      d.values(dv);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc = __builtin_fmaf(yv[i], dv[i], acc);
    }
  }
  acc = wave_sum(acc);
  if (lane == 0) dweights[c] = acc;
}

}  // namespace

size_t moe_group_workspace_bytes(int64_t C, int E) {
  return C <= kSingle ? 0 : (size_t)((C + kChunk - 1) / kChunk) * E * sizeof(uint32_t);
}

hipError_t launch_moe_group(const int32_t* ids, int64_t C, int top, int E, int32_t* offsets, int32_t* rows, int32_t* slots,
                            uint32_t* work, hipStream_t stream) {
  const int waves = group_waves(E);
  const dim3 block(64 * waves);
  int bits = 0;
  while (1 << bits < E) ++bits;
  if (C <= kSingle) {
    const int per = (int)((C + 64 * waves - 1) / (64 * waves));   // choices of a lane: at most 16, or 32 with 8 waves
    auto* kernel = per <= 2 ? group_single_kernel<2> : per <= 8 ? group_single_kernel<8>
                   : per <= 16 ? group_single_kernel<16> : group_single_kernel<32>;
    hipLaunchKernelGGL(kernel, dim3(1), block, sizeof(uint32_t) * (waves + 1) * E, stream, ids, (int)C, E, bits, top, offsets,
                       rows, slots);
    return hipGetLastError();
  }
  const int chunks = (int)((C + kChunk - 1) / kChunk);
  hipLaunchKernelGGL(group_count_kernel, dim3(chunks), block, sizeof(uint32_t) * E, stream, ids, C, E, work);
  hipLaunchKernelGGL(group_starts_kernel, dim3(1), dim3(1024), sizeof(uint32_t) * E, stream, chunks, E, work, offsets);
  hipLaunchKernelGGL(group_place_kernel, dim3(chunks), block, sizeof(uint32_t) * waves * E, stream, ids, C, E, bits, top, work,
                     rows, slots);
  return hipGetLastError();
}

hipError_t launch_moe_group_quantize(const int32_t* ids, int64_t C, int top, int E, int32_t* offsets, int32_t* rows,
                                     int32_t* slots, uint32_t* work, const void* X, bool x_bf16, int64_t T, int64_t K,
                                     int64_t ldx, uint8_t* codes, float* scales, hipStream_t stream) {
  if (C > kSingle) {
    const hipError_t e = launch_moe_group(ids, C, top, E, offsets, rows, slots, work, stream);
    return e != hipSuccess ? e : launch_fp8_quantize(X, x_bf16, 1, T, K, ldx, false, codes, scales, stream);
  }
  const int waves = group_waves(E), nkb = (int)((K + fp8::kBlock - 1) / fp8::kBlock);
  int bits = 0;
  while (1 << bits < E) ++bits;
  const uint32_t items = (uint32_t)(T * nkb);
  const int per = (int)((C + 64 * waves - 1) / (64 * waves));
  auto run = [&](auto* kernel) {
    hipLaunchKernelGGL(kernel, dim3(1 + (items + 4 * waves - 1) / (4 * waves)), dim3(64 * waves),
                       sizeof(uint32_t) * (waves + 1) * E, stream, ids, (int)C, E, bits, top, offsets, rows, slots, X, items,
                       (int)K, ldx, nkb, codes, scales);
    return hipGetLastError();
  };
  if (x_bf16)
    return run(per <= 2 ? group_quantize_kernel<2, true> : per <= 8 ? group_quantize_kernel<8, true>
               : per <= 16 ? group_quantize_kernel<16, true> : group_quantize_kernel<32, true>);
  return run(per <= 2 ? group_quantize_kernel<2, false> : per <= 8 ? group_quantize_kernel<8, false>
             : per <= 16 ? group_quantize_kernel<16, false> : group_quantize_kernel<32, false>);
}

hipError_t launch_fp8_swiglu_quantize(const void* H, bool h_bf16, int64_t M, int I, const int32_t* end, uint8_t* codes,
                                      float* scales, hipStream_t stream) {
  const int nkb = (I + 127) / 128;
  const uint32_t items = (uint32_t)(M * nkb);
  const dim3 grid((items + kGroups - 1) / kGroups);
  auto* kernel = h_bf16 ? swiglu_quantize_kernel<true> : swiglu_quantize_kernel<false>;
  hipLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, stream, H, items, I, nkb, end, codes, scales);
  return hipGetLastError();
}

hipError_t launch_moe_combine(const void* Y, bool y_bf16, int64_t R, int64_t K, const int32_t* slots, const float* weights,
                              int64_t T, int top, void* out, bool out_bf16, hipStream_t stream) {
  const int64_t threads = T * (K / 8);
  const dim3 grid((unsigned)((threads + kThreads - 1) / kThreads));
  auto* kernel = y_bf16 ? out_bf16 ? combine_kernel<true, true> : combine_kernel<true, false>
                        : out_bf16 ? combine_kernel<false, true> : combine_kernel<false, false>;
  hipLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, stream, Y, R, (int)(K / 8), slots, weights, T, top, out);
  return hipGetLastError();
}

hipError_t launch_moe_combine_backward(const void* Y, bool y_bf16, int64_t R, int64_t K, const int32_t* slots, int64_t T,
                                       int top, const void* dout, bool dout_bf16, float* dweights, hipStream_t stream) {
  const int64_t C = T * top;
  const dim3 grid((unsigned)((C + kThreads / 64 - 1) / (kThreads / 64)));
  auto* kernel = y_bf16 ? dout_bf16 ? combine_backward_kernel<true, true> : combine_backward_kernel<true, false>
                        : dout_bf16 ? combine_backward_kernel<false, true> : combine_backward_kernel<false, false>;
  hipLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, stream, Y, R, (int)(K / 8), slots, C, top, dout, dweights);
  return hipGetLastError();
}

}  // namespace aq
