// Products with MXFP4 weights (gfx950): dense and grouped by expert, with bf16 (A16) or
// MXFP4 (A4) activations.
//
//   A16  Y[m, n] = sum_k x[m, k] * e2m1(c[n, k]) * 2^(s[n, k / 32] - 127)
//   A4   Y[m, n] = sum_b 2^(sx[m, b] + s[n, b] - 254) sum_{k in b} e2m1(cx[m, k]) e2m1(c[n, k])
//
// with fp32 sums, stored as fp32 or rounded once to bf16.  Grouped: the rows
// offsets[e] .. offsets[e + 1] - 1 of Y belong to expert e and are multiplied with its
// weights; row r reads activation row rows[r] (or r without a row list).
//
// A16 runs on the bf16 matrix instructions: the weights' values have two significant bits
// and an exponent in bf16's range, so v_cvt_scalef32_pk_bf16_fp4 turns a code pair and its
// block factor into the exact bf16 pair (row by row: fp32 multiply-adds).  A4 runs on the
// block-scaled matrix instructions, which take the codes and the E8M0 bytes as they are: four
// times the bf16 rate, and the products of one block are exact.
//
// A block of a row is 32 k, 16 bytes of codes: one lane's operand of one A4 instruction
// and of four A16 instructions.  A sum may take its k in any order as long as both
// operands agree, so the lane groups of an instruction are given the blocks whose
// scale bytes lie side by side in memory, and one dword serves four instructions.
//
// Rows of scale bytes start at any address (K / 32 bytes apart), so they are loaded
// through registers with unaligned loads, 16 bytes (512 k) a row at a time.
//
// The lanes that a ragged edge leaves over read clamped addresses inside the same row or
// the last row; the activations (or both scale bytes) of a block past K are zero, rows
// past the end are not stored.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdio>
#include <iterator>
#include <type_traits>

#include "aq_device.h"
#include "aq_kernels.h"
#include "gemm_lds.h"
#include "gemm_tiles.h"

namespace aq {

namespace {

using namespace gemm;

typedef int i32x8 __attribute__((ext_vector_type(8)));

struct MxArgs {
  const uint8_t* X;        // A16: bf16 rows; A4: code rows
  const uint8_t* XS;       // A4: scale rows
  int64_t xrow;            // bytes between rows of X
  const uint8_t* W;        // [E, N, K/2]
  const uint8_t* WS;       // [E, N, K/32]
  int M, N, K;             // M: rows of Y
  const int32_t* offsets;  // grouped: [E + 1]
  const int32_t* rows;     // grouped: [M] activation rows, or NULL
  int E, T;                // experts; rows of X
  void* Y;
};

// The tile kernel's matrix instructions, accumulating in place in AGPRs.  Written out because
// the compiler gives a 16 x 16 instruction another destination than its addend and then moves
// accumulators about (60 moves for 64 instructions in the loop).  It does not see the hazards
// either: s_nop 1 covers an operand that a VALU instruction wrote just before (free, the matrix
// core is busy with the instruction before), settle() the results' first reads after the loop:
// eight wait states have to lie between a result and its reader, and an accumulator is copied
// nowhere before settle() (tests/test_mxfp4_code.py walks the compiled code for both).  A kernel
// whose accumulators meet at a branch must not use these: the compiler may copy them there, ahead
// of any wait that follows.
template <int Q>   // the scale byte of both dwords that applies
__device__ __forceinline__ void mfma_a4(f32x4& c, u32x4 x, u32x4 w, uint32_t sx, uint32_t sw) {
  asm volatile("s_nop 1\n\tv_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:[%5,%5,0] "
               "op_sel_hi:[%6,%6,0] cbsz:4 blgp:4"
               : "+a"(c) : "v"(x), "v"(w), "v"(sx), "v"(sw), "n"(Q & 1), "n"(Q >> 1));
}
__device__ __forceinline__ void mfma_a16(f32x4& c, u32x4 x, bf16x8 w) {
  asm volatile("s_nop 1\n\tv_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(c) : "v"(x), "v"(w));
}
template <int FM, int FN>
__device__ __forceinline__ void settle(f32x4 (&acc)[FM][FN]) {
  asm volatile("s_nop 15\n\ts_nop 7" ::: "memory");
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) asm volatile("" : "+a"(acc[i][j]));
}

// the four bf16 pairs of code dword w times the block factor f
__device__ __forceinline__ bf16x8 mx_bf16x8(uint32_t w, float f) {
  const u32x4 v = {__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, f, 0)),
                   __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, f, 1)),
                   __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, f, 2)),
                   __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, f, 3))};
  return __builtin_bit_cast(bf16x8, v);
}

__device__ __forceinline__ i32x8 codes8(u32x4 v) {
  return i32x8{(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0};
}

// ---- single rows, A16 ----------------------------------------------------------------------
// Every row of Y by itself, a block of it for each 4 NR / NW columns; bound by the weight bytes,
// so every wave has all it can in flight: NR weight rows, a 16-byte unit (a block of 32 k) of
// each per lane and 2048 k, straight to registers, the next 2048 k requested before these are
// used.  The products are fp32 fused multiply-adds of the weights' exact fp32 values (1.5 VALU
// operations a weight; the matrix instructions of the form below would leave 15 of 16 rows
// empty, and its LDS ring holds fewer bytes in flight: one row on [11008, 2048] 5.0 against 6.3
// us, on [2048, 11008] 5.3 against 9.2, 8 experts' rows of [1536, 2048] 5.9 against 7.9,
// graph-replayed).  NW waves of a block share long rows ([2048, 11008] by one wave each 8.8),
// their sums are added in wave order.
//   More rows read the weights again, which the L2 holds for small ones: several rows take this
// form too where tiles of 16 rows would leave the device empty (16 rows on [512, 2048] 3.6
// against 4.3 us, 40 on [70, 576] 3.0 against 3.4, 64 on [94, 31424] 22.9 against 25.8, two on
// [11008, 2048] 6.3 of either form).
template <int NR_, int NW_>
struct MxVec {
  static constexpr bool SPLIT = true, VEC = true;
  static constexpr int NR = NR_, NW = NW_;
  static constexpr int NT = 256;
  static constexpr int BM = 1, BN = 4 / NW * NR;
  static constexpr int KS = 2048;
  static constexpr int TILE_BYTES = 4096 + 1088 * BN;   // a stage's activations, codes and scale bytes
  static constexpr int PER_CU = 8;                      // blocks that a compute unit holds
  static int describe(char* to, size_t n) { return snprintf(to, n, "vec %d over %d", NR, NW); }
  static_assert(4 % NW == 0, "whole groups of waves");
};

template <class C, bool GROUPED, bool BF16>
__global__ __launch_bounds__(C::NT) void mxfp4_gemv_kernel(MxArgs a) {
  __shared__ float part[C::NW > 1 ? 4 * C::NR : 1];
  const int lane = threadIdx.x & 63;
  const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tiles_n = (a.N + C::BN - 1) / C::BN;
  Tile t;
  if constexpr (GROUPED) {
    if (!grouped_tile<C::BM>(a, tiles_n, C::BN, blockIdx.x, t)) return;   // the whole block
  } else {
    const int i = tile_of_block(blockIdx.x, a.M * tiles_n);
    t.e = 0;
    t.r0 = i % a.M;
    t.n0 = (i / a.M) * C::BN;
  }
  const int nblk = a.K >> 5;
  const int n0 = t.n0 + wid / C::NW * C::NR;
  const uint8_t *wrow[C::NR], *srow[C::NR];
#pragma unroll
  for (int r = 0; r < C::NR; ++r) {
    const int64_t n = (int64_t)t.e * a.N + min(n0 + r, a.N - 1);
    wrow[r] = a.W + n * (a.K >> 1);
    srow[r] = a.WS + n * nblk;
  }
  const int src = GROUPED ? source_row(a, t.r0) : t.r0;
  const uint8_t* xrow = a.X + (int64_t)max(src, 0) * a.xrow;

  float acc[C::NR];
#pragma unroll
  for (int r = 0; r < C::NR; ++r) acc[r] = 0.0f;
  u32x4 w[C::NR];
  uint32_t sc[C::NR];
  auto fetch = [&](int b0) {
    const int b = min(b0 + lane, nblk - 1);
#pragma unroll
    for (int r = 0; r < C::NR; ++r) {
      w[r] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(wrow[r] + 16 * b));
      sc[r] = srow[r][b];
    }
  };
  int b0 = 64 * (wid % C::NW);
  if (b0 < nblk) fetch(b0);
  for (; b0 < nblk; b0 += 64 * C::NW) {
    const int b = min(b0 + lane, nblk - 1);
    u32x4 x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = *reinterpret_cast<const u32x4*>(xrow + 64 * b + 16 * i);
      if (b0 + lane >= nblk) x[i] = u32x4{0, 0, 0, 0};   // past the row
    }
    u32x4 wnow[C::NR];
    float f[C::NR];
#pragma unroll
    for (int r = 0; r < C::NR; ++r) {
      wnow[r] = w[r];
      f[r] = __uint_as_float(sc[r] << 23);
    }
    if (b0 + 64 * C::NW < nblk) fetch(b0 + 64 * C::NW);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float xf[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        xf[2 * j] = __uint_as_float(x[i][j] << 16);
        xf[2 * j + 1] = __uint_as_float(x[i][j] & 0xffff0000u);
      }
#pragma unroll
      for (int r = 0; r < C::NR; ++r) {
        const uint32_t c = wnow[r][i];
        const auto v0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, f[r], 0);
        const auto v1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, f[r], 1);
        const auto v2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, f[r], 2);
        const auto v3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, f[r], 3);
        const float v[8] = {v0[0], v0[1], v1[0], v1[1], v2[0], v2[1], v3[0], v3[1]};
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[r] = __builtin_fmaf(xf[j], v[j], acc[r]);
      }
    }
  }

  wave_sums<C::NR>(acc);
  auto store = [&](int r, float v) {
    if (n0 + r < a.N) store_one<BF16>(a.Y, (int64_t)t.r0 * a.N + n0 + r, src < 0 ? __builtin_nanf("") : v);
  };
  const bool owner = wave_sums_owner<C::NR>(lane);
  if constexpr (C::NW == 1) {
    if (owner) {
#pragma unroll
      for (int j = 0; j < wave_sums_out<C::NR>; ++j) store(wave_sums_index<C::NR>(j, lane >> 4), acc[j]);
    }
  } else {
    if (owner) {
#pragma unroll
      for (int j = 0; j < wave_sums_out<C::NR>; ++j) part[wid * C::NR + wave_sums_index<C::NR>(j, lane >> 4)] = acc[j];
    }
    __syncthreads();
    if (wid % C::NW == 0 && lane < C::NR) {
      float v = part[wid * C::NR + lane];
#pragma unroll
      for (int w = 1; w < C::NW; ++w) v += part[(wid + w) * C::NR + lane];
      store(lane, v);
    }
  }
}

// ---- few rows -----------------------------------------------------------------------------
// Bound by the weight bytes (and from some ten rows on by the activation bytes that every
// block reads from its L2).  A block's NW waves share K: each takes a contiguous run of
// stages (A4: 256 k, A16: 64 k) of the (16 FM) x (16 FN) tile through LDS buffers of its own,
// filled by its own LDS-DMA loads, so there is no barrier before the sums are joined: a wave
// only waits for its own oldest loads, with R stages in flight.  The LDS layout and the
// order of the weight rows are those of the larger tiles below; the scale bytes come straight
// to the lanes that use them, 16 bytes of a row at a time.  A wave may run out of stages at any of
// them, so accumulators meet at branches: the matrix instructions are builtins, whose waits the
// compiler keeps (against inline assembly with its own wait at every stage's end: 16 rows on
// [4096, 14336] 13.9 against 14.3 us (A16) and 8.0 against 8.3 (A4), 36 products 2% on average).
//   16 rows, graph-replayed, over several runs: on [11008, 2048] 6.7 to 7.1 us (A16) and 4.6 to 5.0
// (A4), on [4096, 14336] 13.3 to 14.3 and 8.0 to 8.1; there the blocks of 16 columns read 118 MB of
// activations beside 31 MB of weights, some 40 bytes a clock and compute unit.
template <int ROWB>
__device__ __forceinline__ int lds_unit(int r, int u) {
  return ROWB == 128 ? u ^ ((r >> 1) & 7) : u ^ ((r >> 3) & 1);
}

// 16 scale bytes from byte `at` of a row of nblk, zeros past its end
__device__ __forceinline__ u32x4 scales16(const uint8_t* row, int at, int nblk) {
  if (nblk >= 16) {
    const int from = min(at, nblk - 16);
    const unsigned __int128 v = load_any<unsigned __int128>(row + from);
    const int sh = 8 * (at - from);
    return __builtin_bit_cast(u32x4, sh < 128 ? v >> sh : (unsigned __int128)0);
  }
  unsigned __int128 v = 0;
  for (int i = at; i < nblk; ++i) v |= (unsigned __int128)row[i] << (8 * (i - at));
  return __builtin_bit_cast(u32x4, v);
}

template <bool A4_, int FM_, int FN_, int NW_, int R_>
struct MxSplit {
  static constexpr bool A4 = A4_;
  static constexpr int FM = FM_, FN = FN_, NW = NW_, R = R_;
  static constexpr int BM = 16 * FM, BN = 16 * FN, NT = 64 * NW;
  static constexpr int KS = A4 ? 256 : 64;
  static constexpr int WB = A4 ? 128 : 32;
  static constexpr int A_DMA = 2 * FM;
  static constexpr int B_DMA = A4 ? 2 * FN : (FN + 1) / 2;
  static constexpr int DMA = A_DMA + B_DMA;
  static constexpr int STAGE = 1024 * DMA;                  // LDS bytes of a wave's stage
  static constexpr int SB = KS / 32;
  static constexpr int SC = 16 / SB;                        // stages whose scale bytes are loaded at once
  static constexpr int PART = 4 * FM * FN * 64 * 4;         // bytes of a wave's sums
  static constexpr int LDS = NW * (R * STAGE > PART ? R * STAGE : PART);
  static constexpr bool SPLIT = true, VEC = false;
  static constexpr int TILE_BYTES = BM * 128 + BN * WB;
  static constexpr int PER_CU = std::max(1, std::min(160 * 1024 / LDS, 32 / NW));   // blocks that a compute unit holds
  static int describe(char* to, size_t n) { return snprintf(to, n, "split %d x %d over %d", FM, FN, NW); }
  static_assert((R - 1) * DMA < 64, "the loads in flight are counted in six bits");
};

template <class C, bool GROUPED, bool BF16>
__global__ __launch_bounds__(C::NT) void mxfp4_split_kernel(MxArgs a) {
  extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
  const int lane = threadIdx.x & 63;
  const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const int tiles_n = (a.N + C::BN - 1) / C::BN;
  Tile t;
  if constexpr (GROUPED) {
    if (!grouped_tile<C::BM>(a, tiles_n, C::BN, blockIdx.x, t)) return;   // the whole block
  } else {
    // the row tiles of a column run side by side: they share its weights in the L2
    const int tiles_m = (a.M + C::BM - 1) / C::BM;
    const int i = tile_of_block(blockIdx.x, tiles_m * tiles_n);
    t.e = 0;
    t.r0 = (i % tiles_m) * C::BM;
    t.r1 = min(t.r0 + C::BM, a.M);
    t.n0 = (i / tiles_m) * C::BN;
  }
  const int nblk = a.K >> 5, krow = a.K >> 1;
  const int stages = (a.K + C::KS - 1) / C::KS;
  const int first = (int)((int64_t)wid * stages / C::NW), end = (int)((int64_t)(wid + 1) * stages / C::NW);
  uint8_t* mine = lds + wid * C::R * C::STAGE;

  auto brow = [&](int i) { return min(C::FN * (i & 15) + (i >> 4), a.N - 1 - t.n0); };
  auto xrow = [&](int i) -> int64_t {
    const int r = min(t.r0 + i, t.r1 - 1);
    return GROUPED ? max(source_row(a, r), 0) : r;
  };
  constexpr int WU = C::WB / 16;
  const int aunit = lds_unit<128>(lane >> 3, lane & 7);
  const int bunit = lds_unit<C::WB>(lane / WU, lane % WU);
  const int64_t wfirst = (int64_t)t.e * a.N + t.n0;
  const uint8_t* wtile = a.W + wfirst * krow;
  uint32_t asrc[C::A_DMA], bsrc[C::B_DMA];
#pragma unroll
  for (int j = 0; j < C::A_DMA; ++j) asrc[j] = (uint32_t)((xrow(8 * j + (lane >> 3)) * a.xrow) >> 4) + (aunit ^ (4 * (j & 1)));
#pragma unroll
  for (int j = 0; j < C::B_DMA; ++j) {
    // (rows past the tile, when it has fewer than a load covers: the last row again)
    const int i = min((64 / WU) * j + lane / WU, C::BN - 1);
    bsrc[j] = (uint32_t)brow(i) * (uint32_t)krow + 16u * (C::A4 ? bunit ^ (4 * (j & 1)) : bunit);
  }
  // units past the row's end in a part-filled last stage: its last unit instead
  const int left = a.K - (stages - 1) * C::KS;
  auto issue = [&](int s, int slot) {
    const uint8_t* x = a.X + (int64_t)s * 128;
    const uint8_t* w = uniform(wtile + (int64_t)s * C::WB);
    const bool tail = s == stages - 1;
    const uint32_t base = lds_addr(mine + slot * C::STAGE);
#pragma unroll
    for (int j = 0; j < C::A_DMA; ++j) {
      const int back = max((aunit ^ (4 * (j & 1))) - (C::A4 ? left >> 5 : left >> 3) + 1, 0);
      dma16_at(x + 16 * (uint64_t)(asrc[j] - (tail ? back : 0)), __builtin_amdgcn_readfirstlane(base + 1024 * j));
    }
#pragma unroll
    for (int j = 0; j < C::B_DMA; ++j) {
      const int back = max((C::A4 ? bunit ^ (4 * (j & 1)) : bunit) - (left >> 5) + 1, 0);
      dma16_from(w, bsrc[j] - (tail ? 16 * back : 0), __builtin_amdgcn_readfirstlane(base + 1024 * (C::A_DMA + j)));
    }
  };

  const uint8_t* wscale[C::FN];
  const uint8_t* xscale[C::A4 ? C::FM : 1];
#pragma unroll
  for (int j = 0; j < C::FN; ++j) wscale[j] = a.WS + (wfirst + brow(16 * j + l16)) * nblk;
#pragma unroll
  for (int i = 0; i < C::FM; ++i)
    if constexpr (C::A4) xscale[i] = a.XS + xrow(16 * i + l16) * nblk;

  f32x4 acc[C::FM][C::FN];
#pragma unroll
  for (int i = 0; i < C::FM; ++i)
#pragma unroll
    for (int j = 0; j < C::FN; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

#pragma unroll
  for (int s = 0; s < C::R; ++s)
    if (first + s < end) issue(first + s, s);
  u32x4 sw[C::FN], sx[C::FM];
  auto fetch_scales = [&](int s) {
#pragma unroll
    for (int j = 0; j < C::FN; ++j) sw[j] = scales16(wscale[j], s * C::SB, nblk);
    if constexpr (C::A4) {
#pragma unroll
      for (int i = 0; i < C::FM; ++i) sx[i] = scales16(xscale[i], s * C::SB, nblk);
    }
  };
  auto row = [&](const uint8_t* tile, int r, int u) { return *reinterpret_cast<const u32x4*>(tile + 128 * r + 16 * lds_unit<128>(r, u)); };
  // stage s, the ST-th of those whose scale bytes are at hand
  auto stage = [&](int s, auto st_) {
    constexpr int ST = decltype(st_)::value;
    if (s >= end) return;
    const int slot = (s - first) % C::R;
    if (s + C::R < end) asm volatile("s_waitcnt vmcnt(%0)" ::"n"((C::R - 1) * C::DMA) : "memory");
    else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    const uint8_t* xt = mine + slot * C::STAGE;
    const uint8_t* wt = xt + 1024 * C::A_DMA;
    const int valid = nblk - s * C::SB;
    u32x4 x[2][C::FM];
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int i = 0; i < C::FM; ++i) {
        x[q][i] = row(xt, 16 * i + l16, C::A4 ? 4 * q + g : 2 * g + q);
        if (!C::A4 && (g >> 1) >= valid) x[q][i] = u32x4{0, 0, 0, 0};
      }
    if constexpr (C::A4) {
      u32x4 w[2][C::FN];
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int j = 0; j < C::FN; ++j) w[q][j] = row(wt, 16 * j + l16, 4 * q + g);
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      if (s + C::R < end) issue(s + C::R, slot);
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int i = 0; i < C::FM; ++i)
#pragma unroll
          for (int j = 0; j < C::FN; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(codes8(x[q][i]), codes8(w[q][j]), acc[i][j], 4, 4, 0,
                                                                         sx[i][2 * ST + q] >> (8 * g), 0,
                                                                         sw[j][2 * ST + q] >> (8 * g));
    } else {
      uint64_t wc[C::FN];
#pragma unroll
      for (int j = 0; j < C::FN; ++j) {
        const int r = 16 * j + l16;
        wc[j] = *reinterpret_cast<const uint64_t*>(wt + 32 * r + 16 * lds_unit<32>(r, g >> 1) + 8 * (g & 1));
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      if (s + C::R < end) issue(s + C::R, slot);
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int j = 0; j < C::FN; ++j) {
          const uint32_t byte = (sw[j][ST >> 1] >> (16 * (ST & 1) + 8 * (g >> 1))) & 255u;
          const bf16x8 b = mx_bf16x8((uint32_t)(wc[j] >> (32 * q)), __uint_as_float(byte << 23));
#pragma unroll
          for (int i = 0; i < C::FM; ++i)
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x[q][i]), b, acc[i][j], 0, 0, 0);
        }
    }
  };
  for (int s = first; s < end; s += C::SC) {
    fetch_scales(s);
    stage(s, std::integral_constant<int, 0>{});
    stage(s + 1, std::integral_constant<int, 1>{});
    if constexpr (C::SC == 8) {
      stage(s + 2, std::integral_constant<int, 2>{});
      stage(s + 3, std::integral_constant<int, 3>{});
      stage(s + 4, std::integral_constant<int, 4>{});
      stage(s + 5, std::integral_constant<int, 5>{});
      stage(s + 6, std::integral_constant<int, 6>{});
      stage(s + 7, std::integral_constant<int, 7>{});
    }
  }

  // ---- the waves' sums, added in wave order; lane c of operand j: column FN c + j ----
  float* part = reinterpret_cast<float*>(lds);
  __syncthreads();   // (every wave has read its last stage)
#pragma unroll
  for (int i = 0; i < C::FM; ++i)
#pragma unroll
    for (int v = 0; v < 4; ++v)
#pragma unroll
      for (int j = 0; j < C::FN; ++j) part[(((wid * C::FM + i) * 4 + v) * C::FN + j) * 64 + lane] = acc[i][j][v];
  __syncthreads();
  const int col = t.n0 + C::FN * l16;
  for (int o = wid; o < 4 * C::FM; o += C::NW) {
    float sum[C::FN];
#pragma unroll
    for (int j = 0; j < C::FN; ++j) sum[j] = part[(o * C::FN + j) * 64 + lane];
#pragma unroll
    for (int w = 1; w < C::NW; ++w)
#pragma unroll
      for (int j = 0; j < C::FN; ++j) sum[j] += part[((w * 4 * C::FM + o) * C::FN + j) * 64 + lane];
    const int r = t.r0 + 16 * (o >> 2) + 4 * g + (o & 3);
    if (r < t.r1) {
      if (GROUPED && source_row(a, r) < 0) {
#pragma unroll
        for (int j = 0; j < C::FN; ++j) sum[j] = __builtin_nanf("");
      }
      store_row<BF16, C::FN>(a, (int64_t)r * a.N + col, col, sum);
    }
  }
}

// ---- many rows ----------------------------------------------------------------------------
// WM x WN waves, each a (16 FM) x (16 FN) tile of 16 x 16 outputs.  (Against 32 x 32 x 64 and
// 32 x 32 x 16 the instructions 16 x 16 x 128 and 16 x 16 x 32 touch each accumulator half as
// often: on random operands, where the card's power sets the clock, 7.1 against 6.3 PFLOP/s
// and 2.0 against 1.8 in a loop of nothing else that adds in place; on zeros both run at 2.4 GHz,
// 9.6 and 2.4.)  K advances in stages of 128 bytes of an
// activation row (A4: 256 k, A16: 64 k) through two LDS buffers filled by LDS-DMA, one
// barrier a stage.  The scale bytes of two stages are loaded at once, through registers.
// A tile row keeps its 16-byte units permuted so that the 16 rows which a phase of a
// ds_read takes fall into all 64 banks: unit u of row r is at u ^ ((r >> 1) & 7) in rows of
// 128 bytes, at u ^ ((r >> 3) & 1) in rows of 32.
// The weight rows of a wave are stored so that lane c of its FN operands holds rows
// FN c .. FN c + FN - 1: its outputs of one row are neighbours and leave in one store, 16
// lanes 64 to 256 contiguous bytes.
//   M = 4096 on [11008, 2048], bf16 out, graph-replayed: A4 67 us (2.7 PFLOP/s), A16 159 to 163 (1.15);
// M = N = 4096, K = 14336: A4 118 (4.1), A16 364 (1.32).  A stage's matrix instructions are 2048
// cycles of the 3050 (A4) and 2850 (A16) that it takes, the LDS is active for 990 and 1160; a tile
// of 2048 k spends 36% (A4) and 10% (A16) of its cycles outside its loop, where the one block of a
// compute unit leaves the matrix cores idle, and 688 tiles are 2.7 rounds.  The cycles are the same
// on zeros, at 2.39 GHz (A4 51 us) in place of the 1.95 that the card's power allows on random
// operands.  Deeper rings, larger wave tiles, 32 x 32 instructions and two blocks a compute unit
// were within 5% or slower.
template <bool A4_, int WM_, int WN_, int FM_, int FN_>
struct MxCfg {
  static constexpr bool A4 = A4_;
  static constexpr int WM = WM_, WN = WN_, FM = FM_, FN = FN_;
  static constexpr int NW = WM * WN, NT = 64 * NW;
  static constexpr int BM = 16 * FM * WM, BN = 16 * FN * WN;
  static constexpr int KS = A4 ? 256 : 64;           // k per stage, two instructions
  static constexpr int XB = 128;                     // activation bytes per row and stage
  static constexpr int WB = A4 ? 128 : 32;           // weight bytes per row and stage
  static constexpr int A_DMA = BM * XB / 1024 / NW;  // loads per wave and stage, 1 KiB each
  static constexpr int B_DMA = BN * WB / 1024 / NW;
  static constexpr int DMA = A_DMA + B_DMA;
  static constexpr int SB = KS / 32;                 // scale bytes per row and stage
  static constexpr int CB = 2 * SB;                  // and per row and chunk of two stages
  static constexpr int SROWS = A4 ? BM + BN : BN;    // rows of scale bytes
  static constexpr int SPT = (SROWS + NT - 1) / NT;  // of them per thread
  static constexpr bool SPLIT = false, VEC = false;
  static constexpr int TILE_BYTES = BM * XB + BN * WB;
  // blocks that a compute unit holds; their registers leave room for 8 waves, or 12
  static constexpr int PER_CU = std::max(1, std::min(160 * 1024 / (2 * (BM * XB + BN * WB)), (FM * FN >= 16 ? 8 : 12) / NW));
  static int describe(char* to, size_t n) { return snprintf(to, n, "tile %d x %d of %d x %d", WM, WN, FM, FN); }
  static_assert(BM * XB % (1024 * NW) == 0 && BN * WB % (1024 * NW) == 0, "whole loads per wave");
};

// the 4 x 4 bytes of v transposed: byte j of word i becomes byte i of word j
__device__ __forceinline__ u32x4 transpose4(u32x4 v) {
  const uint32_t a = __builtin_amdgcn_perm(v[1], v[0], 0x05010400u), b = __builtin_amdgcn_perm(v[1], v[0], 0x07030602u);
  const uint32_t c = __builtin_amdgcn_perm(v[3], v[2], 0x05010400u), d = __builtin_amdgcn_perm(v[3], v[2], 0x07030602u);
  return u32x4{__builtin_amdgcn_perm(c, a, 0x05040100u), __builtin_amdgcn_perm(c, a, 0x07060302u),
               __builtin_amdgcn_perm(d, b, 0x05040100u), __builtin_amdgcn_perm(d, b, 0x07060302u)};
}

template <class C, bool GROUPED, bool BF16>
__global__ __launch_bounds__(C::NT, 1) void mxfp4_tile_kernel(MxArgs a) {
  __shared__ __attribute__((aligned(1024))) uint8_t As[2][C::BM * C::XB];
  __shared__ __attribute__((aligned(1024))) uint8_t Bs[2][C::BN * C::WB];
  __shared__ __attribute__((aligned(16))) uint8_t Ss[2][C::SROWS * C::CB];
  __shared__ uint8_t lost[GROUPED ? C::BM : 1];
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wid = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wid / C::WN, wn = wid % C::WN;
  const int l16 = lane & 15, g = lane >> 4;
  const int tiles_n = (a.N + C::BN - 1) / C::BN;
  Tile t;
  if constexpr (GROUPED) {
    if (!grouped_tile<C::BM>(a, tiles_n, C::BN, blockIdx.x, t)) return;   // the whole block
  } else {
    // groups of row tiles walked column by column, so the tiles that an XCD runs together
    // share their rows and columns in its L2
    const int tiles_m = (a.M + C::BM - 1) / C::BM;
    const int i = tile_of_block(blockIdx.x, tiles_m * tiles_n);
    const int gmax = max(1, (tiles_m + 7) / 8);
    const int grp = i / (gmax * tiles_n);
    const int gm = min(tiles_m - grp * gmax, gmax);
    const int within = i - grp * gmax * tiles_n;
    t.e = 0;
    t.r0 = __builtin_amdgcn_readfirstlane((grp * gmax + within % gm) * C::BM);
    t.r1 = min(t.r0 + C::BM, a.M);
    t.n0 = __builtin_amdgcn_readfirstlane((within / gm) * C::BN);
  }
  const int nblk = a.K >> 5;
  const int last = (a.K + C::KS - 1) / C::KS - 1;   // the last stage, perhaps part-filled
  const int krow = a.K >> 1;                        // bytes of a code row

  // ---- sources of the LDS-DMA loads ----
  // weight row of LDS row i, from the tile's first: wave region i / (16 FN), operand
  // (i / 16) % FN, lane i % 16
  auto brow = [&](int i) {
    const int n = (i / (16 * C::FN)) * (16 * C::FN) + C::FN * (i & 15) + (i / 16) % C::FN;
    return min(n, a.N - 1 - t.n0);
  };
  auto xrow = [&](int i) -> int64_t {
    const int r = min(t.r0 + i, t.r1 - 1);
    return GROUPED ? max(source_row(a, r), 0) : r;
  };
  const int64_t wfirst = (int64_t)t.e * a.N + t.n0;
  const uint8_t* wtile = a.W + wfirst * krow;
  // load j of wave w covers 8 activation rows (A4: or weight rows) or 32 weight rows from 8
  // (32) (j NW + w) on; the unit that a lane fetches is the same in all of them, since
  // their rows differ by whole periods of the permutation, 16 rows
  constexpr int WU = C::WB / 16;
  const int aunit = lds_unit<128>(8 * wid + (lane >> 3), lane & 7);
  const int bunit = lds_unit<C::WB>((64 / WU) * wid + lane / WU, lane % WU);
  static_assert(C::NW % 2 == 0, "the permutation's period");
  uint32_t asrc[C::A_DMA];   // units from X (X is below 2^36 bytes)
  uint32_t bsrc[C::B_DMA];   // bytes from wtile; below 2^31 for K < 2^22
#pragma unroll
  for (int j = 0; j < C::A_DMA; ++j)
    asrc[j] = (uint32_t)((xrow(8 * (j * C::NW + wid) + (lane >> 3)) * a.xrow) >> 4) + aunit;
#pragma unroll
  for (int j = 0; j < C::B_DMA; ++j)
    bsrc[j] = (uint32_t)brow((64 / WU) * (j * C::NW + wid) + lane / WU) * (uint32_t)krow + 16u * bunit;
  // In a part-filled last stage the units past the row's end read its last unit instead.  A
  // unit is 32 k of an A4 row and of a weight row, 8 k of a bf16 row.
  const int left = a.K - last * C::KS;
  const uint32_t aback = max(aunit - (C::A4 ? left >> 5 : left >> 3) + 1, 0);
  const uint32_t bback = 16 * max(bunit - (left >> 5) + 1, 0);
  struct Source { const uint8_t *x, *w; uint32_t aback, bback; };
  auto source = [&](int s) {
    return Source{a.X + (int64_t)s * C::XB, uniform(wtile + (int64_t)s * C::WB), s == last ? aback : 0u, s == last ? bback : 0u};
  };
  auto issue_one = [&](const Source& f, int buf, int j) {
    if (j < C::A_DMA)
      dma16_at(f.x + 16 * (uint64_t)(asrc[j] - f.aback), lds_addr(&As[buf][1024 * (C::NW * j + wid)]));
    else
      dma16_from(f.w, bsrc[j - C::A_DMA] - f.bback, lds_addr(&Bs[buf][1024 * (C::NW * (j - C::A_DMA) + wid)]));
  };
  auto issue = [&](int s, int buf) {
    const Source f = source(s);
#pragma unroll
    for (int j = 0; j < C::DMA; ++j) issue_one(f, buf, j);
  };

  // the loads of stage s that go out after the products of the i-th of n row blocks
  auto issue_slice = [&](int s, int buf, int i, int n) {
    const Source f = source(s);
#pragma unroll
    for (int j = 0; j < C::DMA; ++j)
      if (j >= i * C::DMA / n && j < (i + 1) * C::DMA / n) issue_one(f, buf, j);
  };

  // ---- scale bytes: CB per row and chunk of two stages, through registers ----
  using Sword = std::conditional_t<C::A4, unsigned __int128, uint32_t>;
  const uint8_t* ssrc[C::SPT];
  Sword sreg[C::SPT];
#pragma unroll
  for (int j = 0; j < C::SPT; ++j) {
    const int i = min(j * C::NT + tid, C::SROWS - 1);
    ssrc[j] = C::A4 && i < C::BM ? a.XS + xrow(i) * nblk : a.WS + (wfirst + brow(C::A4 ? i - C::BM : i)) * nblk;
  }
  // of a chunk that the row ends in: its last CB bytes; those of the chunk before are
  // shifted out when the word is written, so the bytes past the row's end are zero
  int sshift = 0;
  auto load_scales = [&](int c) {
    const int at = min(c * C::CB, nblk - C::CB);
    sshift = 8 * (c * C::CB - at);
#pragma unroll
    for (int j = 0; j < C::SPT; ++j) sreg[j] = load_any<Sword>(ssrc[j] + at);
  };
  auto load_short = [&]() {   // rows of fewer than CB bytes
#pragma unroll
    for (int j = 0; j < C::SPT; ++j) {
      sreg[j] = 0;
      for (int i = 0; i < nblk; ++i) sreg[j] |= (Sword)ssrc[j][i] << (8 * i);
    }
  };
  // A4: byte 4 q + g, block g of instruction q of the chunk, goes to byte q of dword g,
  // which is what lane group g reads
  auto write_scales = [&](int buf) {
#pragma unroll
    for (int j = 0; j < C::SPT; ++j) {
      const Sword v = sshift < 8 * C::CB ? sreg[j] >> sshift : 0;
      if ((j + 1) * C::NT <= C::SROWS || j * C::NT + tid < C::SROWS) {
        uint8_t* to = &Ss[buf][C::CB * (j * C::NT + tid)];
        if constexpr (C::A4) *reinterpret_cast<u32x4*>(to) = transpose4(__builtin_bit_cast(u32x4, v));
        else *reinterpret_cast<Sword*>(to) = v;
      }
    }
  };

  f32x4 acc[C::FM][C::FN];
#pragma unroll
  for (int i = 0; i < C::FM; ++i)
#pragma unroll
    for (int j = 0; j < C::FN; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  const int am = wm * 16 * C::FM + l16, bn = wn * 16 * C::FN + l16;   // this lane's first LDS rows
  // A stage is two steps of FM x FN instructions.  A4: lane group g takes block 4 q + g of
  // the stage in step q.  A16: it takes 16 k, units 2 g and 2 g + 1 of its activation row
  // and half of block g / 2 of its weight row, 8 k a step.  Operands are read a step ahead:
  // the activations of row block i into the registers that its products have just used,
  // A4's weights into a second set.
  u32x4 xr[C::FM];
  u32x4 wr[2][C::FN];              // A4: the two steps' codes
  uint64_t wc[C::FN], wcnext[C::FN];   // A16: the stage's codes
  uint32_t sa[C::FM], sb[C::FN], sbnext[C::FN];   // A4: the chunk's scale bytes; A16: sb, the stage's
  auto load_x = [&](int buf, int q, int i) {
    const int r = am + 16 * i;
    xr[i] = *reinterpret_cast<const u32x4*>(&As[buf][128 * r + 16 * lds_unit<128>(r, C::A4 ? 4 * q + g : 2 * g + q)]);
  };
  auto load_w = [&](int buf, int q) {
#pragma unroll
    for (int j = 0; j < C::FN; ++j) {
      const int r = bn + 16 * j;
      wr[q][j] = *reinterpret_cast<const u32x4*>(&Bs[buf][128 * r + 16 * lds_unit<128>(r, 4 * q + g)]);
    }
  };
  auto load_wc = [&](int buf, int st, int chunk) {
#pragma unroll
    for (int j = 0; j < C::FN; ++j) {
      const int r = bn + 16 * j;
      wcnext[j] = *reinterpret_cast<const uint64_t*>(&Bs[buf][32 * r + 16 * lds_unit<32>(r, g >> 1) + 8 * (g & 1)]);
      sbnext[j] = Ss[chunk & 1][4 * r + 2 * st + (g >> 1)];
    }
  };
  auto load_sa = [&](int chunk, int i) {
    sa[i] = *reinterpret_cast<const uint32_t*>(&Ss[chunk & 1][16 * (am + 16 * i) + 4 * g]);
  };
  auto load_sb = [&](int chunk) {
#pragma unroll
    for (int j = 0; j < C::FN; ++j)
      sbnext[j] = *reinterpret_cast<const uint32_t*>(&Ss[chunk & 1][16 * (C::BM + bn + 16 * j) + 4 * g]);
  };
  auto take = [&](bool fresh) {   // the scale bytes (and A16's codes) requested last
#pragma unroll
    for (int j = 0; j < C::FN; ++j) {
      if (C::A4 ? fresh : true) sb[j] = sbnext[j];
      if constexpr (!C::A4) wc[j] = wcnext[j];
    }
  };
  // A16: the bf16 weights of step q from the stage's codes
  bf16x8 b[C::FN];
  auto convert = [&](int q) {
    if constexpr (!C::A4) {
#pragma unroll
      for (int j = 0; j < C::FN; ++j) b[j] = mx_bf16x8((uint32_t)(wc[j] >> (32 * q)), __uint_as_float(sb[j] << 23));
    }
  };
  // the products of row blocks from .. to - 1 in step q of stage st of a chunk; after those
  // of row block i, next(i) requests what comes next
  auto products = [&](auto st_, auto q_, int from, int to, auto next) {
    constexpr int ST = decltype(st_)::value, Q = decltype(q_)::value;
#pragma unroll
    for (int i = 0; i < C::FM; ++i) {
      if (i < from || i >= to) continue;
#pragma unroll
      for (int j = 0; j < C::FN; ++j) {
        if constexpr (C::A4) mfma_a4<2 * ST + Q>(acc[i][j], xr[i], wr[Q][j], sa[i], sb[j]);
        else mfma_a16(acc[i][j], xr[i], b[j]);
      }
      next(i);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  constexpr std::integral_constant<int, 0> c0{};
  constexpr std::integral_constant<int, 1> c1{};

  if constexpr (GROUPED) {
    for (int i = tid; i < C::BM; i += C::NT) lost[i] = source_row(a, min(t.r0 + i, t.r1 - 1)) < 0;
  }
  // stage 0 and its scale bytes first; stage 1 goes out between the first products
  issue(0, 0);
  if (nblk >= C::CB) load_scales(0);
  else load_short();
  write_scales(0);
  drain_barrier();
#pragma unroll
  for (int i = 0; i < C::FM; ++i) {
    load_x(0, 0, i);
    if constexpr (C::A4) load_sa(0, i);
  }
  if constexpr (C::A4) {
    load_w(0, 0);
    load_sb(0);
  } else {
    load_wc(0, 0, 0);
  }

  // One stage that is not the last, whole by that.  The hand-over to the next stage comes
  // among the second step's products: by then every wave has had time to receive its last
  // operands, so the buffer is free for the stage after next, whose loads go out between the
  // products, and the rest of the products covers the first reads of the next stage.  There
  // is no branch, which would let the compiler move the products past it: at the end the
  // last stage is requested again, into the buffer that is not read.  (s is 2 chunk + ST,
  // its buffer ST.)
  constexpr int HEAD = C::FM / 4;   // row blocks before the hand-over
  auto stage = [&](int s, auto st_) {
    constexpr int ST = decltype(st_)::value, buf = ST, nbuf = ST ^ 1;
    const int chunk = s >> 1;
    take(ST == 0);
    if constexpr (C::A4) load_w(buf, 1);
    convert(0);
    products(st_, c0, 0, C::FM, [&](int i) {
      load_x(buf, 1, i);
      if (ST == 0 && s == 0) issue_slice(1, 1, i, C::FM);
    });
    convert(1);
    products(st_, c1, 0, HEAD, [](int) {});
    if constexpr (ST == 1) write_scales((chunk + 1) & 1);
    drain_barrier();
    if constexpr (ST == 0) load_scales(min((chunk + 1) * 2, last) >> 1);
    const Source f = source(min(s + 2, last));
    if constexpr (C::A4) {
      load_w(nbuf, 0);
      if constexpr (ST == 1) load_sb(chunk + 1);
    } else {
      load_wc(nbuf, ST ^ 1, ST == 1 ? chunk + 1 : chunk);
    }
    auto next = [&](int i) {
      load_x(nbuf, 0, i);
      if constexpr (C::A4 && ST == 1) load_sa(chunk + 1, i);
    };
#pragma unroll
    for (int i = 0; i < HEAD; ++i) next(i);
    products(st_, c1, HEAD, C::FM, [&](int i) {
      next(i);
      constexpr int L = C::FM - HEAD;
#pragma unroll
      for (int j = (i - HEAD) * C::DMA / L; j < (i - HEAD + 1) * C::DMA / L; ++j) issue_one(f, buf, j);
    });
  };
  int s = 0;
  for (; s + 2 <= last; s += 2) {
    stage(s, c0);
    stage(s + 1, c1);
  }
  // the last chunk: one or two stages, the last perhaps part-filled: its blocks past K have
  // activations (A16) or both scale bytes (A4) zero, and an A4 step without any block is
  // left out
  auto rest = [&](auto st_, int valid) {
    constexpr int ST = decltype(st_)::value, buf = ST;
    if constexpr (ST == 1) {
      drain_barrier();
#pragma unroll
      for (int i = 0; i < C::FM; ++i) load_x(buf, 0, i);
      if constexpr (C::A4) load_w(buf, 0);
      else load_wc(buf, 1, s >> 1);
    }
    take(ST == 0);
    auto cut = [&]() {
      if constexpr (!C::A4) {
        if ((g >> 1) >= valid) {
#pragma unroll
          for (int i = 0; i < C::FM; ++i) xr[i] = u32x4{0, 0, 0, 0};
        }
      }
    };
    cut();
    convert(0);
    products(st_, c0, 0, C::FM, [](int) {});
    if (C::A4 && valid <= 4) return;
#pragma unroll
    for (int i = 0; i < C::FM; ++i) load_x(buf, 1, i);
    if constexpr (C::A4) load_w(buf, 1);
    cut();
    convert(1);
    products(st_, c1, 0, C::FM, [](int) {});
  };
  if (s == 0 && last == 1) issue(1, 1);
  rest(c0, nblk - s * C::SB);
  if (s < last) rest(c1, nblk - (s + 1) * C::SB);
  settle(acc);
  // no load may land in LDS that the next block owns by then
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");

  // ---- outputs: lane c of operand j holds column FN c + j of its wave's columns ----
  const int col = t.n0 + wn * 16 * C::FN + C::FN * l16;
#pragma unroll
  for (int i = 0; i < C::FM; ++i)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int rl = wm * 16 * C::FM + 16 * i + 4 * g + v;
      const int r = t.r0 + rl;
      if (r >= t.r1) continue;
      const int64_t at = (int64_t)r * a.N + col;
      float o[C::FN];
#pragma unroll
      for (int j = 0; j < C::FN; ++j) {
        o[j] = acc[i][j][v];
        if (GROUPED && lost[rl]) o[j] = __builtin_nanf("");
      }
      store_row<BF16, C::FN>(a, at, col, o);
    }
}

// the most row tiles that a launch can have; grouped: at most one part-filled one per expert
// with rows
template <class C, bool GROUPED>
int64_t row_tiles(const MxArgs& a) {
  return GROUPED ? std::min<int64_t>(a.M, a.M / C::BM + a.E) : (a.M + C::BM - 1) / C::BM;
}

template <class C, bool GROUPED>
hipError_t launch(const MxArgs& a, bool y_bf16, hipStream_t stream) {
  const int64_t tiles_n = (a.N + C::BN - 1) / C::BN;
  const dim3 grid((unsigned)(row_tiles<C, GROUPED>(a) * tiles_n)), block(C::NT);
  if constexpr (C::VEC) {
    if (y_bf16) hipLaunchKernelGGL((mxfp4_gemv_kernel<C, GROUPED, true>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((mxfp4_gemv_kernel<C, GROUPED, false>), grid, block, 0, stream, a);
    return hipGetLastError();
  } else if constexpr (C::SPLIT) {
    auto run = [&](auto kernel, std::atomic<uint64_t>& done) -> hipError_t {
      if (C::LDS > 64 * 1024) {
        // the kernel's limit of dynamic LDS, raised once per device (bit d of done)
        int dev = 0;
        hipError_t e = hipGetDevice(&dev);
        if (e != hipSuccess) return e;
        const uint64_t bit = uint64_t(1) << (dev & 63);
        if (!(done.load(std::memory_order_acquire) & bit)) {
          e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, C::LDS);
          if (e != hipSuccess) return e;
          done.fetch_or(bit, std::memory_order_acq_rel);
        }
      }
      hipLaunchKernelGGL(kernel, grid, block, C::LDS, stream, a);
      return hipGetLastError();
    };
    static std::atomic<uint64_t> done_bf16{0}, done_f32{0};
    return y_bf16 ? run(mxfp4_split_kernel<C, GROUPED, true>, done_bf16) : run(mxfp4_split_kernel<C, GROUPED, false>, done_f32);
  } else {
    if (y_bf16) hipLaunchKernelGGL((mxfp4_tile_kernel<C, GROUPED, true>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((mxfp4_tile_kernel<C, GROUPED, false>), grid, block, 0, stream, a);
    return hipGetLastError();
  }
}

// The form of a product: the one whose estimated time is the least,
//   fixed + r (round + stage * stages of a wave) + mb * (MB through LDS-DMA)     [us]
// with r = the tiles over those that the device holds at once, at least 1: a block takes its
// run of stages whether or not others run beside it, and every tile adds its traffic.
//   The four figures of a form are least-squares fits of the relative error to graph-replayed
// times of 660 products (drawn ones, M to 4100, N and K to 14400, to 100 experts; and M = 1 to
// 4096 on weights of 512 to 14336 rows and columns, 8 to 128 experts with 1 to 400 rows each),
// of 27 forms; the single-row forms' to 135 products of one row or a few experts' rows.  The forms
// kept lose 4% (A4), 5% (A16) and 3% (one row) of geometric-mean time against the best of all;
// a rule on tile counts alone lost 12 and 14% on the drawn ones, one row without the single-row
// forms 29%.  Outside their fit, over 220 dense products of 2 to 2000 rows for which the estimates
// choose a single-row form and 110 grouped ones of 2 to 500 rows, the choice loses 1.7 and 2.5%
// against the best form (1.38 and 1.41 times at worst), and 28 and 30% if they were kept for one
// row.  Both sides, graph-replayed, us:
//   M = 64 on [2048, 2048], A4: 16 x 16 over 4 waves 3.6, 32 x 64 5.3, tiles of 64 x 128 6.4
//   M = 128 on [11008, 2048], A4: tiles of 64 x 128 9.3, of 128 x 128 10.4, 32 x 64 11.6;
//     A16: 64 x 64 over 4 waves 15.0, 32 x 32 over 8 waves 18.0, tiles of 64 x 128 20.8
//   M = 1024 there, A4: tiles of 256 x 256 24.1, of 128 x 128 26.3 (what the estimates
//     choose); A16: 54.3 against 51.1
//   M = 16 on [4096, 14336]: 16 x 16 over 16 waves 8.1 (A4) and 13.3 (A16), over 4 10.6 and 18.7
//   4 rows for each of 128 experts of [4096, 2048], A4: 16 x 64 by one wave 121, 16 x 16 over
//     4 waves 191; dense it would be chosen above some 80000 columns alone, where tiles of 64 x 128
//     are faster (1 to 16 rows on [131072, 2048] 29 to 30 against 26 to 28, on [120000, 256] 14
//     against 11), so it is compiled for experts only
//   M = 1 on [131072, 2048], A16, wider than any product of the fit: 16 x 32 over 4 waves 43 (what
//     the estimates choose), a row by itself 32; on [65536, 2048] 19.7 and 18.8
struct MxCost {
  float fixed, round, stage, mb;
};

template <class C, bool GROUPED>
float estimate(const MxArgs& a, MxCost c, int cus) {
  const int64_t tiles_n = (a.N + C::BN - 1) / C::BN;
  if (row_tiles<C, GROUPED>(a) * tiles_n >= (int64_t(1) << 32) / C::NT) return INFINITY;   // threads of a launch
  // grouped: an expert's last tile with half its rows, the lists being on the device
  const float products = (float)std::min(a.M, a.E);
  const float tiles = (float)tiles_n * (GROUPED ? std::max(products, (float)a.M / C::BM + 0.5f * products * (C::BM > 1))
                                                : (float)row_tiles<C, GROUPED>(a));
  const int64_t stages = (a.K + C::KS - 1) / C::KS, mine = C::SPLIT ? (stages + C::NW - 1) / C::NW : stages;
  const float r = std::max(1.0f, tiles / (float)(cus * C::PER_CU));
  const float mb = 1e-6f * tiles * (float)(mine * (C::SPLIT ? C::NW : 1)) * (float)C::TILE_BYTES;
  return c.fixed + r * (c.round + c.stage * (float)mine) + c.mb * mb;
}

template <class C_, bool DENSE = true>   // MxVec, MxSplit or MxCfg; for products by expert alone without DENSE
struct MxForm {
  using C = C_;
  template <bool GROUPED>
  static constexpr bool HAS = DENSE || GROUPED;
  MxCost cost;
};

// f(the forms of a product)
template <bool A4, class F>
auto with_forms(F f) {
  if constexpr (A4)
    return f(MxForm<MxSplit<A4, 1, 1, 16, 2>>{2.97f, 2.02f, 0.363f, 0.023f},
             MxForm<MxSplit<A4, 1, 1, 4, 2>>{2.49f, 2.33f, 0.187f, 0.043f},
             MxForm<MxSplit<A4, 1, 4, 1, 2>, false>{0.63f, 4.79f, 0.617f, 0.045f},
             MxForm<MxSplit<A4, 2, 4, 4, 1>>{0.00f, 5.76f, 0.707f, 0.052f},
             MxForm<MxSplit<A4, 4, 2, 8, 1>>{2.66f, 3.16f, 1.033f, 0.036f},
             MxForm<MxCfg<A4, 2, 2, 2, 4>>{0.00f, 5.02f, 0.372f, 0.056f},
             MxForm<MxCfg<A4, 2, 2, 4, 4>>{0.00f, 5.88f, 0.541f, 0.049f},
             MxForm<MxCfg<A4, 2, 4, 8, 4>>{0.00f, 8.83f, 1.121f, 0.058f});
  else
    return f(MxForm<MxVec<4, 1>>{0.16f, 3.38f, 0.660f, 0.127f},
             MxForm<MxVec<2, 4>>{2.65f, 0.43f, 0.915f, 0.030f},
             MxForm<MxSplit<A4, 1, 1, 16, 2>>{2.83f, 2.05f, 0.429f, 0.022f},
             MxForm<MxSplit<A4, 1, 1, 4, 2>>{3.35f, 1.48f, 0.185f, 0.036f},
             MxForm<MxSplit<A4, 1, 2, 4, 2>>{2.92f, 1.95f, 0.233f, 0.045f},
             MxForm<MxSplit<A4, 1, 4, 1, 2>>{0.00f, 5.66f, 0.319f, 0.061f},
             MxForm<MxSplit<A4, 2, 2, 8, 1>>{3.10f, 1.74f, 0.276f, 0.062f},
             MxForm<MxSplit<A4, 4, 2, 8, 1>>{3.09f, 2.36f, 0.466f, 0.044f},
             MxForm<MxSplit<A4, 4, 4, 4, 1>>{2.29f, 3.89f, 0.546f, 0.046f},
             MxForm<MxCfg<A4, 1, 4, 4, 2>>{0.90f, 3.84f, 0.333f, 0.055f},
             MxForm<MxCfg<A4, 2, 2, 4, 4>>{0.61f, 5.20f, 0.491f, 0.039f},
             MxForm<MxCfg<A4, 2, 4, 8, 4>>{0.00f, 8.91f, 1.030f, 0.053f});
}

// the index of the form that the product takes on a device of `cus` compute units
template <bool A4, bool GROUPED>
int least(const MxArgs& a, int cus) {
  return with_forms<A4>([&](auto... form) {
    const float t[] = {decltype(form)::template HAS<GROUPED> ? estimate<typename decltype(form)::C, GROUPED>(a, form.cost, cus)
                                                              : INFINITY...};
    return (int)(std::min_element(std::begin(t), std::end(t)) - std::begin(t));
  });
}

template <class Form, bool GROUPED>
auto launch_of() -> hipError_t (*)(const MxArgs&, bool, hipStream_t) {
  if constexpr (Form::template HAS<GROUPED>) return launch<typename Form::C, GROUPED>;
  else return nullptr;
}

template <bool A4, bool GROUPED>
hipError_t launch_any(const MxArgs& a, bool y_bf16, hipStream_t stream) {
  return with_forms<A4>([&](auto... form) {
    using Fn = hipError_t (*)(const MxArgs&, bool, hipStream_t);
    const Fn fn[] = {launch_of<decltype(form), GROUPED>()...};
    return fn[least<A4, GROUPED>(a, device_cu_count())](a, y_bf16, stream);
  });
}

}  // namespace

int mxfp4_form(bool a4, bool grouped, int M, int K, int N, int E, int cus) {
  MxArgs a = {};
  a.M = M, a.N = N, a.K = K, a.E = E;
  return a4 ? grouped ? least<true, true>(a, cus) : least<true, false>(a, cus)
            : grouped ? least<false, true>(a, cus) : least<false, false>(a, cus);
}

int mxfp4_form_name(bool a4, bool grouped, int i, char* to, size_t n) {
  auto describe = [&](auto... form) {
    using Fn = int (*)(char*, size_t);
    const Fn fn[] = {decltype(form)::C::describe...};
    const bool has[] = {(grouped ? decltype(form)::template HAS<true> : decltype(form)::template HAS<false>)...};
    return i < 0 || i >= (int)std::size(fn) ? -1 : has[i] ? fn[i](to, n) : snprintf(to, n, "%s", "");
  };
  return a4 ? with_forms<true>(describe) : with_forms<false>(describe);
}

hipError_t launch_mxfp4_gemm(const void* X, const uint8_t* XS, int64_t xrow, int M, int K, const uint8_t* codes,
                             const uint8_t* scales, int N, void* Y, bool y_bf16, hipStream_t stream) {
  const MxArgs a = {static_cast<const uint8_t*>(X), XS, xrow, codes, scales, M, N, K, nullptr, nullptr, 1, M, Y};
  return XS ? launch_any<true, false>(a, y_bf16, stream) : launch_any<false, false>(a, y_bf16, stream);
}

hipError_t launch_mxfp4_grouped_gemm(const void* X, const uint8_t* XS, int64_t xrow, int T, int K,
                                     const uint8_t* codes, const uint8_t* scales, int E, int N, const int32_t* offsets,
                                     const int32_t* rows, int M, void* Y, bool y_bf16, hipStream_t stream) {
  const MxArgs a = {static_cast<const uint8_t*>(X), XS, xrow, codes, scales, M, N, K, offsets, rows, E, T, Y};
  return XS ? launch_any<true, true>(a, y_bf16, stream) : launch_any<false, true>(a, y_bf16, stream);
}

}  // namespace aq
