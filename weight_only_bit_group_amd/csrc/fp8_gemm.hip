// Products of FP8 activations and FP8 weights (gfx950), dense and grouped by expert:
//
//   Y[m, n] = sum_b sx[m, b] sw[n / 128, b] sum_{k in b} cx[m, k] cw[n, k]        b: blocks of 128 k
//
// with fp32 sums, stored as fp32 or rounded once to bf16.  Grouped: the rows offsets[e] .. offsets[e + 1] - 1 of Y
// belong to expert e and are multiplied with its weights; row r reads activation row rows[r] (or r without a list).
//
// A block's sum of 16 x 16 outputs starts from zero in the matrix cores and is added to the fp32 sums by a fused
// multiply-add with the factor sx sw, four of them a lane.  (The FP8 instructions' own block scales are powers of two
// for 32 k, which these scales are not.)  The weights are the instruction's rows and the activations its columns, so
// a lane's four results share one activation row and with it one factor.
//
// The output's type says how a block is added up.
//   bf16 out: one v_mfma_f32_16x16x128_f8f6f4 (32 cycles).  It adds groups of eight neighbouring products cut off at
// 2^-13 of the largest of the eight, and the groups in fp32: on normal values 1.5e-5 of the result (rms), a
// hundredth of the rounding to bf16 that follows.
//   fp32 out: the codes converted to bf16 (exact) and four v_mfma_f32_16x16x32_bf16, whose sums are fp32 throughout
// (1e-8 on the same values), at half the rate.
//
// A lane's operand is 32 bytes of a row, two units of 16; which two is free as long as both operands agree.  The
// rows of a tile are stored so that a lane's results of its FN operands are 4 FN neighbouring columns of one row.
//
// The lanes that a ragged edge leaves over read clamped addresses inside the same row or the last row; the
// activations of units past K are zero (the weights beside them are real codes of the row), rows past the end are
// not stored.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdio>
#include <iterator>
#include <type_traits>

#include "aq_kernels.h"
#include "fp8_device.h"
#include "gemm_tiles.h"

namespace aq {

namespace {

using namespace gemm;

typedef int i32x8 __attribute__((ext_vector_type(8)));

struct F8Args {
  const uint8_t* X;        // [T, K] codes
  const float* XS;         // [T, nkb]
  const uint8_t* W;        // [E, N, K]
  const float* WS;         // [E, nnb, nkb]
  int M, N, K;             // M: rows of Y
  int nkb, nnb;
  const int32_t* offsets;  // grouped: [E + 1]
  const int32_t* rows;     // grouped: [M] activation rows, or NULL
  int E, T;                // experts; rows of X
  void* Y;
};

// 4 bytes per lane from the lane's own address; lane l lands at lds + 4 l
__device__ __forceinline__ void dma4_at(const void* src, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %0, off" ::"v"(src), "s"(lds) : "memory");
}

__device__ __forceinline__ int swizzle(int r, int u) { return u ^ ((r >> 1) & 7); }

// a lane's 32 codes of one row and block, as the instructions take them
template <bool WIDE>
struct Operand {   // FP8
  i32x8 v;
  __device__ __forceinline__ Operand() = default;
  __device__ __forceinline__ Operand(u32x4 a, u32x4 b)
      : v{(int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)b[0], (int)b[1], (int)b[2], (int)b[3]} {}
};
template <>
struct Operand<true> {   // bf16
  bf16x8 v[4];
  __device__ __forceinline__ Operand() = default;
  __device__ __forceinline__ Operand(u32x4 a, u32x4 b) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t lo = q < 2 ? a[2 * q] : b[2 * q - 4], hi = q < 2 ? a[2 * q + 1] : b[2 * q - 3];
      const u32x4 w = {__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false)),
                       __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true)),
                       __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false)),
                       __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true))};
      v[q] = __builtin_bit_cast(bf16x8, w);
    }
  }
};

// 16 weight rows times 16 activation rows over one block of 128 k
__device__ __forceinline__ f32x4 block_sum(const Operand<false>& w, const Operand<false>& x) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w.v, x.v, f32x4{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ f32x4 block_sum(const Operand<true>& w, const Operand<true>& x) {
  f32x4 p = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int q = 0; q < 4; ++q) p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w.v[q], x.v[q], p, 0, 0, 0);
  return p;
}

// v[0 .. N - 1] as the neighbouring columns from `col` on of row r, 16 bytes a store where all of them are inside
template <bool BF16, int N>
__device__ __forceinline__ void store_columns(const F8Args& a, int r, int col, const float (&v)[N]) {
  const int64_t at = (int64_t)r * a.N + col;
  constexpr int S = BF16 ? 8 : 4;   // columns of a store
#pragma unroll
  for (int i = 0; i < N; i += S) {
    constexpr int C = N < S ? N : S;
    float o[C];
#pragma unroll
    for (int j = 0; j < C; ++j) o[j] = v[i + j];
    store_row<BF16, C>(a, at + i, col + i, o);
  }
}

// ---- tiles ----------------------------------------------------------------------------------
// WM x WN waves, each (16 FM) activation rows x (16 FN) weight rows.  K advances in stages of one block, 128 bytes of
// a row, through two LDS buffers filled by LDS-DMA.
template <int WM_, int WN_, int FM_, int FN_>
struct F8Cfg {
  static constexpr int WM = WM_, WN = WN_, FM = FM_, FN = FN_;
  static constexpr int NW = WM * WN, NT = 64 * NW;
  static constexpr int BM = 16 * FM * WM, BN = 16 * FN * WN;
  static constexpr int A_DMA = BM / 8 / NW;   // loads per wave and stage, 1 KiB each
  static constexpr int B_DMA = BN / 8 / NW;
  static constexpr int S_DMA = (BM + 63) / 64;   // loads of the activations' scales per stage, one a wave
  static_assert(BM % (8 * NW) == 0 && BN % (8 * NW) == 0 && S_DMA <= NW && 128 % (16 * FN) == 0, "whole loads per wave");
};

template <class C, bool GROUPED, bool BF16>
__global__ __launch_bounds__(C::NT, 1) void fp8_tile_kernel(F8Args a) {
  using Op = Operand<!BF16>;
  __shared__ __attribute__((aligned(1024))) uint8_t Xs[2][C::BM * 128];
  __shared__ __attribute__((aligned(1024))) uint8_t Ws[2][C::BN * 128];
  __shared__ __attribute__((aligned(256))) float Ss[2][C::S_DMA * 64];
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
  // LDS row i of the weights: row i's wave region, operand j = (i / 16) % FN, operand row i % 16 = 4 g + v
  auto wrow = [&](int i) {
    const int n = (i / (16 * C::FN)) * (16 * C::FN) + ((i & 15) >> 2) * (4 * C::FN) + 4 * ((i / 16) % C::FN) + (i & 3);
    return min(n, a.N - 1 - t.n0);
  };
  auto xrow = [&](int i) -> int64_t {
    const int r = min(t.r0 + i, t.r1 - 1);
    return GROUPED ? max(source_row(a, r), 0) : r;
  };
  const int last = a.nkb - 1;
  const uint8_t* wtile = a.W + ((int64_t)t.e * a.N + t.n0) * a.K;
  // load j of wave w covers 8 rows from 8 (j NW + w) on; the unit that a lane fetches is the same in all of them
  static_assert(C::NW % 2 == 0, "the permutation's period is 16 rows");
  const int unit = swizzle(8 * wid + (lane >> 3), lane & 7);
  uint32_t xsrc[C::A_DMA], wsrc[C::B_DMA];   // units from X (X is below 2^36 bytes), bytes from wtile (below 2^31)
#pragma unroll
  for (int j = 0; j < C::A_DMA; ++j)
    xsrc[j] = (uint32_t)((xrow(8 * (j * C::NW + wid) + (lane >> 3)) * a.K) >> 4) + unit;
#pragma unroll
  for (int j = 0; j < C::B_DMA; ++j) wsrc[j] = (uint32_t)wrow(8 * (j * C::NW + wid) + (lane >> 3)) * (uint32_t)a.K + 16u * unit;
  const float* ssrc = a.XS + xrow(min(64 * wid + lane, C::BM - 1)) * a.nkb;
  const int left = (a.K - last * 128) >> 4;   // units of the last block
  const uint32_t back = max(unit - left + 1, 0);
  auto issue = [&](int s, int buf) {
    const uint8_t* x = a.X + (int64_t)s * 128;
    const uint8_t* w = uniform(wtile + (int64_t)s * 128);
    const uint32_t b = s == last ? back : 0u;
#pragma unroll
    for (int j = 0; j < C::A_DMA; ++j)
      dma16_at(x + 16 * (uint64_t)(xsrc[j] - b), lds_addr(&Xs[buf][1024 * (C::NW * j + wid)]));
#pragma unroll
    for (int j = 0; j < C::B_DMA; ++j) dma16_from(w, wsrc[j] - 16 * b, lds_addr(&Ws[buf][1024 * (C::NW * j + wid)]));
    if (wid < C::S_DMA) dma4_at(ssrc + s, lds_addr(&Ss[buf][64 * wid]));
  };
  // (uniform over the wave: the constant address space makes it a scalar load)
  const auto* wscale = (const __attribute__((address_space(4))) float*)(uint64_t)uniform(reinterpret_cast<const uint8_t*>(
      a.WS + ((int64_t)t.e * a.nnb + ((t.n0 + wn * 16 * C::FN) >> 7)) * a.nkb));

  f32x4 acc[C::FM][C::FN];
#pragma unroll
  for (int i = 0; i < C::FM; ++i)
#pragma unroll
    for (int j = 0; j < C::FN; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  // units g and 4 + g of this lane's first operand rows; the rows of the next operand, 16 further, are permuted alike
  const int xat = 128 * (wm * 16 * C::FM + l16) + 16 * swizzle(l16, g), wat = 128 * (wn * 16 * C::FN + l16) + 16 * swizzle(l16, g);
  auto half = [](const uint8_t* p) { return *reinterpret_cast<const u32x4*>(p); };
  // One stage.  Row block i's operand is read while the products of the one before run, and a block's results are
  // added one row block later, when they have left the matrix core.  The last stage, which may be part-filled, is
  // compiled apart, so that the others have no branch; it requests nothing.
  auto stage = [&](int s, auto last_) {
    constexpr bool LAST = decltype(last_)::value;
    const int buf = s & 1;
    if constexpr (!LAST) issue(s + 1, buf ^ 1);
    const float sw = wscale[s];
    const uint8_t *wlo = &Ws[buf][wat], *whi = &Ws[buf][wat ^ 64], *xlo = &Xs[buf][xat], *xhi = &Xs[buf][xat ^ 64];
    const float* sx = &Ss[buf][wm * 16 * C::FM + l16];
    Op w[C::FN];
#pragma unroll
    for (int j = 0; j < C::FN; ++j) w[j] = Op(half(wlo + 2048 * j), half(whi + 2048 * j));
    u32x4 x[2][2];
    f32x4 p[2][C::FN];
    float f[2];
    auto load_x = [&](int i) {
      x[i & 1][0] = half(xlo + 2048 * i);
      x[i & 1][1] = half(xhi + 2048 * i);
      f[i & 1] = sx[16 * i] * sw;
      if constexpr (LAST) {
        if (g >= left) x[i & 1][0] = u32x4{0, 0, 0, 0};
        if (4 + g >= left) x[i & 1][1] = u32x4{0, 0, 0, 0};
      }
    };
    auto add = [&](int i, float by) {
#pragma unroll
      for (int j = 0; j < C::FN; ++j)
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[i][j][v] = __builtin_fmaf(p[i & 1][j][v], by, acc[i][j][v]);
    };
    load_x(0);
    float before = 0.0f;
#pragma unroll
    for (int i = 0; i < C::FM; ++i) {
      const float now = f[i & 1];
      const Op xi(x[i & 1][0], x[i & 1][1]);
      if (i + 1 < C::FM) load_x(i + 1);
#pragma unroll
      for (int j = 0; j < C::FN; ++j) p[i & 1][j] = block_sum(w[j], xi);
      if (i > 0) add(i - 1, before);
      before = now;
      __builtin_amdgcn_sched_barrier(0);
    }
    add(C::FM - 1, before);
  };
  issue(0, 0);
  drain_barrier();
  for (int s = 0; s < last; ++s) {
    stage(s, std::false_type{});
    drain_barrier();
  }
  stage(last, std::true_type{});

#pragma unroll
  for (int i = 0; i < C::FM; ++i) {
    const int r = t.r0 + wm * 16 * C::FM + 16 * i + l16;
    if (r >= t.r1) continue;
    const bool lost = GROUPED && source_row(a, r) < 0;
    float o[4 * C::FN];
#pragma unroll
    for (int j = 0; j < C::FN; ++j)
#pragma unroll
      for (int v = 0; v < 4; ++v) o[4 * j + v] = lost ? __builtin_nanf("") : acc[i][j][v];
    store_columns<BF16, 4 * C::FN>(a, r, t.n0 + wn * 16 * C::FN + 4 * C::FN * g, o);
  }
}

// the most row tiles that a launch can have; grouped: at most one part-filled one per expert with rows
template <class C, bool GROUPED>
int64_t row_tiles(const F8Args& a) {
  return GROUPED ? std::min<int64_t>(a.M, a.M / C::BM + a.E) : (a.M + C::BM - 1) / C::BM;
}

template <class C, bool GROUPED, bool BF16>
hipError_t launch(const F8Args& a, hipStream_t stream) {
  const int64_t tiles_n = (a.N + C::BN - 1) / C::BN;
  const dim3 grid((unsigned)(row_tiles<C, GROUPED>(a) * tiles_n)), block(C::NT);
  hipLaunchKernelGGL((fp8_tile_kernel<C, GROUPED, BF16>), grid, block, 0, stream, a);
  return hipGetLastError();
}

template <bool GROUPED, bool BF16>
hipError_t launch_any(const F8Args& a, hipStream_t stream) {
  using Large = F8Cfg<2, 4, BF16 ? 8 : 4, 4>;
  using Small = F8Cfg<2, 2, 2, 4>;
  const int64_t tiles = row_tiles<Large, GROUPED>(a) * ((a.N + Large::BN - 1) / Large::BN);
  return tiles >= device_cu_count() ? launch<Large, GROUPED, BF16>(a, stream) : launch<Small, GROUPED, BF16>(a, stream);
}

}  // namespace

hipError_t launch_fp8_gemm(const uint8_t* X, const float* XS, int T, int K, const uint8_t* codes, const float* scales, int E,
                           int N, const int32_t* offsets, const int32_t* rows, int M, void* Y, bool y_bf16,
                           hipStream_t stream) {
  const F8Args a = {X, XS, codes, scales, M, N, K, (K + 127) / 128, (N + 127) / 128, offsets, rows, E, T, Y};
  if (offsets) return y_bf16 ? launch_any<true, true>(a, stream) : launch_any<true, false>(a, stream);
  return y_bf16 ? launch_any<false, true>(a, stream) : launch_any<false, false>(a, stream);
}

}  // namespace aq
