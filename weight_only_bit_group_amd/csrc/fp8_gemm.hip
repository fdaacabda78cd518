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
  void* Y;                 // [M, N], or the codes [M, N / 2] of the gated activation
  float* YS;               // the codes' scales [M, nnb / 2]
  int64_t ldx;             // rows that are rounded on the way in: elements between them
  int64_t tiles;           // of a tile kernel, at most (set by the launch)
};

// the activations: FP8 codes, or fp32 or bf16 rows that are rounded on the way in
enum class In { CODES, F32, BF16 };

// what becomes of a tile's sums: fp32, rounded to bf16, or h = silu(g) u of the columns [g | u] in FP8
enum class Out { F32, BF16, GATED };

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

// ---- few rows -------------------------------------------------------------------------------
// Bound by the weight bytes.  A block's NW waves share K: each takes every NW-th stage (one block of 128 k) of the
// (16 FM) x (16 FN) tile through LDS buffers of its own, filled by its own LDS-DMA, so there is no barrier before the
// sums are joined, in wave order: a wave only waits for its own oldest loads, with R stages in flight.  (Straight to
// registers, in the order that the instructions take, neighbouring lanes read 16 bytes of different rows: four times
// the requests, 23 us against 16 for 16 rows on [4096, 14336].)
//   Activation rows past the tile's are not fetched: their LDS bytes are whatever was there, in columns of the result
// that are not stored.
//   Up to 16 short rows are rounded by every block for itself, while its first weights are under way: one token on
// [11008, 2048] takes 5.7 us, with a rounding kernel in front 7.2; 8 rows of 1024 on [4096, 1024] 5.0 and 5.8, on
// [11008, 1024] 5.7 and 6.7 (bf16 out: equal); 16 rows of 512 on [4096, 512] 5.3 and 5.2, the worst of the rule's sizes
// tried (graph-replayed, weights in the cache; called from the host 4.3 to 5.4 and 7.1 to 7.4, a launch less).
constexpr int kRounded = 8192;   // their values at most (32 KiB of fp32 a block)
template <int FM_, int FN_, int NW_, int R_>
struct F8Split {
  static constexpr int FM = FM_, FN = FN_, NW = NW_, R = R_;
  static constexpr int BM = 16 * FM, BN = 16 * FN, NT = 64 * NW;
  static constexpr bool SPLIT = true;
  static constexpr int DMA = 2 * FM + 2 * FN + 1;               // loads of a stage
  static constexpr int STAGE = 2048 * (FM + FN) + 256;          // its LDS bytes: activations, weights, scales
  static constexpr int PART = FM * FN * 1024;                   // bytes of a wave's sums
  static constexpr int LDS = NW * (R * STAGE > PART ? R * STAGE : PART);
  static constexpr int per_cu(bool) { return std::max(1, std::min(160 * 1024 / LDS, 32 / NW)); }   // blocks that a compute unit holds
  static int describe(char* to, size_t n) { return snprintf(to, n, "split %d x %d over %d", FM, FN, NW); }
  static_assert(FM <= 4 && 128 % BN == 0, "one load of scales, one weight scale a stage");
  static_assert((R - 1) * DMA < 64 && LDS <= 160 * 1024, "loads in flight are counted in six bits");
};

template <class C, In IN>
struct SplitStage {
  static constexpr bool ROUND = IN != In::CODES;
  static constexpr int X = ROUND ? 0 : 2048 * C::FM;
  static constexpr int BYTES = ROUND ? 2048 * C::FN : C::STAGE, DMA = ROUND ? 2 * C::FN : C::DMA;
  static constexpr int LDS = C::NW * std::max(C::R * BYTES, C::PART);
  static constexpr int SIZE = IN == In::F32 ? 4 : 2;   // of a value
  // behind the waves' buffers: codes, rows of `row` bytes (16 more than whole blocks: other banks); scales; values
  static constexpr int row(int nkb) { return 128 * nkb + 16; }
  static constexpr int lds(int M, int K, int nkb) { return LDS + (ROUND ? M * row(nkb) + (4 * M * nkb + 15) / 16 * 16 + SIZE * M * K : 0); }
};

template <class C, bool GROUPED, bool WIDE, Out OUT, In IN = In::CODES>
__global__ __launch_bounds__(C::NT) void fp8_split_kernel(F8Args a) {
  using Op = Operand<WIDE>;
  using S = SplitStage<C, IN>;
  static_assert(!S::ROUND || (!GROUPED && C::FM == 1), "rows that are rounded are one tile's");
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
  const int count = (a.nkb - wid + C::NW - 1) / C::NW;   // this wave's stages: wid, wid + NW, ..
  uint8_t* mine = lds + wid * C::R * S::BYTES;
  auto xrow = [&](int i) -> int64_t {
    const int r = min(t.r0 + i, t.r1 - 1);
    return GROUPED ? max(source_row(a, r), 0) : r;
  };
  // LDS row 16 j + 4 g' + v of the weights is row 4 FN g' + 4 j + v of the tile
  auto wrow = [&](int i) { return min(4 * C::FN * ((i & 15) >> 2) + 4 * (i >> 4) + (i & 3), a.N - 1 - t.n0); };
  // load j covers rows 8 j .. 8 j + 7; the permutation's period is 16 rows
  const int unit = swizzle(lane >> 3, lane & 7);
  const uint8_t* wtile = a.W + ((int64_t)t.e * a.N + t.n0) * a.K;
  uint32_t xsrc[2 * C::FM], wsrc[2 * C::FN];   // units from X (X is below 2^36 bytes), bytes from wtile
#pragma unroll
  for (int j = 0; j < 2 * C::FM; ++j)
    if (!S::ROUND) xsrc[j] = (uint32_t)((xrow(8 * j + (lane >> 3)) * a.K) >> 4) + (unit ^ (4 * (j & 1)));
#pragma unroll
  for (int j = 0; j < 2 * C::FN; ++j)
    wsrc[j] = (uint32_t)wrow(8 * j + (lane >> 3)) * (uint32_t)a.K + 16u * (unit ^ (4 * (j & 1)));
  const float* ssrc = a.XS + xrow(lane % C::BM) * a.nkb;
  const int last = a.nkb - 1, left = (a.K - last * 128) >> 4;   // units of the last block; those past it: its last one
  const int rows = t.r1 - t.r0;
  auto issue = [&](int i, int slot) {
    const int s = wid + i * C::NW;
    const uint8_t* x = a.X + (int64_t)s * 128;
    const uint8_t* w = uniform(wtile + (int64_t)s * 128);
    const uint32_t base = lds_addr(mine + slot * S::BYTES);
    const bool tail = s == last;
#pragma unroll
    for (int j = 0; j < (S::ROUND ? 0 : 2 * C::FM); ++j) {
      const int back = tail ? max((unit ^ (4 * (j & 1))) - left + 1, 0) : 0;
      // (eight lanes at least, so that the load is counted)
      if (lane < 8 || 8 * j + (lane >> 3) < rows)
        dma16_at(x + 16 * (uint64_t)(xsrc[j] - back), __builtin_amdgcn_readfirstlane(base + 1024 * j));
    }
#pragma unroll
    for (int j = 0; j < 2 * C::FN; ++j) {
      const int back = tail ? max((unit ^ (4 * (j & 1))) - left + 1, 0) : 0;
      dma16_from(w, wsrc[j] - 16 * back, __builtin_amdgcn_readfirstlane(base + S::X + 1024 * j));
    }
    if constexpr (!S::ROUND) dma4_at(ssrc + s, __builtin_amdgcn_readfirstlane(base + 2048 * (C::FM + C::FN)));
  };
  f32x4 acc[C::FM][C::FN];
#pragma unroll
  for (int i = 0; i < C::FM; ++i)
#pragma unroll
    for (int j = 0; j < C::FN; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  const float* wscale = a.WS + ((int64_t)t.e * a.nnb + (t.n0 >> 7)) * a.nkb;
  float scales = 0.0f;   // lane l: the weights' scale of the wave's stage i0 + l
  uint8_t* const codes = lds + S::LDS;
  float* const xscales = reinterpret_cast<float*>(codes + rows * S::row(a.nkb));
  if constexpr (S::ROUND) {
    uint8_t* const values = codes + rows * S::row(a.nkb) + (4 * rows * a.nkb + 15) / 16 * 16;
    const int units = a.K * S::SIZE / 16;   // of a row
    for (int i0 = 64 * wid; i0 < rows * units; i0 += C::NT) {
      const int i = i0 + lane, r = i / units;
      if (i < rows * units)
        dma16_at(a.X + (r * a.ldx * S::SIZE + 16 * (i - r * units)), __builtin_amdgcn_readfirstlane(lds_addr(values) + 16 * i0));
    }
  }
#pragma unroll
  for (int i = 0; i < C::R; ++i)
    if (i < count) issue(i, i);
  if constexpr (S::ROUND) {
    const uint8_t* const values = codes + rows * S::row(a.nkb) + (4 * rows * a.nkb + 15) / 16 * 16;
    // every wave's values have landed, the weights behind them need not
    if (count >= C::R) asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(C::R * S::DMA) : "memory");
    else asm volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");
    for (int item = threadIdx.x >> 4; item < rows * a.nkb; item += C::NT / 16) {
      const int r = item / a.nkb, kb = item - r * a.nkb, k = 128 * kb + 8 * l16;
      fp8::Eight<IN == In::BF16> in;
      in.clear();
      if (k < a.K) in.load(values, (int64_t)r * a.K + k);
      const float s = fp8::scale_of(fp8::row_umax(in.amax()));
      float v[8];
      in.values(v);
      uint32_t w[2];
      fp8::codes_of<2>(v, s, w);
      *reinterpret_cast<uint64_t*>(codes + r * S::row(a.nkb) + k) = w[0] | ((uint64_t)w[1] << 32);
      if (l16 == 0) xscales[item] = s;
    }
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  }
  for (int i0 = 0; i0 < count; i0 += 64) {
    scales = wscale[min(wid + (i0 + lane) * C::NW, last)];
    const int stop = min(i0 + 64, count);
    for (int n = i0; n < stop; ++n) {
      const int s = wid + n * C::NW, slot = n % C::R;
      if (n + C::R < count) asm volatile("s_waitcnt vmcnt(%0)" ::"n"((C::R - 1) * S::DMA) : "memory");
      else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      const uint8_t* xt = mine + slot * S::BYTES;
      const uint8_t* wt = xt + S::X;
      const float* st = reinterpret_cast<const float*>(xt + 2048 * (C::FM + C::FN));
      auto half = [](const uint8_t* tile, int r, int u) {
        return *reinterpret_cast<const u32x4*>(tile + 128 * r + 16 * swizzle(r, u));
      };
      u32x4 x[C::FM][2], w[C::FN][2];
      float f[C::FM];
#pragma unroll
      for (int i = 0; i < C::FM; ++i) {
        if constexpr (S::ROUND) {
          const int r = min(l16, rows - 1);
          const uint8_t* at = codes + r * S::row(a.nkb) + 128 * s + 16 * g;
          x[i][0] = *reinterpret_cast<const u32x4*>(at);
          x[i][1] = *reinterpret_cast<const u32x4*>(at + 64);
          f[i] = xscales[r * a.nkb + s];
        } else {
          x[i][0] = half(xt, 16 * i + l16, g);
          x[i][1] = half(xt, 16 * i + l16, 4 + g);
          f[i] = st[16 * i + l16];
        }
      }
#pragma unroll
      for (int j = 0; j < C::FN; ++j) {
        w[j][0] = half(wt, 16 * j + l16, g);
        w[j][1] = half(wt, 16 * j + l16, 4 + g);
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      if (n + C::R < count) issue(n + C::R, slot);
      // units past K are zero; by a mask: the compiler loses the wait between a matrix instruction and its result's
      // reader where a branch comes between them
      const uint32_t keep0 = s == last && g >= left ? 0u : ~0u, keep1 = s == last && 4 + g >= left ? 0u : ~0u;
      const float sw = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(scales), n - i0));
      Op wo[C::FN];
#pragma unroll
      for (int j = 0; j < C::FN; ++j) wo[j] = Op(w[j][0], w[j][1]);
#pragma unroll
      for (int i = 0; i < C::FM; ++i) {
        const Op xo(x[i][0] & keep0, x[i][1] & keep1);
        const float by = f[i] * sw;
#pragma unroll
        for (int j = 0; j < C::FN; ++j) {
          const f32x4 p = block_sum(wo[j], xo);
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[i][j][v] = __builtin_fmaf(p[v], by, acc[i][j][v]);
        }
      }
    }
  }

  auto store = [&](int i, const f32x4 (&v)[C::FN]) {
    const int r = t.r0 + 16 * i + l16;
    if (r >= t.r1) return;
    const bool lost = GROUPED && source_row(a, r) < 0;
    float o[4 * C::FN];
#pragma unroll
    for (int j = 0; j < C::FN; ++j)
#pragma unroll
      for (int c = 0; c < 4; ++c) o[4 * j + c] = lost ? __builtin_nanf("") : v[j][c];
    store_columns<OUT == Out::BF16, 4 * C::FN>(a, r, t.n0 + 4 * C::FN * g, o);
  };
  if constexpr (C::NW == 1) {
#pragma unroll
    for (int i = 0; i < C::FM; ++i) store(i, acc[i]);
  } else {
    f32x4* sums = reinterpret_cast<f32x4*>(lds);
    __syncthreads();   // (every wave has read its last stage)
#pragma unroll
    for (int i = 0; i < C::FM; ++i)
#pragma unroll
      for (int j = 0; j < C::FN; ++j) sums[((wid * C::FM + i) * C::FN + j) * 64 + lane] = acc[i][j];
    __syncthreads();
    for (int i = wid; i < C::FM; i += C::NW) {
      f32x4 v[C::FN];
#pragma unroll
      for (int j = 0; j < C::FN; ++j) v[j] = sums[(i * C::FN + j) * 64 + lane];
#pragma unroll
      for (int k = 1; k < C::NW; ++k)
#pragma unroll
        for (int j = 0; j < C::FN; ++j) v[j] += sums[((k * C::FM + i) * C::FN + j) * 64 + lane];
      store(i, v);
    }
  }
}

// ---- tiles ----------------------------------------------------------------------------------
// WM x WN waves, each (16 FM) activation rows x (16 FN) weight rows.  K advances in stages of one block, 128 bytes of
// a row, through two LDS buffers filled by LDS-DMA.
//   M = 4096 on [11008, 2048], bf16 out: 94 to 102 us, 1.8 to 2.0 PFLOP/s (a library product of FP8 with one scale a
// tensor 101); K = 14336 on 4096 columns 196 to 205 us, 2.4 (171).  The matrix cores work 48% of the loop's cycles: a
// stage of a 256 x 256 tile has 2048 cycles of matrix instructions on a SIMD and takes 4290, a third of them waiting for
// the hand-over; four fused multiply-adds follow every instruction, and 64 KB of a stage come from the L2 and LDS alike.
// fp32 out: 196 us (0.94 PFLOP/s) and 421, the codes' conversion (16 instructions an operand) beside four matrix
// instructions a product.
template <int WM_, int WN_, int FM_, int FN_>
struct F8Cfg {
  static constexpr int WM = WM_, WN = WN_, FM = FM_, FN = FN_;
  static constexpr int NW = WM * WN, NT = 64 * NW;
  static constexpr int BM = 16 * FM * WM, BN = 16 * FN * WN;
  static constexpr int A_DMA = BM / 8 / NW;   // loads per wave and stage, 1 KiB each
  static constexpr int B_DMA = BN / 8 / NW;
  static constexpr bool SPLIT = false;
  // rows whose scales a wave loads per stage, by one load of a dword a lane (fewer than 16 a wave: some are loaded twice)
  static constexpr int S_ROWS = std::max(16, BM / NW);
  static constexpr int SOURCES = A_DMA + 1 + B_DMA;   // a thread's
  static constexpr int changed(bool gated) { return gated ? A_DMA + 1 : SOURCES; }   // from tile to tile
  static constexpr int lds(bool gated) { return 2 * 128 * (BM + BN) + 512 * NW + (gated ? 4 * BM * WN : 0); }
  // blocks that a compute unit holds; their registers leave room for 8 waves, or 12
  static constexpr int per_cu(bool gated) { return std::max(1, std::min(160 * 1024 / (lds(gated) + 1024), (FM * FN >= 16 ? 8 : 12) / NW)); }
  // Whether a block takes one tile after the other: where a compute unit holds one block, whose first loads and last
  // stores nothing would cover.  It gains little: calls of linear_prefill's sizes (4096 rows on [11008, 2048]) take 112 us
  // alone and 115 one behind the other, with a block a tile 115 and 113; 32768 rows over 64 experts of [2048, 2048] 224
  // and 226; and the experts' layer of 2048 tokens loses by it, 435 and 418 (three sets of inputs, both in turn).
  static constexpr bool chain(bool gated) { return per_cu(gated) == 1; }
  static int describe(char* to, size_t n) { return snprintf(to, n, "tile %d x %d of %d x %d", WM, WN, FM, FN); }
  static_assert(BM % (8 * NW) == 0 && BN % (8 * NW) == 0 && 128 % (16 * FN) == 0, "whole loads per wave");
  static_assert(S_ROWS % 16 == 0 && S_ROWS <= 64, "the scales of 16 rows lie together");
};

__device__ const u32x4 kZeros = {0, 0, 0, 0};   // in place of activations past K

template <class C, bool GROUPED, bool WIDE, Out OUT>
__global__ __launch_bounds__(C::NT, C::per_cu(OUT == Out::GATED) * C::NW / 4) void fp8_tile_kernel(F8Args a) {
  using Op = Operand<WIDE>;
  constexpr bool GATED = OUT == Out::GATED;
  static_assert(!GATED || (GROUPED && C::BN == 256 && C::FN == 4), "a block of 128 columns of h, 8 of them a lane");
  constexpr int COLS = GATED ? 128 : C::BN;   // columns of the output that a tile has
  __shared__ __attribute__((aligned(1024))) uint8_t Xs[2][C::BM * 128];
  __shared__ __attribute__((aligned(1024))) uint8_t Ws[2][C::BN * 128];
  __shared__ __attribute__((aligned(256))) float Ss[2][C::NW * 64];
  constexpr bool CHAIN = C::chain(GATED);
  constexpr int CHANGED = CHAIN ? C::changed(GATED) : 1;
  __shared__ uint32_t sources[CHANGED][C::NT];   // of the next tile, each thread's own
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wid = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wid / C::WN, wn = wid % C::WN;
  const int l16 = lane & 15, g = lane >> 4;
  const int inner = a.N / 2;                  // gated: columns of g and of u
  const int tiles_n = GATED ? inner / 128 : (a.N + C::BN - 1) / C::BN;
  int ntiles = (int)a.tiles;
  auto find = [&](int i, Tile& t) -> bool {
    if constexpr (GROUPED) {
      const bool found = grouped_tile<C::BM>(a, tiles_n, COLS, i, t, a.tiles, ntiles);
      return __builtin_amdgcn_readfirstlane(found);   // (the same in every lane, which the compiler does not see)
    } else {
      // groups of four row tiles walked column by column: the 32 tiles that an XCD runs together are four rows of
      // eight (an eighth of the row tiles, two rows of 16, costs 3% at 4096 rows)
      const int tiles_m = (a.M + C::BM - 1) / C::BM;
      i = tile_of_block(i, ntiles);
      const int gmax = min(tiles_m, 4);
      const int grp = i / (gmax * tiles_n);
      const int gm = min(tiles_m - grp * gmax, gmax);
      const int within = i - grp * gmax * tiles_n;
      t.e = 0;
      t.r0 = __builtin_amdgcn_readfirstlane((grp * gmax + within % gm) * C::BM);
      t.r1 = min(t.r0 + C::BM, a.M);
      t.n0 = __builtin_amdgcn_readfirstlane((within / gm) * C::BN);
      return true;
    }
  };
  // Tiles blockIdx, blockIdx + blocks, ..  The stages of a block's tiles follow one another without a pause: while a
  // tile's last stages are computed the first of the next one is under way, its second while the results are stored.
  int i = blockIdx.x;
  Tile t, next;
  while (!find(i, t)) {   // (a tile below ntiles is only missing where offsets overlap)
    i += gridDim.x;
    if (!CHAIN || i >= ntiles) return;   // the whole block
  }

  const int real = a.nkb - 1, last = max(real, 1);   // (a single stage is followed by one of zeros)
  const int left = (a.K - real * 128) >> 4;          // units of the last block; activations past them are zero
  // load j of wave w covers 8 rows from 8 (j NW + w) on; the unit that a lane fetches is the same in all of them
  static_assert(C::NW % 2 == 0, "the permutation's period is 16 rows");
  const int unit = swizzle(8 * wid + (lane >> 3), lane & 7);
  const uint32_t back = max(unit - left + 1, 0);
  typedef const __attribute__((address_space(4))) float* Uniform;
  // A_DMA units from X (X is below 2^36 bytes), a row of XS, B_DMA bytes from wtile (below 2^32; gated: of every tile)
  uint32_t src[C::SOURCES];
  const uint8_t* wtile;
  // (what the store of a row works out is kept out of the registers until then)
  auto anew = [](int v) {
    asm volatile("" : "+v"(v));
    return v;
  };
  // a tile's sources, given to f(index, source)
  auto sources_of = [&](const Tile& t, auto f) {
    // LDS row i of the weights: row i's wave region, operand j = (i / 16) % FN, operand row i % 16 = 4 g + v.  Gated: a
    // wave's first FN / 2 operands are rows of G, the others the same rows of U, so a lane has both of 2 FN columns of h.
    auto wrow = [&](int i) {
      const int j = (i / 16) % C::FN;
      if constexpr (GATED)
        return (i / (16 * C::FN)) * (8 * C::FN) + ((i & 15) >> 2) * (2 * C::FN) + 4 * (j % (C::FN / 2)) + (i & 3) +
               (j < C::FN / 2 ? 0 : inner);
      return min((i / (16 * C::FN)) * (16 * C::FN) + ((i & 15) >> 2) * (4 * C::FN) + 4 * j + (i & 3), a.N - 1 - t.n0);
    };
    auto xrow = [&](int i) -> int64_t {
      const int r = min(t.r0 + i, t.r1 - 1);
      return GROUPED ? max(source_row(a, r), 0) : r;
    };
    const int lane = anew(tid) & 63, unit = swizzle(8 * wid + (lane >> 3), lane & 7);
#pragma unroll
    for (int j = 0; j < C::A_DMA; ++j)
      f(j, (uint32_t)((xrow(8 * (j * C::NW + wid) + (lane >> 3)) * a.K) >> 4) + unit);
    f(C::A_DMA, (uint32_t)xrow((C::S_ROWS * wid + lane % C::S_ROWS) % C::BM));
#pragma unroll
    for (int j = 0; j < C::B_DMA; ++j)
      f(C::A_DMA + 1 + j, (uint32_t)wrow(8 * (j * C::NW + wid) + (lane >> 3)) * (uint32_t)a.K + 16u * unit);
  };
  auto weights_of = [&](const Tile& t) { return a.W + ((int64_t)t.e * a.N + t.n0) * a.K; };
  auto scales_of = [&](const Tile& t) {
    // (uniform over the wave: the constant address space makes it a scalar load; a wave whose columns are all past N
    // reads the last block's)
    return (Uniform)(uint64_t)uniform(reinterpret_cast<const uint8_t*>(
        a.WS + ((int64_t)t.e * a.nnb + (GATED ? t.n0 >> 7 : min((t.n0 + wn * 16 * C::FN) >> 7, a.nnb - 1))) * a.nkb));
  };
  const int64_t uscale = GATED ? (int64_t)(a.nnb / 2) * a.nkb : 0;   // gated: the scales of U behind those of G
  auto issue = [&](int s, int buf) {
    const uint32_t b = s >= real ? back : 0u;
    const bool zero = unit >= (s < real ? 8 : s == real ? left : 0);
    const uint8_t* none = reinterpret_cast<const uint8_t*>(&kZeros);
    const uint8_t* x = a.X + (int64_t)s * 128;
    const uint8_t* w = uniform(wtile + (int64_t)min(s, real) * 128);
#pragma unroll
    for (int j = 0; j < C::A_DMA; ++j)
      dma16_at(zero ? none : x + 16 * (uint64_t)src[j], lds_addr(&Xs[buf][1024 * (C::NW * j + wid)]));
#pragma unroll
    for (int j = 0; j < C::B_DMA; ++j) dma16_from(w, src[C::A_DMA + 1 + j] - 16 * b, lds_addr(&Ws[buf][1024 * (C::NW * j + wid)]));
    dma4_at(s > real ? reinterpret_cast<const float*>(none) : a.XS + ((int64_t)src[C::A_DMA] * a.nkb + s),
            lds_addr(&Ss[buf][64 * wid]));
  };

  f32x4 acc[C::FM][C::FN];
  // units g and 4 + g of this lane's first operand rows; the rows of the next operand, 16 further, are permuted alike
  const int xat = 128 * (wm * 16 * C::FM + l16) + 16 * swizzle(l16, g), wat = 128 * (wn * 16 * C::FN + l16) + 16 * swizzle(l16, g);
  // Operands are read ahead: row block i + 1's activations while the products of row block i run, the next stage's
  // weights into the registers that the last row block's products have just used.  Before those comes the hand-over:
  // by then every wave has its last operands of the stage, so its buffer is free for the stage after next.  A result
  // is added when its registers are needed again, FN products later, when it has left the matrix core; the order of
  // additions and products is fixed, or the compiler gathers the products and waits for their results.
  static_assert(C::FM % 2 == 0, "row blocks alternate between two sets of registers");
  u32x4 wr[C::FN][2], xr[2][2];
  f32x4 p[C::FN];
  float fr[2], sw, swnext, uw = 0.0f, uwnext = 0.0f, before = 0.0f, ubefore = 0.0f;
  auto load_w = [&](const uint8_t* tile, int j) {
    wr[j][0] = *reinterpret_cast<const u32x4*>(tile + wat + 2048 * j);
    wr[j][1] = *reinterpret_cast<const u32x4*>(tile + (wat ^ 64) + 2048 * j);
  };
  auto load_x = [&](int buf, int i) {
    xr[i & 1][0] = *reinterpret_cast<const u32x4*>(&Xs[buf][xat + 2048 * i]);
    xr[i & 1][1] = *reinterpret_cast<const u32x4*>(&Xs[buf][(xat ^ 64) + 2048 * i]);
    // (row r's is the r % S_ROWS-th of wave r / S_ROWS)
    const int r = wm * 16 * C::FM + 16 * i;
    fr[i & 1] = Ss[buf][64 * (r / C::S_ROWS) + r % C::S_ROWS + l16];
  };
  auto add = [&](int i, int j) {
#pragma unroll
    for (int v = 0; v < 4; ++v)
      acc[i][j][v] = __builtin_fmaf(p[j][v], GATED && j >= C::FN / 2 ? ubefore : before, acc[i][j][v]);
  };
  // the stage in buffer buf; the factor of the one behind it is at `at`, that of U ustep behind it
  auto stage = [&](int buf, Uniform at, int64_t ustep) {
    Op w[C::FN];
#pragma unroll
    for (int j = 0; j < C::FN; ++j) w[j] = Op(wr[j][0], wr[j][1]);
    const float by = sw, uby = uw;
#pragma unroll
    for (int i = 0; i < C::FM; ++i) {
      const bool hand = i + 1 == C::FM;
      if (hand) {
        drain_barrier();
        swnext = at[0];
        if (GATED) uwnext = at[ustep];
      }
      const Op x(xr[i & 1][0], xr[i & 1][1]);
      const float f = fr[i & 1] * by, uf = fr[i & 1] * uby;
      if (hand) load_x(buf ^ 1, 0);
      else load_x(buf, i + 1);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < C::FN; ++j) {
        add((i + C::FM - 1) % C::FM, j);
        p[j] = block_sum(w[j], x);
        if (hand) load_w(&Ws[buf ^ 1][0], j);
        __builtin_amdgcn_sched_barrier(0);
      }
      before = f;
      ubefore = uf;
      __builtin_amdgcn_sched_barrier(0);
    }
    sw = swnext;
    uw = uwnext;
    // (branches follow: the compiler loses the wait between a matrix instruction and its result's reader across one)
    asm volatile("s_nop 7\n\ts_nop 3");
    __builtin_amdgcn_sched_barrier(0);
  };
  auto begin = [&]() {   // nothing summed, nothing pending
#pragma unroll
    for (int j = 0; j < C::FN; ++j) {
      p[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < C::FM; ++i) acc[i][j] = p[j];
    }
    before = ubefore = 0.0f;
  };

  sources_of(t, [&](int k, uint32_t v) { src[k] = v; });
  wtile = weights_of(t);
  Uniform wscale = scales_of(t);
  issue(0, 0);
  drain_barrier();
  issue(1, 1);
#pragma unroll
  for (int j = 0; j < C::FN; ++j) load_w(&Ws[0][0], j);
  load_x(0, 0);
  sw = wscale[0];
  if (GATED) uw = wscale[uscale];
  int buf = 0;
  for (;;) {
    // the next tile, while there is room: the sums' registers are free
    bool more = false;
    if constexpr (CHAIN)
      while (!more && (i += gridDim.x) < ntiles) more = find(i, next);
    if (more)
      sources_of(next, [&](int k, uint32_t v) {
        if (CHAIN && k < CHANGED) sources[k][tid] = v;
      });
    begin();
    // All stages but two; those two, beside whose products the next tile's first stages are requested; without a next
    // tile they are alone.  The sources change between the loops: a branch within one costs it its registers.
    Uniform nscale = wscale;
    auto behind = [&](int s) {   // the factors of the stage behind stage s; none behind a single one
      return s >= last ? nscale : s >= real ? (Uniform)(uint64_t)&kZeros : wscale + s + 1;
    };
    auto step = [&](int s) { return s < last && s >= real ? 0 : uscale; };
    int s = 0;
    for (int stop = last - 1, ahead = 2;;) {
#pragma clang loop unroll(disable)
      for (; s < stop; ++s) {
        stage(buf, behind(s), step(s));
        issue(s + ahead, buf);
        buf ^= 1;
      }
      if (!CHAIN || !more || s > last) break;
      if constexpr (CHAIN) {
#pragma unroll
        for (int k = 0; k < CHANGED; ++k) src[k] = sources[k][tid];
        wtile = weights_of(next);
        nscale = scales_of(next);
        stop = last + 1, ahead = 1 - last;
      }
    }
#pragma clang loop unroll(disable)
    for (; s <= last; ++s) {
      stage(buf, behind(s), step(s));
      buf ^= 1;
    }
    wscale = nscale;
#pragma unroll
    for (int j = 0; j < C::FN; ++j) add(C::FM - 1, j);
    if constexpr (GATED) {
      // a block of h: 8 columns a lane, 32 a wave, its largest magnitude over the WN waves of the row through LDS
      __shared__ uint32_t top[C::BM * C::WN];
#pragma unroll
      for (int i = 0; i < C::FM; ++i) {
        const int lane = anew(tid) & 63, l16 = lane & 15, g = lane >> 4;
        const int r = t.r0 + wm * 16 * C::FM + 16 * i + l16;
        const bool lost = r < t.r1 && source_row(a, r) < 0;
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < C::FN / 2; ++j)
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const float h = lost ? __builtin_nanf("") : fp8::gated(acc[i][j][v], acc[i][j + C::FN / 2][v]);
            acc[i][j][v] = h;
            m = max(m, fp8::abs_bits(h));
          }
        m = max(m, (uint32_t)__shfl_xor((int)m, 16, 64));
        m = max(m, (uint32_t)__shfl_xor((int)m, 32, 64));
        if (g == 0) top[(wm * 16 * C::FM + 16 * i + l16) * C::WN + wn] = m;
      }
      asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");   // (loads of the next tile stay under way)
#pragma unroll
      for (int i = 0; i < C::FM; ++i) {
        const int lane = anew(tid) & 63, l16 = lane & 15, g = lane >> 4;
        const int at = wm * 16 * C::FM + 16 * i + l16, r = t.r0 + at;
        if (r >= t.r1) continue;
        uint32_t m = 0;
#pragma unroll
        for (int w = 0; w < C::WN; ++w) m = max(m, top[at * C::WN + w]);
        const float scale = fp8::scale_of(m);
        float h[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) h[c] = acc[i][c / 4][c % 4];
        uint32_t w[2];
        fp8::codes_of<2>(h, scale, w);
        *reinterpret_cast<uint64_t*>(static_cast<uint8_t*>(a.Y) + (int64_t)r * inner + t.n0 + 8 * C::FN * wn + 8 * g) =
            w[0] | ((uint64_t)w[1] << 32);
        if (wn == 0 && g == 0) a.YS[(int64_t)r * (a.nnb / 2) + (t.n0 >> 7)] = scale;
      }
    } else {
#pragma unroll
      for (int i = 0; i < C::FM; ++i) {
        const int lane = anew(tid) & 63, l16 = lane & 15, g = lane >> 4;
        const int r = t.r0 + wm * 16 * C::FM + 16 * i + l16;
        if (r >= t.r1) continue;
        const bool lost = GROUPED && source_row(a, r) < 0;
        float o[4 * C::FN];
#pragma unroll
        for (int j = 0; j < C::FN; ++j)
#pragma unroll
          for (int v = 0; v < 4; ++v) o[4 * j + v] = lost ? __builtin_nanf("") : acc[i][j][v];
        store_columns<OUT == Out::BF16, 4 * C::FN>(a, r, t.n0 + wn * 16 * C::FN + 4 * C::FN * g, o);
      }
    }
    if (!more) break;
    t = next;
  }
  // no load may land in LDS that the next block owns by then
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

// the most row tiles that a launch can have; grouped: at most one part-filled one per expert with rows
template <class C, bool GROUPED>
int64_t row_tiles(const F8Args& a) {
  return GROUPED ? std::min<int64_t>(a.M, a.M / C::BM + a.E) : (a.M + C::BM - 1) / C::BM;
}

template <class C, bool GROUPED, bool WIDE, Out OUT, In IN = In::CODES>
hipError_t launch(const F8Args& a, hipStream_t stream) {
  const int64_t tiles = row_tiles<C, GROUPED>(a) * ((a.N + C::BN - 1) / C::BN);   // (gated: BN / 2 columns of each half of N)
  const dim3 block(C::NT);
  if constexpr (C::SPLIT) {
    const auto kernel = fp8_split_kernel<C, GROUPED, WIDE, OUT, IN>;
    using S = SplitStage<C, IN>;
    const int lds = S::lds(a.M, a.K, a.nkb);
    constexpr int most = S::LDS + (S::ROUND ? kRounded * (1 + S::SIZE) + 16 * (128 + 16 + 8) : 0);
    static_assert(most <= 160 * 1024, "of a compute unit");
    if (most > 64 * 1024) {
      // the kernel's limit of dynamic LDS, raised once per device (bit d of done)
      static std::atomic<uint64_t> done{0};
      int dev = 0;
      hipError_t e = hipGetDevice(&dev);
      if (e != hipSuccess) return e;
      const uint64_t bit = uint64_t(1) << (dev & 63);
      if (!(done.load(std::memory_order_acquire) & bit)) {
        e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, most);
        if (e != hipSuccess) return e;
        done.fetch_or(bit, std::memory_order_acq_rel);
      }
    }
    hipLaunchKernelGGL(kernel, dim3((unsigned)tiles), block, lds, stream, a);
  } else {
    F8Args b = a;
    b.tiles = tiles;
    const dim3 grid((unsigned)(C::chain(OUT == Out::GATED) ? std::min<int64_t>(tiles, device_cu_count()) : tiles));
    hipLaunchKernelGGL((fp8_tile_kernel<C, GROUPED, WIDE, OUT>), grid, block, 0, stream, b);
  }
  return hipGetLastError();
}

// The form of a product: the one whose estimated time is the least,
//   fixed + r (round + stage * stages of a wave) + mb * (MB through LDS-DMA)     [us]
// with r = the tiles over those that the device holds at once, at least 1: a block takes its run of stages whether or
// not others run beside it, and every tile adds its traffic.  The four figures of a form are fitted to graph-replayed
// times of 469 products (1 to 16384 rows on weights of 512 to 14336 rows and columns, drawn ones of 64 to 14336, up to
// 128 experts with 1 to 32768 rows): least squares of the relative error, then the choice's loss against the best form
// in the geometric mean, which is 1.1% (bf16 out) and 1.3% (fp32 out) and at worst 1.27 times.  Forms without which that
// mean would be 0.6% higher at most were left out.  Both sides, us of the product alone, graph-replayed on the same
// operands (what the 256 MB cache holds comes from there):
//   M = 1 on [11008, 2048], fp32 out: 16 x 64 over 8 waves 5.0, 16 x 16 over 4 waves 6.6, tiles of 32 x 128 12.2
//   M = 16 on [4096, 14336], fp32 out: 16 x 16 over 16 waves 11.9, 16 x 32 over 8 waves 13.8, 16 x 64 over 8 waves 18.1
//   M = 32 there, bf16 out: 16 x 32 over 8 waves 13.4, 32 x 32 over 8 waves 16.3, 16 x 16 over 16 waves 18.0
//   M = 333 on [1003, 2064], fp32 out: 32 x 32 over 8 waves 7.0, 32 x 64 over 4 waves 7.7, 16 x 64 over 8 waves 9.3
//   M = 128 on [11008, 2048], bf16 out: 32 x 64 over 4 waves 10.1, tiles of 32 x 128 11.5, of 128 x 128 14.5
//   M = 4096 there: tiles of 256 x 256 94, of 128 x 128 114, of 32 x 128 210; fp32 out: 128 x 128 196, 32 x 128 266
//   (256 x 256, not compiled for them, was slower than 128 x 128)
//   64 x 8 rows of 128 experts [2048, 1024], bf16 out: tiles of 32 x 128 43.3, 32 x 64 over 4 waves 48.4, tiles of 128 x
//   128 49.6
//   4096 x 8 rows of 64 experts [2048, 2048]: tiles of 256 x 256 211, of 128 x 128 238; fp32 out: 128 x 128 352, 32 x
//   128 482
struct F8Cost {
  float fixed, round, stage, mb;
};

template <class C, bool GROUPED, Out OUT>
float estimate(const F8Args& a, F8Cost c, int cus) {
  const int64_t tiles_n = (a.N + C::BN - 1) / C::BN;
  if (row_tiles<C, GROUPED>(a) * tiles_n >= (int64_t(1) << 32) / C::NT) return INFINITY;   // threads of a launch
  // grouped: an expert's last tile with half its rows, the lists being on the device
  const float products = (float)std::min(a.M, a.E);
  const float tiles = (float)tiles_n * (GROUPED ? std::max(products, (float)a.M / C::BM + 0.5f * products)
                                                : (float)row_tiles<C, GROUPED>(a));
  const int mine = C::SPLIT ? (a.nkb + C::NW - 1) / C::NW : a.nkb;
  const float r = std::max(1.0f, tiles / (float)(cus * C::per_cu(OUT == Out::GATED)));
  const float mb = 1e-6f * tiles * (float)(mine * (C::SPLIT ? C::NW : 1)) * 128.0f * (float)(C::BM + C::BN);
  return c.fixed + r * (c.round + c.stage * (float)mine) + c.mb * mb;
}

template <class C_>
struct F8Form {
  using C = C_;
  F8Cost cost;
};

// f(the forms of a product)
template <bool WIDE, Out OUT, class F>
auto with_forms(F f) {
  if constexpr (OUT == Out::GATED)
    return f(F8Form<F8Cfg<1, 4, 2, 4>>{{3.531f, 2.168f, 0.933f, 0.053f}}, F8Form<F8Cfg<2, 4, 4, 4>>{{2.818f, 7.496f, 1.926f, 0.024f}});
  else if constexpr (!WIDE)
    return f(F8Form<F8Split<1, 1, 16, 1>>{{0.626f, 2.525f, 0.349f, 0.067f}}, F8Form<F8Split<1, 1, 4, 4>>{{1.191f, 1.726f, 0.202f, 0.075f}},
             F8Form<F8Split<1, 2, 8, 2>>{{0.987f, 1.871f, 0.692f, 0.028f}}, F8Form<F8Split<1, 4, 8, 1>>{{1.065f, 2.724f, 0.665f, 0.030f}},
             F8Form<F8Split<2, 2, 8, 1>>{{1.195f, 1.698f, 0.658f, 0.051f}}, F8Form<F8Split<2, 4, 4, 1>>{{1.632f, 1.905f, 0.556f, 0.058f}},
             F8Form<F8Cfg<1, 4, 2, 2>>{{1.019f, 2.687f, 0.520f, 0.038f}}, F8Form<F8Cfg<2, 2, 4, 4>>{{0.377f, 4.681f, 0.614f, 0.070f}},
             F8Form<F8Cfg<2, 4, 8, 4>>{{0.637f, 7.304f, 1.551f, 0.044f}});
  else
    return f(F8Form<F8Split<1, 1, 16, 1>>{{3.237f, 0.434f, 0.454f, 0.049f}}, F8Form<F8Split<1, 1, 4, 4>>{{2.325f, 0.828f, 0.385f, 0.054f}},
             F8Form<F8Split<1, 2, 8, 2>>{{1.768f, 1.542f, 0.623f, 0.035f}}, F8Form<F8Split<1, 4, 8, 1>>{{1.855f, 1.343f, 1.033f, 0.043f}},
             F8Form<F8Split<2, 2, 8, 1>>{{2.363f, 1.040f, 0.775f, 0.049f}}, F8Form<F8Split<2, 4, 4, 1>>{{1.029f, 2.163f, 0.757f, 0.059f}},
             F8Form<F8Cfg<1, 4, 2, 2>>{{0.121f, 3.236f, 0.645f, 0.044f}}, F8Form<F8Cfg<2, 2, 4, 4>>{{3.510f, 2.694f, 0.983f, 0.082f}});
}

// the index of the form that the product takes on a device of `cus` compute units, and its estimated time
struct Choice {
  int form;
  float us;
};
template <bool GROUPED, bool WIDE, Out OUT>
Choice least(const F8Args& a, int cus) {
  return with_forms<WIDE, OUT>([&](auto... form) {
    const float t[] = {estimate<typename decltype(form)::C, GROUPED, OUT>(a, form.cost, cus)...};
    const auto* best = std::min_element(std::begin(t), std::end(t));
    return Choice{(int)(best - std::begin(t)), *best};
  });
}

template <bool GROUPED, bool WIDE, Out OUT>
hipError_t launch_any(const F8Args& a, hipStream_t stream) {
  return with_forms<WIDE, OUT>([&](auto... form) {
    using Fn = hipError_t (*)(const F8Args&, hipStream_t);
    const Fn fn[] = {launch<typename decltype(form)::C, GROUPED, WIDE, OUT>...};
    return fn[least<GROUPED, WIDE, OUT>(a, device_cu_count()).form](a, stream);
  });
}

// rows of fp32 or bf16 that the chosen form rounds itself
template <bool WIDE, Out OUT, In IN>
bool launch_rounded(const F8Args& a, hipStream_t stream, hipError_t& e) {
  return with_forms<WIDE, OUT>([&](auto... form) {
    using Fn = hipError_t (*)(const F8Args&, hipStream_t);
    constexpr auto one = [](auto f) -> Fn {
      using C = typename decltype(f)::C;
      if constexpr (C::SPLIT && C::BM == 16) return launch<C, false, WIDE, OUT, IN>;
      else return nullptr;
    };
    const Fn fn[] = {one(form)...};
    const Fn f = fn[least<false, WIDE, OUT>(a, device_cu_count()).form];
    if (f) e = f(a, stream);
    return f != nullptr;
  });
}

F8Args sizes(int M, int K, int N, int E) {
  F8Args a = {};
  a.M = M, a.N = N, a.K = K, a.E = E, a.nkb = (K + 127) / 128, a.nnb = (N + 127) / 128;
  return a;
}

}  // namespace

int fp8_form(bool y_bf16, bool grouped, int M, int K, int N, int E, int cus) {
  const F8Args a = sizes(M, K, N, E);
  return (y_bf16 ? grouped ? least<true, false, Out::BF16>(a, cus) : least<false, false, Out::BF16>(a, cus)
                 : grouped ? least<true, true, Out::F32>(a, cus) : least<false, true, Out::F32>(a, cus)).form;
}

// Whether h = silu(g) u is rounded to FP8 by the product that makes g and u (whole blocks of h, an expert's weights within
// 32 bits of offset), or written in fp32 and rounded by a kernel of its own: the least estimated time, with figures fitted
// like the products' to 58 sizes.  By sizes alone, so that a workspace can be told from them.  Both sides, us of the whole
// layer with bf16 outputs (graph-replayed) on 64 experts of [2 x 1408, 2048]: 16 tokens of 8 choices 124 fused, 113 apart;
// 64 tokens 136 and 122; 256 tokens 142 and 155; 2048 tokens 417 and 445 (fp32 outputs 128 and 114, 137 and 123, 156 and
// 157, 441 and 477).
//   g and u are summed by the bf16 instructions whatever the output: the FP8 ones' cut moves a value of h in a few
// thousand to its neighbouring code, which is half as much again as the rounding of a bf16 output, for 199 us.
bool fp8_gated_fused(int M, int K, int I, int E) { return fp8_gated_form(M, K, I, E, 256) >= 0; }

int fp8_gated_form(int M, int K, int I, int E, int cus) {
  if (I % 128 || (int64_t)2 * I * K >= (int64_t(1) << 32)) return -1;
  const F8Args a = sizes(M, K, 2 * I, E);
  const Choice one = least<true, true, Out::GATED>(a, cus), two = least<true, true, Out::F32>(a, cus);
  const float rows = 9e-6f * (float)M * (float)I;   // MB of [g | u] and h
  return one.us < 0.837f * two.us + 4.808f + 0.484f * rows ? one.form : -1;
}

int fp8_form_name(bool y_bf16, int i, char* to, size_t n) {
  auto describe = [&](auto... form) {
    using Fn = int (*)(char*, size_t);
    const Fn fn[] = {decltype(form)::C::describe...};
    return i < 0 || i >= (int)std::size(fn) ? -1 : fn[i](to, n);
  };
  return y_bf16 ? with_forms<false, Out::BF16>(describe) : with_forms<true, Out::F32>(describe);
}

hipError_t launch_fp8_gemm(const uint8_t* X, const float* XS, int T, int K, const uint8_t* codes, const float* scales, int E,
                           int N, const int32_t* offsets, const int32_t* rows, int M, void* Y, bool y_bf16, bool fast,
                           hipStream_t stream) {
  const F8Args a = {X, XS, codes, scales, M, N, K, (K + 127) / 128, (N + 127) / 128, offsets, rows, E, T, Y, nullptr, 0};
  if (!offsets) return y_bf16 ? launch_any<false, false, Out::BF16>(a, stream) : launch_any<false, true, Out::F32>(a, stream);
  if (fast && !y_bf16) return launch_any<true, false, Out::F32>(a, stream);
  return y_bf16 ? launch_any<true, false, Out::BF16>(a, stream) : launch_any<true, true, Out::F32>(a, stream);
}

hipError_t launch_fp8_linear(const void* X, bool x_bf16, int64_t ldx, int M, int K, const uint8_t* codes, const float* scales,
                             int N, void* Y, bool y_bf16, uint8_t* x_codes, float* x_scales, hipStream_t stream) {
  hipError_t e = hipSuccess;
  if (M <= 16 && M * (int64_t)K <= kRounded) {
    F8Args a = {static_cast<const uint8_t*>(X), nullptr, codes, scales, M, N, K, (K + 127) / 128, (N + 127) / 128, nullptr,
                nullptr, 1, M, Y, nullptr, ldx};
    if (y_bf16 ? x_bf16 ? launch_rounded<false, Out::BF16, In::BF16>(a, stream, e) : launch_rounded<false, Out::BF16, In::F32>(a, stream, e)
               : x_bf16 ? launch_rounded<true, Out::F32, In::BF16>(a, stream, e) : launch_rounded<true, Out::F32, In::F32>(a, stream, e))
      return e;
  }
  e = launch_fp8_quantize(X, x_bf16, 1, M, K, ldx, false, x_codes, x_scales, stream);
  if (e != hipSuccess) return e;
  return launch_fp8_gemm(x_codes, x_scales, M, K, codes, scales, 1, N, nullptr, nullptr, M, Y, y_bf16, false, stream);
}

hipError_t launch_fp8_gated(const uint8_t* X, const float* XS, int T, int K, const uint8_t* codes, const float* scales, int E,
                            int I, const int32_t* offsets, const int32_t* rows, int M, uint8_t* h_codes, float* h_scales,
                            hipStream_t stream) {
  const F8Args a = {X, XS, codes, scales, M, 2 * I, K, (K + 127) / 128, I / 64, offsets, rows, E, T, h_codes, h_scales, 0};
  return launch_any<true, true, Out::GATED>(a, stream);
}

}  // namespace aq
