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
// block factor into the exact bf16 pair.  A4 runs on the block-scaled matrix instructions,
// which take the codes and the E8M0 bytes as they are: four times the bf16 rate, and the
// products of one block are exact.
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
#include <type_traits>

#include "aq_device.h"
#include "aq_kernels.h"
#include "gemm_lds.h"

namespace aq {

namespace {

using gemm::lds_addr;
using gemm::tile_of_block;

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

template <typename V>
__device__ __forceinline__ V load_any(const uint8_t* p) {
  V v;
  __builtin_memcpy(&v, p, sizeof(V));   // one unaligned load
  return v;
}

// LDS-DMA of 16 bytes per lane from the lane's own address; lane l lands at lds + 16 l.
// (M0 is a reserved register: the compiler keeps no value in it, so it is no clobber.)
__device__ __forceinline__ void dma16_at(const uint8_t* src, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(src), "s"(lds) : "memory");
}

// every load and LDS write of this wave done, then the workgroup's barrier
__device__ __forceinline__ void drain_barrier() {
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

struct MxTile {
  int e;        // expert
  int r0, r1;   // its rows of Y that the tile covers, r0 < r1
  int n0;
};

// Tile t of a grouped launch: the experts' rows cut into pieces of BM, each times the
// column tiles, the columns fastest.  The launch has at least as many blocks as tiles;
// blocks past them get false.  Every wave scans the offsets by itself, 64 experts at a
// time.  Offsets are clamped to the rows of Y and to be ascending, so no value of theirs
// leads outside the buffers.
template <int BM>
__device__ __forceinline__ bool grouped_tile(const MxArgs& a, int tiles_n, int bn, int block, MxTile& out) {
  const int lane = threadIdx.x & 63;
  auto span = [&](int e, int& lo, int& hi) {
    lo = hi = 0;
    if (e < a.E) {
      lo = min(max(a.offsets[e], 0), a.M);
      hi = min(max(a.offsets[e + 1], lo), a.M);
    }
  };
  auto scan = [&](int v) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int u = __shfl_up(v, d, 64);
      if (lane >= d) v += u;
    }
    return v;
  };
  int lo, hi, incl = 0, total = 0;
  for (int e0 = 0; e0 < a.E; e0 += 64) {
    span(e0 + lane, lo, hi);
    incl = scan((hi - lo + BM - 1) / BM);
    total += __shfl(incl, 63, 64);
  }
  const int64_t ntiles = (int64_t)total * tiles_n;
  if (block >= ntiles) return false;
  const int t = tile_of_block(block, (int)ntiles);
  const int mt = t / tiles_n;
  int base = 0;
  for (int e0 = 0; e0 < a.E; e0 += 64) {
    if (a.E > 64) {
      span(e0 + lane, lo, hi);
      incl = scan((hi - lo + BM - 1) / BM);
    }
    const uint64_t past = __ballot(base + incl > mt);
    if (past) {
      const int src = __builtin_ctzll(past);
      const int before = src ? __shfl(incl, src - 1, 64) : 0;
      const int first = __shfl(lo, src, 64), end = __shfl(hi, src, 64);
      out.e = __builtin_amdgcn_readfirstlane(e0 + src);
      out.r0 = __builtin_amdgcn_readfirstlane(first + (mt - base - before) * BM);
      out.r1 = __builtin_amdgcn_readfirstlane(min(out.r0 + BM, end));
      out.n0 = __builtin_amdgcn_readfirstlane((t - mt * tiles_n) * bn);
      return out.r0 >= first && out.r0 < end;   // false only if overlapping offsets overflowed the count
    }
    base += __shfl(incl, 63, 64);
  }
  return false;
}

// The activation row that row r of Y reads; -1 (and the address of row 0) for a listed row
// outside X.
__device__ __forceinline__ int source_row(const MxArgs& a, int r) {
  if (a.rows == nullptr) return r;
  const int i = a.rows[r];
  return i >= 0 && i < a.T ? i : -1;
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  const bf16x2 v = {(__bf16)lo, (__bf16)hi};
  return __builtin_bit_cast(uint32_t, v);
}

template <bool BF16>
__device__ __forceinline__ void store_one(void* Y, int64_t i, float v) {
  if constexpr (BF16) reinterpret_cast<__bf16*>(Y)[i] = (__bf16)v;
  else reinterpret_cast<float*>(Y)[i] = v;
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

// ---- few rows -----------------------------------------------------------------------------
// Bound by the weight bytes: a block takes 16 weight rows and up to 16 MT activation rows,
// its waves share K in chunks of 512 (lane group g of 16 lanes: blocks 4 g .. 4 g + 3 of the
// chunk, 64 contiguous bytes of its row), codes straight from memory into the operands, the
// next chunk's codes requested before the current one is multiplied.  The waves' sums are
// added in LDS in wave order.
template <bool A4, int MT, int NW, bool GROUPED, bool BF16>
__global__ __launch_bounds__(64 * NW) void mxfp4_rows_kernel(MxArgs a) {
  __shared__ float part[NW][MT][4][64];
  const int lane = threadIdx.x & 63;
  const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tiles_n = (a.N + 15) >> 4;
  MxTile t;
  if constexpr (GROUPED) {
    if (!grouped_tile<16 * MT>(a, tiles_n, 16, blockIdx.x, t)) return;   // the whole block
  } else {
    t = MxTile{0, 0, a.M, 16 * tile_of_block(blockIdx.x, tiles_n)};
  }
  const int l16 = lane & 15, g = lane >> 4;
  const int nblk = a.K >> 5;
  const int64_t wr = (int64_t)t.e * a.N + min(t.n0 + l16, a.N - 1);
  const uint8_t* wc = a.W + wr * (a.K >> 1);
  const uint8_t* ws = a.WS + wr * nblk;
  const uint8_t* xc[MT];
  const uint8_t* xs[MT];
  bool live[MT], lost[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int r = t.r0 + 16 * i + l16;
    live[i] = r < t.r1;
    const int src = live[i] ? source_row(a, r) : 0;
    lost[i] = src < 0;
    xc[i] = a.X + (int64_t)max(src, 0) * a.xrow;
    xs[i] = A4 ? a.XS + (int64_t)max(src, 0) * nblk : nullptr;
  }
  // the dword of scale bytes of blocks b .. b + 3 (zero past the row's end)
  auto scales4 = [&](const uint8_t* row, int b) -> uint32_t {
    if (nblk >= 4) {
      const int at = min(b, nblk - 4);
      const int sh = 8 * (b - at);
      const uint32_t v = load_any<uint32_t>(row + at);
      return sh < 32 ? v >> sh : 0u;
    }
    uint32_t v = 0;
    for (int i = 0; i < 4; ++i)
      if (b + i < nblk) v |= (uint32_t)row[b + i] << (8 * i);
    return v;
  };
  f32x4 acc[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  const int nchunk = (nblk + 15) >> 4;
  u32x4 wq[4];
  uint32_t wsc = 0;
  auto fetch = [&](int c) {
    const int b = 16 * c + 4 * g;
#pragma unroll
    for (int u = 0; u < 4; ++u) wq[u] = *reinterpret_cast<const u32x4*>(wc + 16 * min(b + u, nblk - 1));
    wsc = scales4(ws, b);
  };
  if (wid < nchunk) fetch(wid);
  for (int c = wid; c < nchunk; c += NW) {
    const int b = 16 * c + 4 * g;
    u32x4 w[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) w[u] = wq[u];
    const uint32_t sw = wsc;
    if constexpr (A4) {
      u32x4 x[MT][4];
      uint32_t sx[MT];
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        sx[i] = scales4(xs[i], b);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          x[i][u] = *reinterpret_cast<const u32x4*>(xc[i] + 16 * min(b + u, nblk - 1));
          if (b + u >= nblk) x[i][u] = u32x4{0, 0, 0, 0};
        }
      }
      if (c + NW < nchunk) fetch(c + NW);
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        acc[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(codes8(x[i][0]), codes8(w[0]), acc[i], 4, 4, 0, (int)sx[i], 0, (int)sw);
        acc[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(codes8(x[i][1]), codes8(w[1]), acc[i], 4, 4, 1, (int)sx[i], 1, (int)sw);
        acc[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(codes8(x[i][2]), codes8(w[2]), acc[i], 4, 4, 2, (int)sx[i], 2, (int)sw);
        acc[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(codes8(x[i][3]), codes8(w[3]), acc[i], 4, 4, 3, (int)sx[i], 3, (int)sw);
      }
    } else {
      if (c + NW < nchunk) fetch(c + NW);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float f = __uint_as_float(((sw >> (8 * u)) & 255u) << 23);
        u32x4 x[MT][4];
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            x[i][q] = u32x4{0, 0, 0, 0};
            if (live[i] && b + u < nblk) x[i][q] = *reinterpret_cast<const u32x4*>(xc[i] + 64 * (b + u) + 16 * q);
          }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const bf16x8 bw = mx_bf16x8(w[u][q], f);
#pragma unroll
          for (int i = 0; i < MT; ++i)
            acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x[i][q]), bw, acc[i], 0, 0, 0);
        }
      }
    }
  }
  // rows of Y whose listed activation row is outside X become NaN: the lane that holds
  // operand row r tells the lanes that hold it as outputs
  uint64_t lostm[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) lostm[i] = __ballot(lost[i]);
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) part[wid][i][j][lane] = acc[i][j];
  __syncthreads();
  const int n = t.n0 + l16;
#pragma unroll
  for (int o = 0; o < MT * 4; o += NW) {
    const int idx = o + wid;   // (i, j) of the outputs this wave adds and stores
    if (idx < MT * 4) {
      const int i = idx >> 2, j = idx & 3;
      float v = part[0][i][j][lane];
#pragma unroll
      for (int w = 1; w < NW; ++w) v += part[w][i][j][lane];
      const int rl = 4 * g + j;
      const int r = t.r0 + 16 * i + rl;
      if (GROUPED) {
        uint64_t m = 0;
#pragma unroll
        for (int q = 0; q < MT; ++q)
          if (q == i) m = lostm[q];
        if ((m >> rl) & 1) v = __builtin_nanf("");
      }
      if (r < t.r1 && n < a.N) store_one<BF16>(a.Y, (int64_t)r * a.N + n, v);
    }
  }
}

// ---- many rows ----------------------------------------------------------------------------
// WM x WN waves, each a (32 FM) x (32 FN) tile of 32 x 32 outputs.  K advances in stages of
// 128 bytes of an activation row (A4: 256 k, A16: 64 k) through two LDS buffers filled by
// LDS-DMA: while one stage is multiplied the next one is in flight, one barrier a stage.
// Tile rows of 128 bytes keep unit u (16 bytes) of row r at u ^ ((r >> 1) & 7): two rows
// span the 64 banks, so the 16 rows that a phase of a ds_read_b128 takes (the same unit of
// each) fall into all of them.  The 32-byte weight rows of A16 use u ^ ((r >> 3) & 1).
// The weight rows of a wave are stored so that lane c of its FN operands holds rows
// FN c .. FN c + FN - 1: its outputs of one row are neighbours and leave in one store, 32
// lanes 128 or 256 contiguous bytes.
template <bool A4_, int WM_, int WN_, int FM_, int FN_>
struct MxCfg {
  static constexpr bool A4 = A4_;
  static constexpr int WM = WM_, WN = WN_, FM = FM_, FN = FN_;
  static constexpr int NW = WM * WN, NT = 64 * NW;
  static constexpr int BM = 32 * FM * WM, BN = 32 * FN * WN;
  static constexpr int KS = A4 ? 256 : 64;           // k per stage
  static constexpr int WB = A4 ? 128 : 32;           // weight bytes per row and stage
  static constexpr int SPC = 512 / KS;               // stages per chunk of scale bytes
  static constexpr int A_DMA = BM / 8 / NW;          // loads per wave and stage, 1 KiB each
  static constexpr int B_DMA = BN * WB / 1024 / NW;
  static constexpr int SROWS = A4 ? BM + BN : BN;    // rows of scale bytes
  static constexpr int SPT = (SROWS + NT - 1) / NT;  // of them per thread
  static_assert(BM % (8 * NW) == 0 && (BN * WB) % (1024 * NW) == 0, "whole loads per wave");
};

template <class C, bool GROUPED, bool BF16>
__global__ __launch_bounds__(C::NT, 1) void mxfp4_tile_kernel(MxArgs a) {
  __shared__ __attribute__((aligned(1024))) uint8_t As[2][C::BM * 128];
  __shared__ __attribute__((aligned(1024))) uint8_t Bs[2][C::BN * C::WB];
  __shared__ __attribute__((aligned(16))) uint8_t Ss[2][C::SROWS * 16];
  __shared__ uint8_t lost[GROUPED ? C::BM : 1];
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wid = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wid / C::WN, wn = wid % C::WN;
  const int l32 = lane & 31, lh = lane >> 5;
  const int tiles_n = (a.N + C::BN - 1) / C::BN;
  MxTile t;
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
  const int nstage = (a.K + C::KS - 1) / C::KS;
  const int krow = a.K >> 1;   // bytes of a code row

  // ---- sources of the LDS-DMA loads ----
  // weight row of LDS row i: wave region i / (32 FN), operand (i / 32) % FN, lane i % 32
  auto brow = [&](int i) {
    const int n = t.n0 + (i / (32 * C::FN)) * (32 * C::FN) + C::FN * (i & 31) + (i / 32) % C::FN;
    return (int64_t)t.e * a.N + min(n, a.N - 1);
  };
  const uint8_t* asrc[C::A_DMA];
  const uint8_t* bsrc[C::B_DMA];
  int aunit[C::A_DMA], bunit[C::B_DMA];
#pragma unroll
  for (int j = 0; j < C::A_DMA; ++j) {
    const int i = 8 * (j * C::NW + wid) + (lane >> 3);
    aunit[j] = (lane & 7) ^ ((i >> 1) & 7);
    const int src = max(GROUPED ? source_row(a, min(t.r0 + i, t.r1 - 1)) : min(t.r0 + i, t.r1 - 1), 0);
    asrc[j] = a.X + (int64_t)src * a.xrow + 16 * aunit[j];
  }
#pragma unroll
  for (int j = 0; j < C::B_DMA; ++j) {
    if constexpr (C::A4) {
      const int i = 8 * (j * C::NW + wid) + (lane >> 3);
      bunit[j] = (lane & 7) ^ ((i >> 1) & 7);
      bsrc[j] = a.W + brow(i) * krow + 16 * bunit[j];
    } else {
      const int i = 32 * (j * C::NW + wid) + (lane >> 1);
      bunit[j] = (lane & 1) ^ ((i >> 3) & 1);
      bsrc[j] = a.W + brow(i) * krow + 16 * bunit[j];
    }
  }
  // In the last stage the units past the row's end read its last unit instead.  A unit is
  // 32 k of an A4 row and of a weight row, 8 k of a bf16 row.
  auto issue = [&](int s, int buf) {
    const int left = a.K - s * C::KS;
    const bool tail = left < C::KS;
    const int au = C::A4 ? left >> 5 : left >> 3, bu = left >> 5;
#pragma unroll
    for (int j = 0; j < C::A_DMA; ++j) {
      const uint8_t* p = asrc[j] + (int64_t)s * 128;
      if (tail && aunit[j] >= au) p -= 16 * (aunit[j] - au + 1);
      dma16_at(p, __builtin_amdgcn_readfirstlane(lds_addr(&As[buf][1024 * (j * C::NW + wid)])));
    }
#pragma unroll
    for (int j = 0; j < C::B_DMA; ++j) {
      const uint8_t* p = bsrc[j] + (int64_t)s * C::WB;
      if (tail && bunit[j] >= bu) p -= 16 * (bunit[j] - bu + 1);
      dma16_at(p, __builtin_amdgcn_readfirstlane(lds_addr(&Bs[buf][1024 * (j * C::NW + wid)])));
    }
  };

  // ---- scale bytes: 16 per row and chunk of 512 k, through registers ----
  const uint8_t* ssrc[C::SPT];
  u32x4 sreg[C::SPT];
#pragma unroll
  for (int j = 0; j < C::SPT; ++j) {
    const int i = min(j * C::NT + tid, C::SROWS - 1);
    if (C::A4 && i < C::BM) {
      const int src = GROUPED ? source_row(a, min(t.r0 + i, t.r1 - 1)) : min(t.r0 + i, t.r1 - 1);
      ssrc[j] = a.XS + (int64_t)max(src, 0) * nblk;
    } else {
      ssrc[j] = a.WS + brow(C::A4 ? i - C::BM : i) * nblk;
    }
  }
  auto load_scales = [&](int c) {
    const int left = nblk - 16 * c;
#pragma unroll
    for (int j = 0; j < C::SPT; ++j) {
      if (left >= 16) {
        sreg[j] = load_any<u32x4>(ssrc[j] + 16 * c);
      } else if (nblk >= 16) {
        // the row's last 16 bytes, those of earlier chunks shifted out and zeros in
        const u32x4 v = load_any<u32x4>(ssrc[j] + nblk - 16);
        uint64_t lo = ((uint64_t)v[1] << 32) | v[0], hi = ((uint64_t)v[3] << 32) | v[2];
        int sh = 16 - left;   // 1 .. 15 bytes
        if (sh >= 8) {
          lo = hi;
          hi = 0;
          sh -= 8;
        }
        if (sh > 0) {
          lo = (lo >> (8 * sh)) | (hi << (64 - 8 * sh));
          hi >>= 8 * sh;
        }
        sreg[j] = u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
      } else {
        u32x4 v = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 15; ++i)
          if (i < left) v[i >> 2] |= (uint32_t)ssrc[j][i] << (8 * (i & 3));
        sreg[j] = v;
      }
    }
  };
  auto write_scales = [&](int c) {
#pragma unroll
    for (int j = 0; j < C::SPT; ++j)
      if ((j + 1) * C::NT <= C::SROWS || j * C::NT + tid < C::SROWS)
        *reinterpret_cast<u32x4*>(&Ss[c & 1][16 * (j * C::NT + tid)]) = sreg[j];
  };

  f32x16 acc[C::FM][C::FN];
#pragma unroll
  for (int i = 0; i < C::FM; ++i)
#pragma unroll
    for (int j = 0; j < C::FN; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;

  auto row128 = [&](const uint8_t* base, int r, int u) {
    return *reinterpret_cast<const u32x4*>(base + 128 * r + 16 * (u ^ ((r >> 1) & 7)));
  };
  // the products of stage s; valid: its blocks of 32 k
  auto multiply = [&](int s, int buf, auto tail_, int valid) {
    constexpr bool TAIL = decltype(tail_)::value;
    const uint8_t* sc = Ss[(s / C::SPC) & 1];
    const int am = wm * 32 * C::FM, bn = wn * 32 * C::FN;
    if constexpr (C::A4) {
      // half h of the lanes takes blocks 4 h .. 4 h + 3 of the stage, one per instruction
      uint32_t sa[C::FM], sb[C::FN];
#pragma unroll
      for (int i = 0; i < C::FM; ++i)
        sa[i] = *reinterpret_cast<const uint32_t*>(sc + 16 * (am + 32 * i + l32) + 8 * (s & 1) + 4 * lh);
#pragma unroll
      for (int j = 0; j < C::FN; ++j)
        sb[j] = *reinterpret_cast<const uint32_t*>(sc + 16 * (C::BM + bn + 32 * j + l32) + 8 * (s & 1) + 4 * lh);
      auto step = [&](auto q_) {
        constexpr int Q = decltype(q_)::value;
        if (TAIL && Q >= valid) return;
        i32x8 x[C::FM], w[C::FN];
#pragma unroll
        for (int i = 0; i < C::FM; ++i) x[i] = codes8(row128(As[buf], am + 32 * i + l32, 4 * lh + Q));
#pragma unroll
        for (int j = 0; j < C::FN; ++j) w[j] = codes8(row128(Bs[buf], bn + 32 * j + l32, 4 * lh + Q));
#pragma unroll
        for (int i = 0; i < C::FM; ++i)
#pragma unroll
          for (int j = 0; j < C::FN; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x[i], w[j], acc[i][j], 4, 4, Q, (int)sa[i], Q, (int)sb[j]);
      };
      step(std::integral_constant<int, 0>{});
      step(std::integral_constant<int, 1>{});
      step(std::integral_constant<int, 2>{});
      step(std::integral_constant<int, 3>{});
    } else {
      // half h of the lanes takes block h of the stage, 8 k per instruction
      u32x4 w[C::FN];
      float f[C::FN];
#pragma unroll
      for (int j = 0; j < C::FN; ++j) {
        const int r = bn + 32 * j + l32;
        w[j] = *reinterpret_cast<const u32x4*>(Bs[buf] + 32 * r + 16 * (lh ^ ((r >> 3) & 1)));
        f[j] = __uint_as_float((uint32_t)sc[16 * r + 2 * (s % C::SPC) + lh] << 23);
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        bf16x8 x[C::FM], b[C::FN];
#pragma unroll
        for (int i = 0; i < C::FM; ++i) {
          u32x4 v = row128(As[buf], am + 32 * i + l32, 4 * lh + q);
          if (TAIL && lh >= valid) v = u32x4{0, 0, 0, 0};
          x[i] = __builtin_bit_cast(bf16x8, v);
        }
#pragma unroll
        for (int j = 0; j < C::FN; ++j) b[j] = mx_bf16x8(w[j][q], f[j]);
#pragma unroll
        for (int i = 0; i < C::FM; ++i)
#pragma unroll
          for (int j = 0; j < C::FN; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x[i], b[j], acc[i][j], 0, 0, 0);
      }
    }
  };

  if constexpr (GROUPED) {
    for (int i = tid; i < C::BM; i += C::NT) lost[i] = source_row(a, min(t.r0 + i, t.r1 - 1)) < 0;
  }
  load_scales(0);
  issue(0, 0);
  const int nfull = a.K / C::KS;
  for (int s = 0; s < nfull; ++s) {
    if (s % C::SPC == 0) write_scales(s / C::SPC);
    drain_barrier();
    if (s + 1 < nstage) {
      issue(s + 1, (s + 1) & 1);
      if ((s + 1) % C::SPC == 0) load_scales((s + 1) / C::SPC);
    }
    multiply(s, s & 1, std::false_type{}, 0);
  }
  if (nfull < nstage) {
    if (nfull % C::SPC == 0) write_scales(nfull / C::SPC);
    drain_barrier();
    multiply(nfull, nfull & 1, std::true_type{}, nblk - nfull * (C::KS / 32));
  }

  // ---- outputs: lane c of operand pair j holds columns FN c .. of its wave's columns ----
  const int col = t.n0 + wn * 32 * C::FN + C::FN * l32;
  const bool pairs = (a.N & 1) == 0;   // both columns of a pair are inside, and its store aligned
#pragma unroll
  for (int i = 0; i < C::FM; ++i)
#pragma unroll
    for (int v = 0; v < 16; ++v) {
      const int rl = wm * 32 * C::FM + 32 * i + 8 * (v >> 2) + 4 * lh + (v & 3);
      const int r = t.r0 + rl;
      if (r >= t.r1) continue;
      const int64_t at = (int64_t)r * a.N + col;
      float o[C::FN];
#pragma unroll
      for (int j = 0; j < C::FN; ++j) {
        o[j] = acc[i][j][v];
        if (GROUPED && lost[rl]) o[j] = __builtin_nanf("");
      }
      static_assert(C::FN == 2, "outputs leave in pairs");
      if (pairs) {
        if (col < a.N) {
          if constexpr (BF16) *reinterpret_cast<uint32_t*>(reinterpret_cast<uint16_t*>(a.Y) + at) = bf16_pair(o[0], o[1]);
          else *reinterpret_cast<float2*>(reinterpret_cast<float*>(a.Y) + at) = float2{o[0], o[1]};
        }
      } else {
        if (col < a.N) store_one<BF16>(a.Y, at, o[0]);
        if (col + 1 < a.N) store_one<BF16>(a.Y, at + 1, o[1]);
      }
    }
}

template <class C, bool GROUPED>
hipError_t launch_tile(const MxArgs& a, bool y_bf16, hipStream_t stream) {
  const int64_t tiles_n = (a.N + C::BN - 1) / C::BN;
  // a grouped launch has at most one part-filled row tile per expert with rows
  const int64_t tiles_m = GROUPED ? std::min<int64_t>(a.M, a.M / C::BM + a.E) : (a.M + C::BM - 1) / C::BM;
  const dim3 grid((unsigned)(tiles_m * tiles_n)), block(C::NT);
  if (y_bf16) hipLaunchKernelGGL((mxfp4_tile_kernel<C, GROUPED, true>), grid, block, 0, stream, a);
  else hipLaunchKernelGGL((mxfp4_tile_kernel<C, GROUPED, false>), grid, block, 0, stream, a);
  return hipGetLastError();
}

template <bool A4, int MT, int NW, bool GROUPED>
hipError_t launch_rows(const MxArgs& a, bool y_bf16, hipStream_t stream) {
  const int64_t tiles_n = (a.N + 15) / 16;
  const int64_t tiles_m = GROUPED ? std::min<int64_t>(a.M, a.M / (16 * MT) + a.E) : 1;
  const dim3 grid((unsigned)(tiles_m * tiles_n)), block(64 * NW);
  if (y_bf16) hipLaunchKernelGGL((mxfp4_rows_kernel<A4, MT, NW, GROUPED, true>), grid, block, 0, stream, a);
  else hipLaunchKernelGGL((mxfp4_rows_kernel<A4, MT, NW, GROUPED, false>), grid, block, 0, stream, a);
  return hipGetLastError();
}

template <bool A4, bool GROUPED>
hipError_t launch_any(const MxArgs& a, bool y_bf16, hipStream_t stream) {
  const int per = GROUPED ? (a.M + a.E - 1) / a.E : a.M;   // rows of a product (grouped: their mean)
  if (per <= 16) return launch_rows<A4, 1, 4, GROUPED>(a, y_bf16, stream);
  if (per <= 32) return launch_rows<A4, 2, 4, GROUPED>(a, y_bf16, stream);
  if (per <= 64) return launch_rows<A4, 4, 4, GROUPED>(a, y_bf16, stream);
  if (per <= 256) return launch_tile<MxCfg<A4, 2, 2, 2, 2>, GROUPED>(a, y_bf16, stream);
  return launch_tile<MxCfg<A4, 2, 4, 4, 2>, GROUPED>(a, y_bf16, stream);
}

}  // namespace

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
