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

// The same from a wave-uniform base and the lane's 32-bit offset.  s_nop: the compiler does not
// see into the block, and a base that it read out of a vector register just before needs five
// wait states until a load may use it.
__device__ __forceinline__ void dma16_from(const uint8_t* base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base), "s"(lds) : "memory");
}

// every load and LDS write of this wave done, then the workgroup's barrier
__device__ __forceinline__ void drain_barrier() {
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// The tile kernel's matrix instructions, accumulating in place in AGPRs.  Written out because
// the compiler gives a 16 x 16 instruction another destination than its addend and then moves
// accumulators about (60 moves for 64 instructions in the loop).  It does not see the hazards
// either: s_nop 1 covers an operand that a VALU instruction wrote just before (free, the matrix
// core is busy with the instruction before), settle() the results' first reads after the loop.
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

// a wave-uniform address, in scalar registers
__device__ __forceinline__ const uint8_t* uniform(const uint8_t* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v), hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  return reinterpret_cast<const uint8_t*>(((uint64_t)hi << 32) | lo);
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
// WM x WN waves, each a (16 FM) x (16 FN) tile of 16 x 16 outputs.  (Against 32 x 32 x 64 and
// 32 x 32 x 16 the instructions 16 x 16 x 128 and 16 x 16 x 32 touch each accumulator half as
// often: on random operands, where the card's power sets the clock, 7.3 against 6.3 PFLOP/s
// and 2.06 against 1.82 in a loop of nothing else.)  K advances in stages of 128 bytes of an
// activation row (A4: 256 k, A16: 64 k) through two LDS buffers filled by LDS-DMA, one
// barrier a stage.  The scale bytes of two stages are loaded at once, through registers.
// A tile row keeps its 16-byte units permuted so that the 16 rows which a phase of a
// ds_read takes fall into all 64 banks: unit u of row r is at u ^ ((r >> 1) & 7) in rows of
// 128 bytes, at u ^ ((r >> 3) & 1) in rows of 32.
// The weight rows of a wave are stored so that lane c of its FN operands holds rows
// FN c .. FN c + FN - 1: its outputs of one row are neighbours and leave in one store, 16
// lanes 64 to 256 contiguous bytes.
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
  static_assert(BM * XB % (1024 * NW) == 0 && BN * WB % (1024 * NW) == 0, "whole loads per wave");
};

template <int ROWB>
__device__ __forceinline__ int lds_unit(int r, int u) {
  return ROWB == 128 ? u ^ ((r >> 1) & 7) : u ^ ((r >> 3) & 1);
}

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
  // stage 0 and its scale bytes first, stage 1 behind them (with a single stage that one
  // again, into the buffer that is not read)
  issue(0, 0);
  if (nblk >= C::CB) load_scales(0);
  else load_short();
  write_scales(0);
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
  issue(min(1, last), 1);
  asm volatile("s_barrier" ::: "memory");
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
    products(st_, c0, 0, C::FM, [&](int i) { load_x(buf, 1, i); });
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
  rest(c0, nblk - s * C::SB);
  if (s < last) rest(c1, nblk - (s + 1) * C::SB);
  settle(acc);
  // no load may land in LDS that the next block owns by then
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");

  // ---- outputs: lane c of operand j holds column FN c + j of its wave's columns ----
  const int col = t.n0 + wn * 16 * C::FN + C::FN * l16;
  constexpr int ES = BF16 ? 2 : 4;
  // all FN columns are inside or none, and their store aligned
  const bool whole = a.N % C::FN == 0 && (reinterpret_cast<uintptr_t>(a.Y) & (C::FN * ES - 1)) == 0;
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
      if (whole) {
        if (col < a.N) {
          if constexpr (BF16) {
            uint32_t w[C::FN / 2];
#pragma unroll
            for (int j = 0; j < C::FN / 2; ++j) w[j] = bf16_pair(o[2 * j], o[2 * j + 1]);
            __builtin_memcpy(__builtin_assume_aligned(reinterpret_cast<uint16_t*>(a.Y) + at, 2 * C::FN), w, 2 * C::FN);
          } else {
            __builtin_memcpy(__builtin_assume_aligned(reinterpret_cast<float*>(a.Y) + at, 4 * C::FN), o, 4 * C::FN);
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < C::FN; ++j)
          if (col + j < a.N) store_one<BF16>(a.Y, at + j, o[j]);
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
  if (per <= 256) return launch_tile<MxCfg<A4, 2, 2, 4, 4>, GROUPED>(a, y_bf16, stream);
  return launch_tile<MxCfg<A4, 2, 4, 8, 4>, GROUPED>(a, y_bf16, stream);
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
