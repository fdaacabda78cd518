// Parts that the block-scaled products share (gfx950): LDS-DMA with an address for each lane, the tiles of a
// product grouped by expert, and the stores of a tile's rows.
#pragma once

#include "aq_device.h"
#include "gemm_lds.h"

namespace aq {
namespace gemm {

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

// a wave-uniform address, in scalar registers
__device__ __forceinline__ const uint8_t* uniform(const uint8_t* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v), hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  return reinterpret_cast<const uint8_t*>(((uint64_t)hi << 32) | lo);
}

struct Tile {
  int e;        // expert
  int r0, r1;   // its rows of Y that the tile covers, r0 < r1
  int n0;
};

// Tile `block` of a grouped product: the experts' rows cut into pieces of BM, each times the
// column tiles, the columns fastest.  `most` is the host's bound of their number, ntiles becomes the number;
// tiles past it get false.  Every wave scans the offsets by itself, 64 experts at a
// time.  Offsets are clamped to the rows of Y and an expert's end to its start, so no value of
// theirs leads outside the buffers.
template <int BM, class Args>
__device__ __forceinline__ bool grouped_tile(const Args& a, int tiles_n, int bn, int block, Tile& out, int64_t most, int& ntiles) {
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
  // (no more than `most`, unless overlapping offsets count rows twice)
  ntiles = __builtin_amdgcn_readfirstlane((int)min((int64_t)total * tiles_n, most));
  if (block >= ntiles) return false;
  const int t = tile_of_block(block, ntiles);
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

// the tile of this block, in a launch with a block for every tile
template <int BM, class Args>
__device__ __forceinline__ bool grouped_tile(const Args& a, int tiles_n, int bn, int block, Tile& out) {
  int ntiles;
  return grouped_tile<BM>(a, tiles_n, bn, block, out, (int64_t)gridDim.x, ntiles);
}

// The activation row that row r of Y reads; -1 (and the address of row 0) for a listed row
// outside X.
template <class Args>
__device__ __forceinline__ int source_row(const Args& a, int r) {
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

// FN neighbouring outputs of one row from column `col` on, in one store where all are inside
// (rows of Y start at any element: an unaligned store, which the hardware takes)
template <bool BF16, int FN, class Args>
__device__ __forceinline__ void store_row(const Args& a, int64_t at, int col, const float (&o)[FN]) {
  if (col + FN <= a.N) {
    if constexpr (FN == 1) {
      store_one<BF16>(a.Y, at, o[0]);
    } else if constexpr (BF16) {
      typedef uint32_t vec __attribute__((ext_vector_type(FN / 2), aligned(2)));
      vec v;
#pragma unroll
      for (int j = 0; j < FN / 2; ++j) v[j] = bf16_pair(o[2 * j], o[2 * j + 1]);
      *reinterpret_cast<vec*>(reinterpret_cast<uint16_t*>(a.Y) + at) = v;
    } else {
      typedef float vec __attribute__((ext_vector_type(FN), aligned(4)));
      vec v;
#pragma unroll
      for (int j = 0; j < FN; ++j) v[j] = o[j];
      *reinterpret_cast<vec*>(reinterpret_cast<float*>(a.Y) + at) = v;
    }
  } else {
#pragma unroll
    for (int j = 0; j < FN; ++j)
      if (col + j < a.N) store_one<BF16>(a.Y, at + j, o[j]);
  }
}

}  // namespace gemm
}  // namespace aq
