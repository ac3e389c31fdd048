// swa_tile.cuh -- tiles, products and pair arithmetic shared by the sliding-window kernels
// (swa_fwd.cu, swa_bwd.cu).
#pragma once

#include <cuda.h>
#include <stdint.h>

#include "common.cuh"
#include "params.h"

namespace moba {

// A 128-row tile of D columns: a 64-column region with 128-byte swizzle, then columns
// [64, 128) the same way (D = 128) or [64, 80) with 32-byte swizzle (D = 80).
template <int D>
struct SwaTile {
  static constexpr int R0 = 128 * 128;
  static constexpr int R1 = D == 128 ? 128 * 128 : (D == 80 ? 128 * 32 : 0);
  static constexpr int TILE = R0 + R1;
  static constexpr uint32_t BYTES = 128u * D * 2u;
  static_assert(BYTES == (uint32_t)TILE, "a tile is packed");
};

// High descriptor words: 128-byte swizzle (8-row groups 1024 bytes apart) and the 32-byte
// swizzle of the D = 80 tail (256 bytes apart).
constexpr uint32_t kHi128 = desc_hi(1024, kSwizzle128), kHi32 = desc_hi(256, kSwizzle32);

// D[tmem, D columns] (+)= A[tmem] B over the tile's rows [64 half, 64 half + 64): four steps
// of 16 rows, A's in groups of 8 columns, two by two, GAP columns between the pairs.  fresh:
// the first step overwrites.
template <int D, int GAP = 0>
__device__ __forceinline__ void swa_acc(uint32_t d, uint32_t a, uint32_t tile, int half, bool fresh) {
  const uint32_t b = desc_lo(tile, D == 128 ? SwaTile<D>::R0 : 16) + half * 512;
  const uint32_t b1 = desc_lo(tile + SwaTile<D>::R0, 16) + half * 128;
#pragma unroll
  for (int kk = 0; kk < 4; ++kk) {
    const uint32_t acc = (kk == 0 && fresh) ? 0u : 1u;
    umma_ts_w(d, a + kk * 8 + (kk >> 1) * GAP, b + kk * 128, kHi128, idesc_bf16(128, D == 128 ? 128 : 64, 0, 1), acc);
    if (D == 80) umma_ts_w(d + 64, a + kk * 8 + (kk >> 1) * GAP, b1 + kk * 32, kHi32, idesc_bf16(128, 16, 0, 1), acc);
  }
}

// The same over the 32 rows from 32 quarter on: two steps.
template <int D>
__device__ __forceinline__ void swa_acc32(uint32_t d, uint32_t a, uint32_t tile, int quarter, bool fresh) {
  const uint32_t b = desc_lo(tile, D == 128 ? SwaTile<D>::R0 : 16) + quarter * 256;
  const uint32_t b1 = desc_lo(tile + SwaTile<D>::R0, 16) + quarter * 64;
#pragma unroll
  for (int kk = 0; kk < 2; ++kk) {
    const uint32_t acc = (kk == 0 && fresh) ? 0u : 1u;
    umma_ts_w(d, a + kk * 8, b + kk * 128, kHi128, idesc_bf16(128, D == 128 ? 128 : 64, 0, 1), acc);
    if (D == 80) umma_ts_w(d + 64, a + kk * 8, b1 + kk * 32, kHi32, idesc_bf16(128, 16, 0, 1), acc);
  }
}

// S (NB columns) = A B^T over the D columns; A and B K-major tiles, B's NB rows from row0 on.
template <int D, int NB>
__device__ __forceinline__ void swa_scores(uint32_t d, uint32_t a, uint32_t b, int row0) {
  constexpr uint32_t id = idesc_bf16(128, NB, 0, 0);
  const uint32_t al = desc_lo(a, 16), bl = desc_lo(b, 16) + row0 * 8;
#pragma unroll
  for (int ks = 0; ks < D / 16; ++ks) {
    const uint32_t acc = ks > 0 ? 1u : 0u;
    if (D == 80 && ks == 4)
      umma_ss_w(d, al + SwaTile<D>::R0 / 16, kHi32, desc_lo(b + SwaTile<D>::R0, 16) + row0 * 2, kHi32, id, acc);
    else
      umma_ss_w(d, al + (ks & 3) * 2 + (ks >> 2) * (SwaTile<D>::R0 / 16), kHi128,
                bl + (ks & 3) * 2 + (ks >> 2) * (SwaTile<D>::R0 / 16), kHi128, id, acc);
  }
}

// The same with A in TMEM (D / 2 columns from a): the product then takes half of what shared
// memory has to feed it.
template <int D, int NB>
__device__ __forceinline__ void swa_scores_tmem(uint32_t d, uint32_t a, uint32_t b, int row0) {
  constexpr uint32_t id = idesc_bf16(128, NB, 0, 0);
  const uint32_t bl = desc_lo(b, 16) + row0 * 8;
#pragma unroll
  for (int ks = 0; ks < D / 16; ++ks) {
    const uint32_t acc = ks > 0 ? 1u : 0u;
    if (D == 80 && ks == 4)
      umma_ts_w(d, a + ks * 8, desc_lo(b + SwaTile<D>::R0, 16) + row0 * 2, kHi32, id, acc);
    else
      umma_ts_w(d, a + ks * 8, bl + (ks & 3) * 2 + (ks >> 2) * (SwaTile<D>::R0 / 16), kHi128, id, acc);
  }
}

// 16 more columns of such a product: blocks of 32-byte rows with the 32-byte swizzle, A's in
// shared memory or in 8 columns of TMEM.
template <int NB>
__device__ __forceinline__ void swa_extra(uint32_t d, uint32_t a, int row0, uint32_t b) {
  umma_ss_w(d, desc_lo(a, 16), kHi32, desc_lo(b, 16) + row0 * 2, kHi32, idesc_bf16(128, NB, 0, 0), 1u);
}
template <int NB>
__device__ __forceinline__ void swa_extra_tmem(uint32_t d, uint32_t a, int row0, uint32_t b) {
  umma_ts_w(d, a, desc_lo(b, 16) + row0 * 2, kHi32, idesc_bf16(128, NB, 0, 0), 1u);
}

template <int D>
__device__ __forceinline__ void swa_load_tile(unsigned char *dst, const CUtensorMap *m, const CUtensorMap *m1,
                                              uint64_t *bar, int row, int h, int b) {
  tma_load_4d(dst, m, bar, 0, row, h, b);
  if (D != 64) tma_load_4d(dst + SwaTile<D>::R0, m1, bar, 64, row, h, b);
}

// Bulk copy (16-byte aligned on both sides).
__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// The end of a loading warp: the last loads of each stage land (within the limit) before the
// CTA can retire, also when the roles that wait for them have given up.  cnt: loads issued.
__device__ __forceinline__ void drain_ring(uint64_t *full, uint32_t cnt, uint32_t stages, const int *status) {
  for (uint32_t u = cnt > stages ? cnt - stages : 0; u < cnt; ++u) {
    const unsigned long long t0 = global_timer_ns();
    while (!mbar_try_wait(&full[u % stages], (u / stages) & 1) && global_timer_ns() - t0 < wait_limit_ns(status)) {}
  }
}

// Packed fp32 pairs, each lane rounded as the scalar instruction would.
__device__ __forceinline__ void fma2(float &d0, float &d1, float a0, float a1, float b, float c0, float c1) {
  const float2 d = __ffma2_rn(make_float2(a0, a1), make_float2(b, b), make_float2(c0, c1));
  d0 = d.x;
  d1 = d.y;
}
__device__ __forceinline__ void add2(float &d0, float &d1, float a0, float a1) {
  const float2 d = __fadd2_rn(make_float2(d0, d1), make_float2(a0, a1));
  d0 = d.x;
  d1 = d.y;
}
__device__ __forceinline__ void mul2(float &d0, float &d1, float a0, float a1, float b0, float b1) {
  const float2 d = __fmul2_rn(make_float2(a0, a1), make_float2(b0, b1));
  d0 = d.x;
  d1 = d.y;
}
// d = p * (v + c) on pairs.
__device__ __forceinline__ void addmul2(float &d0, float &d1, float v0, float v1, float c0, float c1,
                                        float p0, float p1) {
  const float2 d = __fmul2_rn(__fadd2_rn(make_float2(v0, v1), make_float2(c0, c1)), make_float2(p0, p1));
  d0 = d.x;
  d1 = d.y;
}

// The n lowest of 32 bits (n below 0: none, above 32: all).
__device__ __forceinline__ uint32_t first_bits(int n) {
  return n <= 0 ? 0u : (n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u);
}
// Bits e and e + 1 of b as the halves of a packed pair.
__device__ __forceinline__ uint32_t pair_mask(uint32_t b, int e) {
  return ((b >> e) & 1u ? 0x0000FFFFu : 0u) | ((b >> (e + 1)) & 1u ? 0xFFFF0000u : 0u);
}

// Test hook (moba_debug_fault_next_launch): the warp of CTA 0 that issues the accumulating
// products takes the one-shot flag and does not announce its first products, so that a wait
// for them runs out.  (This warp waits for its first operands anyway.)
__device__ __forceinline__ bool swa_take_fault(int *status, int kind) {
  if (blockIdx.x != 0) return false;
  int mine = 0;
  if ((threadIdx.x & 31) == 0) mine = atomicCAS(&status[3], kind, 0) == kind;
  return __shfl_sync(0xffffffffu, mine, 0) != 0;
}

// The end of an issuing warp: everything it issued completes (within the wait limit)
// before TMEM is released.
__device__ __forceinline__ void swa_issued(uint64_t *done, const int *status) {
  if (elect_one()) {
    umma_commit(done);
    const unsigned long long t0 = global_timer_ns();
    while (!mbar_try_wait(done, 0) && global_timer_ns() - t0 < wait_limit_ns(status)) {}
  }
}

// 16 columns of accumulators, scaled, as bf16 to a row.
__device__ __forceinline__ void store16(uint16_t *dst, const uint32_t (&o)[16], float sc) {
#pragma unroll
  for (int e = 0; e < 16; e += 8) {
    uint4 x;
    x.x = pack_bf16x2(__uint_as_float(o[e]) * sc, __uint_as_float(o[e + 1]) * sc);
    x.y = pack_bf16x2(__uint_as_float(o[e + 2]) * sc, __uint_as_float(o[e + 3]) * sc);
    x.z = pack_bf16x2(__uint_as_float(o[e + 4]) * sc, __uint_as_float(o[e + 5]) * sc);
    x.w = pack_bf16x2(__uint_as_float(o[e + 6]) * sc, __uint_as_float(o[e + 7]) * sc);
    *reinterpret_cast<uint4 *>(dst + e) = x;
  }
}

}  // namespace moba
