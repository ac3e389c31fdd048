// swa_bwd.cu -- backward of sliding-window attention with sinks on sm_100a tensor cores.
//
// [SWA] = "SWA + MoE: 어텐션과 희소 전문가", Bit-Axon architecture page (§"어텐션 공식",
//         §"슬라이딩 윈도우 마스크").
//
// Row i attends the keys j <= i with i - j < window or j < sink.  With z_ij = scale q_i.k_j,
// p_ij = exp(z_ij - lse_i) and the upstream gradient dO:
//     D_i = dO_i . o_i,  dz_ij = p_ij (dO_i . v_j - D_i)
//     dQ_i = scale sum_j dz_ij k_j,  dK_j = scale sum_i dz_ij q_i,  dV_j = sum_i p_ij dO_i
// (a KV head's dK and dV sum over the q-heads that read it).  No atomics: every sum has one
// order, so results repeat bit for bit.
//
//   swa_bwd_prep_kernel   per row -lse log2(e) and -D, in the tiles' order, and the same two
//                         as columns for the products of the dK / dV kernel; HBM-bound
//   swa_bwd_dq_kernel     query-stationary: a 128-row tile walks its key chunks (the sinks'
//                         chunks before the band, then the band): S = Q K^T, dP = dO V^T,
//                         dS = P (dP - D) on the CUDA cores, dQ += dS K in TMEM; written once
//   swa_bwd_dkdv_kernel   key-stationary: a 128-key tile walks the query tiles that attend
//                         it, of every q-head of its group: S^T = K Q^T, dP^T = V dO^T,
//                         dV += P^T dO, dK += dS^T Q in TMEM; written once.  The sinks' key
//                         tiles are attended by every later row, a walk up to N / window
//                         times as long, so theirs are cut into parts that leave fp32 sums
//   swa_bwd_join_kernel   adds the parts of the sinks' key tiles, in order; latency-bound
//
// P and dz are rounded to bf16, their products' operand type (two terms of each would double
// three of the five products): up to 2^-8 of each value, the same step as the results'; gradients
// are then off by 0.0024 of their norm, against 0.0017 by the rounding of the results alone.
// Sums, statistics and accumulators are fp32.  D takes `out` as it was returned, in bf16, so that
// the forward writes nothing more: where one or two keys hold a row, dP - D cancels and gradients
// are off by 0.003 to 0.006.
//
// Both tile kernels compute S and dP again (7 products instead of 5): a single pass would
// have to add dQ in global memory from every key tile, in an order that varies.  They are
// bound by the CUDA cores: per 128 x 128 tile 16384 exponentials at 16 a cycle are 1024
// cycles, against 768 (dQ) or 1024 (dK, dV) cycles of products at D = 128, and a chain
// (scores to registers, exponentials, write-back, product) that must not be waited for.  So
// the elementwise work goes in four groups of four warps with 32 columns each (two groups of
// 64 columns: 1038 against 881 us for dQ), the next scores are issued while these are worked
// on, and the steps of consecutive items run on without a gap: the next item's first products
// are issued before the last item's are summed up.
// Measured (batch 1, 32 heads, d = 80, N = 16384, window 4096, 4 sinks): statistics 46 us
// (4.2 TB/s), dQ 855 us (1056 TFLOP/s over its 3 products), dK and dV 1028 us (1171 TFLOP/s
// over 4), parts 5 us, at a power-capped 1.3-1.6 GHz; a tile takes 1892 and 2270 cycles.
// 8192 tokens, 8 heads over 4, d = 128, window 512, 130 sinks: 11, 48, 85 and 4 us.
//   warp 0      TMA: K and V
//   warp 1      issues S and dP (TMEM owner)
//   warp 2      issues the accumulating products
//   warp 3      TMA: Q with dO (and the row statistics)
//   warps 4-19  elementwise groups 0 - 3 of 32 columns each; a thread owns one TMEM lane
// Issue blocks until the tensor core has room, and a wait costs 85 cycles even when its
// phase is complete, so one warp that issues everything leaves the tensor core idle during
// its waits; two overlap theirs.  Every role runs as a whole warp: a lane that polls alone
// under divergence sees a phase 400-700 cycles late, a whole warp 130.
// Every wait is bounded, as in the forward.
#include <cuda.h>
#include <cuda_bf16.h>
#include <math.h>
#include <stdint.h>

#include "common.cuh"
#include "params.h"
#include "rows.cuh"
#include "swa_tile.cuh"

namespace moba {

constexpr int kSwaBwdThreads = 640;

// The statistics of a query tile as 16 more columns of its Q and dO (dK / dV kernel): there
// a thread holds a key and every query of the tile, so -lse / scale and -D would have to come
// through shared memory for each of them (measured: 1024 cycles a tile of shared-memory
// bandwidth that the products need).  Instead S^T - lse / scale and dP^T - D come out of
// the products: the columns hold each value in three bf16 terms (2^-24 of it left over),
// against a constant block of ones in the columns of the value that is wanted.
// A block: 128 rows of 32 bytes with the 32-byte swizzle, 4 KB.
constexpr int kSwaExtra = 128 * 32;

__device__ __forceinline__ uint32_t extra_offset(int row, int chunk) {
  return row * 32 + ((chunk ^ ((row >> 2) & 1)) << 4);
}

// x = t0 + t1 + t2 in bf16 (bits), up to 2^-24 of it.
__device__ __forceinline__ void split3(float x, uint32_t *t) {
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const uint32_t h = pack_bf16x2(x, 0.f) & 0xFFFFu;
    t[i] = h;
    x -= __uint_as_float(h << 16);
  }
}

// ------------------------------------------------------------------ prep

// nb: blocks of a head; their warps take its groups of rows in turn.
template <int D>
__global__ void __launch_bounds__(256) swa_bwd_prep_kernel(const SwaBwdParams p, int nb) {
  constexpr int LPR = RowLanes<D>::LPR, RPW = RowLanes<D>::RPW;
  const int lane = threadIdx.x & 31;
  const int sub = min(lane / LPR, RPW - 1), v = lane - sub * LPR, base = sub * LPR;
  const bool in = v < LPR;
  const int vv = in ? v : 0;
  const int padded = p.nt * kTileRows;
  const int groups = (padded + RPW - 1) / RPW;
  const long long bh = blockIdx.x / nb;
  const int b = (int)(bh / p.hq), h = (int)(bh % p.hq);
  const uint16_t *op = p.out + b * p.o_sb + h * p.o_sh + vv * 8, *gp = p.dout + b * p.do_sb + h * p.do_sh + vv * 8;
  for (int u = (int)(blockIdx.x % nb) * 8 + (threadIdx.x >> 5); u < groups; u += nb * 8) {
    const int i = u * RPW + sub;
    const bool live = in && i < p.N;
    float acc = 0.f;
    if (live) {
      float x[8], g[8];
      unpack8(__ldg(reinterpret_cast<const uint4 *>(op + (int64_t)i * p.o_sn)), x);
      unpack8(__ldg(reinterpret_cast<const uint4 *>(gp + (int64_t)i * p.do_sn)), g);
#pragma unroll
      for (int e = 0; e < 8; ++e) acc = fmaf(x[e], g[e], acc);
    }
    acc = row_sum<D>(acc, base, vv);
    if (in && v == 0 && i < padded) {
      float *st = p.stat + (bh * p.nt + i / kTileRows) * 256 + (i & 127);
      const float lse = live ? p.lse[bh * p.N + i] : 0.f;
      st[0] = live ? -lse * 1.4426950408889634f : -INFINITY;
      st[128] = live ? -acc : 0.f;
      // (Rows behind the last: far below every score, and finite, since the other product
      // multiplies it by zero.)
      uint32_t t[6];
      split3(live ? -lse / p.scale : -1e30f, t);
      split3(live ? -acc : 0.f, t + 3);
      unsigned char *blk = reinterpret_cast<unsigned char *>(p.extra + (bh * p.nt + i / kTileRows) * (kSwaExtra / 2));
      *reinterpret_cast<uint4 *>(blk + extra_offset(i & 127, 0)) =
          make_uint4(t[0] | t[1] << 16, t[2] | t[3] << 16, t[4] | t[5] << 16, 0u);
      *reinterpret_cast<uint4 *>(blk + extra_offset(i & 127, 1)) = make_uint4(0u, 0u, 0u, 0u);
    }
  }
}

// ------------------------------------------------------------------ dQ

// Work item u: one 128-row query tile; its key chunks: ns chunks of sinks from key 0, then
// the band's from chunk c0.
struct SwaDqItem {
  int b, h, hk, qt, ns, c0, nc;
};

__device__ __forceinline__ SwaDqItem swa_dq_item(const SwaBwdParams &p, int u) {
  SwaDqItem w;
  w.qt = p.nt - 1 - u % p.nt;                    // later (longer) walks first
  const int bh = u / p.nt;
  w.b = bh / p.hq;
  w.h = bh % p.hq;
  w.hk = w.h / p.G;
  w.c0 = max(0, w.qt * kTileRows - p.window + 1) / kTileKeys;
  w.ns = min((p.sink + kTileKeys - 1) / kTileKeys, w.c0);
  w.nc = w.ns + w.qt - w.c0 + 1;
  return w;
}

__device__ __forceinline__ int swa_dq_key(const SwaDqItem &w, int m) {
  return (m < w.ns ? m : w.c0 + m - w.ns) * kTileKeys;
}

template <int D>
struct SwaDqCfg {
  static constexpr int QS = D == 128 ? 1 : 2;              // Q / dO stages
  static constexpr int NK = D == 128 ? 3 : (D == 80 ? 4 : 5);  // K stages (held until dQ)
  static constexpr int NV = D == 128 ? 2 : (D == 80 ? 3 : 4);  // V stages
  // TMEM: S, dP, two dS slots of 64 columns, dQ.
  static constexpr uint32_t P0 = 128, DS0 = 256, ACC = 384;
  static constexpr int Q_OFF = 0;
  static constexpr int DO_OFF = QS * SwaTile<D>::TILE;
  static constexpr int K_OFF = 2 * QS * SwaTile<D>::TILE;
  static constexpr int V_OFF = K_OFF + NK * SwaTile<D>::TILE;
  static constexpr int BAR_OFF = V_OFF + NV * SwaTile<D>::TILE;
  static constexpr int SMEM = BAR_OFF + 1024 + 1024;
  static_assert(SMEM <= 232448, "shared memory of a CTA");
};

struct SwaBars {
  uint64_t q_full[4], q_empty[4];
  uint64_t k_full[5], k_empty[5], v_full[5], v_empty[5];
  // Per group (dQ kernel: of both): products ready; read into registers; dS (and P) written
  // back, of even and odd steps: a step's products are issued before the last step's
  // write-back is waited for, so two write-backs may complete before that wait looks.
  uint64_t s_full[2], p_empty[2], ds_full[2][2];
  uint64_t slot_empty[3];              // a write-back's slot consumed
  uint64_t kv_ready;                   // a unit's K and V in TMEM
  uint64_t acc_full[2], acc_empty[2];  // accumulators final / read out
  uint64_t mma_done[2];                // per issuing warp
  uint32_t tmem_base;
  int abort;
};

// warps: elementwise warps that arrive on the barriers of a step (each once); k_readers:
// arrivals that free a K stage.
__device__ __forceinline__ void swa_init_bars(SwaBars &bar, int warps, int k_readers) {
  for (int s = 0; s < 4; ++s) {
    mbar_init(&bar.q_full[s], 1);
    mbar_init(&bar.q_empty[s], 1);
  }
  for (int s = 0; s < 5; ++s) {
    mbar_init(&bar.k_full[s], 1);
    mbar_init(&bar.k_empty[s], k_readers);
    mbar_init(&bar.v_full[s], 1);
    mbar_init(&bar.v_empty[s], 1);
  }
  for (int x = 0; x < 2; ++x) {
    mbar_init(&bar.s_full[x], 1);
    mbar_init(&bar.p_empty[x], warps);
    mbar_init(&bar.ds_full[x][0], warps);
    mbar_init(&bar.ds_full[x][1], warps);
    mbar_init(&bar.acc_full[x], 1);
    mbar_init(&bar.acc_empty[x], 16);
  }
  for (int x = 0; x < 3; ++x) mbar_init(&bar.slot_empty[x], 1);
  mbar_init(&bar.kv_ready, 16);
  mbar_init(&bar.mma_done[0], 1);
  mbar_init(&bar.mma_done[1], 1);
  bar.abort = 0;
  fence_barrier_init();
}

template <int D>
__global__ void __launch_bounds__(kSwaBwdThreads, 1)
swa_bwd_dq_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmQ1,
                  const __grid_constant__ CUtensorMap tmG, const __grid_constant__ CUtensorMap tmG1,
                  const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmK1,
                  const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmV1,
                  const SwaBwdParams p) {
  using C = SwaDqCfg<D>;
  using T = SwaTile<D>;
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  unsigned char *sbase = smem_raw + (base - raw);
  SwaBars &bar = *reinterpret_cast<SwaBars *>(sbase + C::BAR_OFF);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int site0 = (40 * 16 + (D == 64 ? 0 : (D == 80 ? 1 : 2))) * 256;
  constexpr uint32_t FULL = 0xffffffffu;
  const int nitems = p.batch * p.hq * p.nt;

  if (tid == 0) swa_init_bars(bar, 16, 1);
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmG);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (warp == 1) {
    tmem_alloc(&bar.tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(FULL, bar.tmem_base, 0);   // (uniform)
  volatile int *abort = &bar.abort;

  if (warp == 0) {
    // ------------------------------------------------------------ V and K
    uint32_t nv = 0, nk = 0;                        // issued
    bool ok = true;
    for (int u = blockIdx.x; ok && u < nitems; u += gridDim.x) {
      const SwaDqItem w = swa_dq_item(p, u);
      for (int m = 0; m < w.nc; ++m) {
        const uint32_t vs = nv % C::NV, ks = nk % C::NK;
        if (!(ok = mbar_wait_warp(&bar.v_empty[vs], ((nv / C::NV) & 1) ^ 1, abort, p.status, site0 + 1))) break;
        if (elect_one()) {
          mbar_arrive_expect_tx(&bar.v_full[vs], T::BYTES);
          swa_load_tile<D>(sbase + C::V_OFF + vs * T::TILE, &tmV, &tmV1, &bar.v_full[vs], swa_dq_key(w, m), w.hk, w.b);
        }
        __syncwarp();
        ++nv;
        if (!(ok = mbar_wait_warp(&bar.k_empty[ks], ((nk / C::NK) & 1) ^ 1, abort, p.status, site0 + 1))) break;
        if (elect_one()) {
          mbar_arrive_expect_tx(&bar.k_full[ks], T::BYTES);
          swa_load_tile<D>(sbase + C::K_OFF + ks * T::TILE, &tmK, &tmK1, &bar.k_full[ks], swa_dq_key(w, m), w.hk, w.b);
        }
        __syncwarp();
        ++nk;
      }
    }
    drain_ring(bar.v_full, nv, C::NV, p.status);
    drain_ring(bar.k_full, nk, C::NK, p.status);
  } else if (warp == 3) {
    // ------------------------------------------------------------ Q and dO
    uint32_t cnt = 0;
    for (int u = blockIdx.x; u < nitems; u += gridDim.x, ++cnt) {
      const SwaDqItem w = swa_dq_item(p, u);
      const uint32_t st = cnt % C::QS;
      if (!mbar_wait_warp(&bar.q_empty[st], ((cnt / C::QS) & 1) ^ 1, abort, p.status, site0 + 2)) break;
      if (elect_one()) {
        mbar_arrive_expect_tx(&bar.q_full[st], 2 * T::BYTES);
        swa_load_tile<D>(sbase + C::Q_OFF + st * T::TILE, &tmQ, &tmQ1, &bar.q_full[st], w.qt * kTileRows, w.h, w.b);
        swa_load_tile<D>(sbase + C::DO_OFF + st * T::TILE, &tmG, &tmG1, &bar.q_full[st], w.qt * kTileRows, w.h, w.b);
      }
      __syncwarp();
    }
    drain_ring(bar.q_full, cnt, C::QS, p.status);
  } else if (warp == 1) {
    // ------------------------------------------------------------ S and dP
    // Of each chunk, as soon as the last chunk's have been read into registers.
    uint32_t step = 0, qn = 0;
    bool ok = true;
    for (int u = blockIdx.x; ok && u < nitems; u += gridDim.x, ++qn) {
      const SwaDqItem w = swa_dq_item(p, u);
      const uint32_t qs = qn % C::QS;
      if (!(ok = mbar_wait_warp(&bar.q_full[qs], (qn / C::QS) & 1, abort, p.status, site0 + 3))) break;
      for (int m = 0; m < w.nc; ++m, ++step) {
        const uint32_t vs = step % C::NV, ks = step % C::NK;
        if (!(ok = mbar_wait_warp(&bar.k_full[ks], (step / C::NK) & 1, abort, p.status, site0 + 4))) break;
        if (!(ok = mbar_wait_warp(&bar.v_full[vs], (step / C::NV) & 1, abort, p.status, site0 + 5))) break;
        if (!(ok = mbar_wait_warp(&bar.p_empty[0], (step & 1) ^ 1, abort, p.status, site0 + 10))) break;
        tc_fence_after();
        if (elect_one()) {
          swa_scores<D, 128>(tmem, base + C::Q_OFF + qs * T::TILE, base + C::K_OFF + ks * T::TILE, 0);
          swa_scores<D, 128>(tmem + C::P0, base + C::DO_OFF + qs * T::TILE, base + C::V_OFF + vs * T::TILE, 0);
          umma_commit(&bar.s_full[0]);
          umma_commit(&bar.v_empty[vs]);
          if (m == w.nc - 1) umma_commit(&bar.q_empty[qs]);
        }
        __syncwarp();
      }
    }
    swa_issued(&bar.mma_done[0], p.status);
  } else if (warp == 2) {
    // ------------------------------------------------------------ dQ += dS K
    const bool mute = swa_take_fault(p.status, 1);
    uint32_t step = 0, an = 0;
    bool ok = true;
    for (int u = blockIdx.x; ok && u < nitems; u += gridDim.x, ++an) {
      const SwaDqItem w = swa_dq_item(p, u);
      for (int m = 0; m < w.nc; ++m, ++step) {
        const uint32_t ks = step % C::NK;
        if (!(ok = mbar_wait_warp(&bar.ds_full[0][step & 1], (step >> 1) & 1, abort, p.status, site0 + 6))) break;
        if (m == 0 && !(ok = mbar_wait_warp(&bar.acc_empty[0], (an & 1) ^ 1, abort, p.status, site0 + 7))) break;
        tc_fence_after();
        if (elect_one()) {
          const uint32_t kt = base + C::K_OFF + ks * T::TILE, tS = tmem + C::DS0 + 64 * (step & 1);
          swa_acc<D>(tmem + C::ACC, tS, kt, 0, m == 0);
          swa_acc<D>(tmem + C::ACC, tS + 32, kt, 1, false);
          if (!mute || step > 0) {
            umma_commit(&bar.slot_empty[step & 1]);
            umma_commit(&bar.k_empty[ks]);
            if (m == w.nc - 1) umma_commit(&bar.acc_full[0]);
          }
        }
        __syncwarp();
      }
    }
    swa_issued(&bar.mma_done[1], p.status);
  } else {
    // ------------------------------------------------------------ dS, and dQ out
    // Group grp takes the columns [32 grp, 32 grp + 32) of S and dP.  An item's dQ is read
    // out behind the first chunk of the next item, when its last product is long done.
    const int q4 = warp & 3, grp = (warp - 4) >> 2;
    const int r = 32 * q4 + lane;                   // row == TMEM lane
    const uint32_t lane_off = (uint32_t)(32 * q4) << 16;
    const uint32_t tS = tmem + lane_off + 32 * grp, tP = tS + C::P0;
    const float sl2 = p.scale_log2;
    uint32_t sc = 0, an = 0;
    bool ok = true;
    uint16_t *dst = nullptr;                        // the last item's row of dQ
    bool live = false, pend = false;
    auto read_out = [&]() {
      if (!mbar_wait_warp(&bar.acc_full[0], an & 1, abort, p.status, site0 + 9)) return false;
      ++an;
      tc_fence_after();
      // A lane's 16 columns are one whole 32-byte sector of its row.
#pragma unroll
      for (int c = 0; c < D; c += 16) {
        if ((c / 16 & 3) != grp) continue;
        uint32_t o[16];
        tmem_ld16(tmem + lane_off + C::ACC + c, o);
        tmem_wait_ld();
        if (live) store16(dst + c, o, p.scale);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.acc_empty[0]);
      return true;
    };
    for (int u = blockIdx.x; ok && u < nitems; u += gridDim.x) {
      const SwaDqItem w = swa_dq_item(p, u);
      const int i0 = w.qt * kTileRows, i = i0 + r;
      const float *st = p.stat + (((int64_t)w.b * p.hq + w.h) * p.nt + w.qt) * 256 + r;
      const float nl = st[0], nd = st[128];
      for (int m = 0; m < w.nc; ++m, ++sc) {
        if (!(ok = mbar_wait_warp(&bar.s_full[0], sc & 1, abort, p.status, site0 + 8))) break;
        tc_fence_after();
        const int key0 = swa_dq_key(w, m) + 32 * grp;
        const bool full = key0 + 31 <= i0 && (i0 + kTileRows - 1 - key0 < p.window || key0 + 32 <= p.sink);
        uint32_t sv[32], pv[32];
        tmem_ld32(tS, sv);
        tmem_ld32(tP, pv);
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.p_empty[0]);
        // The dS slot's last product is done (it was issued a step ago; the S issuer waiting
        // for it instead delays the next products: 2135 cycles a tile, not 1892).
        if (!(ok = mbar_wait_warp(&bar.slot_empty[sc & 1], ((sc >> 1) & 1) ^ 1, abort, p.status, site0 + 11))) break;
        uint32_t ds[16];
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          float x0, x1, d0, d1;
          fma2(x0, x1, __uint_as_float(sv[e]), __uint_as_float(sv[e + 1]), sl2, nl, nl);
          addmul2(d0, d1, __uint_as_float(pv[e]), __uint_as_float(pv[e + 1]), nd, nd, ex2_approx(x0), ex2_approx(x1));
          ds[e / 2] = pack_bf16x2(d0, d1);
        }
        if (!full) {
          // Keys that the row does not see: zero halves of the packed pairs.
          const uint32_t b = first_bits(i + 1 - key0) & (~first_bits(i + 1 - p.window - key0) | first_bits(p.sink - key0));
#pragma unroll
          for (int e = 0; e < 32; e += 2) ds[e / 2] &= pair_mask(b, e);
        }
        tmem_st16(tmem + lane_off + C::DS0 + 64 * (sc & 1) + 16 * grp, ds);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.ds_full[0][sc & 1]);
        if (pend) {
          pend = false;
          if (!(ok = read_out())) break;
        }
      }
      if (!ok) break;
      dst = p.dq + (int64_t)w.b * p.dq_sb + (int64_t)w.h * p.dq_sh + (int64_t)i * p.dq_sn;
      live = i < p.N;
      pend = true;
    }
    if (ok && pend) read_out();
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------ dK / dV

// Unit u: first the far parts of the sinks' key tiles (the longest walks), then every key
// tile's band.  Its walk: entries t0 .. t1 - 1 of the list of `len` query tiles from `first`
// on, head after head.
struct SwaDkvUnit {
  int b, hk, kt;
  int first, len, t0, t1;
  int part;        // -1: the gradients themselves; else the part they are a sum of
};

__device__ __forceinline__ int swa_dkv_units(const SwaBwdParams &p) {
  return p.batch * p.hkv * (p.nst * p.nseg + p.nt);
}

__device__ __forceinline__ bool swa_dkv_unit(const SwaBwdParams &p, int u, SwaDkvUnit &w) {
  const int heads = p.batch * p.hkv, nfar = heads * p.nst * p.nseg;
  int seg = -1;
  if (u < nfar) {
    seg = u / (heads * p.nst);
    const int rest = u - seg * heads * p.nst;
    w.kt = rest / heads;
    u = rest - w.kt * heads;
  } else {
    u -= nfar;
    w.kt = u / heads;
    u -= w.kt * heads;
  }
  w.b = u / p.hkv;
  w.hk = u - w.b * p.hkv;
  const int last = swa_last_tile(w.kt, p.window, p.nt);
  const int far = p.nt - 1 - last;
  if (seg >= 0) {
    w.first = last + 1;
    w.len = far;
    w.t0 = seg * p.seg;
    w.t1 = min(w.t0 + p.seg, p.G * far);
    w.part = 1 + seg;
  } else {
    w.first = w.kt;
    w.len = last - w.kt + 1;
    w.t0 = 0;
    w.t1 = p.G * w.len;
    w.part = (w.kt < p.nst && far > 0) ? 0 : -1;
  }
  return w.t0 < w.t1;
}

// TMEM of the dK / dV kernel: the halves' S in a ring of slots of 64 columns (P and dS are
// written back over them), their dP in one slot (a half is read into registers before the
// next one's products), the accumulators, and left operands of the products: from shared
// memory a 64-column product takes 48 cycles instead of 32, and the loads of the query tiles
// compete for the same bandwidth.  D = 64, 80: K, V and the blocks of ones (2708 -> 2502
// cycles a tile at D = 80), and three S slots (two: 147 against 133 us at 32 heads, 4096
// tokens, window 2048).  D = 128: the accumulators' 256 columns leave
// room for K and two slots (two dP slots in its place: 913 against 868 us at 16 heads over 4,
// 16384 tokens, window 4096).
template <int D>
struct SwaTmem {
  static constexpr bool VT = D != 128;                      // V (and the ones) in TMEM
  static constexpr int S = VT ? 3 : 2;
  static constexpr uint32_t P0 = 64 * S, ACC = 64 * (S + 1), K = ACC + 2 * D, V = K + D / 2, ONE = V + D / 2;
  static_assert((VT ? ONE + 16 : V) <= 512, "TMEM columns");
  static __device__ __forceinline__ uint32_t s_at(uint32_t h) { return 64 * (h % S); }
};

template <int D>
struct SwaDkvCfg {
  static constexpr int KS = D == 128 ? 1 : 2;                  // K / V stages
  static constexpr int QS = D == 128 ? 2 : (D == 80 ? 3 : 4);  // Q / dO / statistics stages
  static constexpr int K_OFF = 0;
  static constexpr int V_OFF = KS * SwaTile<D>::TILE;
  static constexpr int Q_OFF = 2 * KS * SwaTile<D>::TILE;
  static constexpr int DO_OFF = Q_OFF + QS * SwaTile<D>::TILE;
  static constexpr int EX_OFF = DO_OFF + QS * SwaTile<D>::TILE;   // a stage's statistics columns
  static constexpr int ONE_OFF = EX_OFF + QS * kSwaExtra;         // ones: lse's columns, D's
  using M = SwaTmem<D>;
  static constexpr int BAR_OFF = ONE_OFF + (M::VT ? 0 : 2 * kSwaExtra);
  static constexpr int SMEM = BAR_OFF + 1024 + 1024;
  static_assert(SMEM <= 232448, "shared memory of a CTA");
};

template <int D>
__global__ void __launch_bounds__(kSwaBwdThreads, 1)
swa_bwd_dkdv_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmQ1,
                    const __grid_constant__ CUtensorMap tmG, const __grid_constant__ CUtensorMap tmG1,
                    const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmK1,
                    const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmV1,
                    const SwaBwdParams p) {
  using C = SwaDkvCfg<D>;
  using T = SwaTile<D>;
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  unsigned char *sbase = smem_raw + (base - raw);
  SwaBars &bar = *reinterpret_cast<SwaBars *>(sbase + C::BAR_OFF);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int site0 = (41 * 16 + (D == 64 ? 0 : (D == 80 ? 1 : 2))) * 256;
  constexpr uint32_t FULL = 0xffffffffu;
  const int nunits = swa_dkv_units(p);

  using M = typename C::M;
  if (tid == 0) swa_init_bars(bar, 8, M::VT ? 16 : 17);   // (every elementwise warp; V's last product)
  // The blocks of ones: columns 0 - 2 (lse) and 3 - 5 (D).
  for (int r = tid; !M::VT && r < 2 * 128; r += kSwaBwdThreads) {
    unsigned char *blk = sbase + C::ONE_OFF + (r >> 7) * kSwaExtra;
    const uint4 ones = r < 128 ? make_uint4(0x3F803F80u, 0x00003F80u, 0u, 0u) : make_uint4(0u, 0x3F800000u, 0x3F803F80u, 0u);
    *reinterpret_cast<uint4 *>(blk + extra_offset(r & 127, 0)) = ones;
    *reinterpret_cast<uint4 *>(blk + extra_offset(r & 127, 1)) = make_uint4(0u, 0u, 0u, 0u);
  }
  fence_proxy_async_smem();
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmG);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (warp == 1) {
    tmem_alloc(&bar.tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(FULL, bar.tmem_base, 0);   // (uniform)
  volatile int *abort = &bar.abort;

  if (warp == 0) {
    // ------------------------------------------------------------ K and V
    uint32_t cnt = 0;
    for (int u = blockIdx.x; u < nunits; u += gridDim.x) {
      SwaDkvUnit w;
      if (!swa_dkv_unit(p, u, w)) continue;
      const uint32_t st = cnt % C::KS;
      if (!mbar_wait_warp(&bar.k_empty[st], ((cnt / C::KS) & 1) ^ 1, abort, p.status, site0 + 1)) break;
      if (elect_one()) {
        mbar_arrive_expect_tx(&bar.k_full[st], 2 * T::BYTES);
        swa_load_tile<D>(sbase + C::K_OFF + st * T::TILE, &tmK, &tmK1, &bar.k_full[st], w.kt * kTileKeys, w.hk, w.b);
        swa_load_tile<D>(sbase + C::V_OFF + st * T::TILE, &tmV, &tmV1, &bar.k_full[st], w.kt * kTileKeys, w.hk, w.b);
      }
      __syncwarp();
      ++cnt;
    }
    drain_ring(bar.k_full, cnt, C::KS, p.status);
  } else if (warp == 3) {
    // ------------------------------------------------------------ Q, dO, row statistics
    uint32_t cnt = 0;
    bool ok = true;
    for (int u = blockIdx.x; ok && u < nunits; u += gridDim.x) {
      SwaDkvUnit w;
      if (!swa_dkv_unit(p, u, w)) continue;
      int g = w.t0 / w.len, qt = w.first + w.t0 % w.len;
      for (int t = w.t0; t < w.t1; ++t, ++cnt) {
        const uint32_t st = cnt % C::QS;
        if (!(ok = mbar_wait_warp(&bar.q_empty[st], ((cnt / C::QS) & 1) ^ 1, abort, p.status, site0 + 2))) break;
        if (elect_one()) {
          const int h = w.hk * p.G + g;
          mbar_arrive_expect_tx(&bar.q_full[st], 2 * T::BYTES + kSwaExtra);
          swa_load_tile<D>(sbase + C::Q_OFF + st * T::TILE, &tmQ, &tmQ1, &bar.q_full[st], qt * kTileRows, h, w.b);
          swa_load_tile<D>(sbase + C::DO_OFF + st * T::TILE, &tmG, &tmG1, &bar.q_full[st], qt * kTileRows, h, w.b);
          bulk_load(sbase + C::EX_OFF + st * kSwaExtra,
                    p.extra + (((int64_t)w.b * p.hq + h) * p.nt + qt) * (kSwaExtra / 2), kSwaExtra, &bar.q_full[st]);
        }
        __syncwarp();
        if (++qt == w.first + w.len) {
          qt = w.first;
          ++g;
        }
      }
    }
    drain_ring(bar.q_full, cnt, C::QS, p.status);
  } else if (warp == 1) {
    // ------------------------------------------------------------ S^T and dP^T
    // Per query tile and half x: S^T as soon as the S slot's write-back has been consumed,
    // dP^T as soon as its slot has been read into registers.
    uint32_t step = 0, kn = 0;
    bool ok = true;
    for (int u = blockIdx.x; ok && u < nunits; u += gridDim.x) {
      SwaDkvUnit w;
      if (!swa_dkv_unit(p, u, w)) continue;
      const uint32_t ks = kn % C::KS;
      if (!(ok = mbar_wait_warp(&bar.kv_ready, kn & 1, abort, p.status, site0 + 3))) break;
      ++kn;
      const uint32_t vt = base + C::V_OFF + ks * T::TILE;
      for (int t = w.t0; ok && t < w.t1; ++t, ++step) {
        const uint32_t st = step % C::QS, ex = base + C::EX_OFF + st * kSwaExtra;
        if (!(ok = mbar_wait_warp(&bar.q_full[st], (step / C::QS) & 1, abort, p.status, site0 + 4))) break;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint32_t h = 2 * step + x;
          if (!(ok = mbar_wait_warp(&bar.slot_empty[h % M::S], ((h / M::S) & 1) ^ 1, abort, p.status, site0 + 11))) break;
          const uint32_t qt = base + C::Q_OFF + st * T::TILE, gt = base + C::DO_OFF + st * T::TILE;
          tc_fence_after();
          if (elect_one()) {
            swa_scores_tmem<D, 64>(tmem + M::s_at(h), tmem + M::K, qt, 64 * x);
            if constexpr (M::VT) swa_extra_tmem<64>(tmem + M::s_at(h), tmem + M::ONE, 64 * x, ex);
            else swa_extra<64>(tmem + M::s_at(h), base + C::ONE_OFF, 64 * x, ex);
          }
          __syncwarp();
          if (!(ok = mbar_wait_warp(&bar.p_empty[0], (h & 1) ^ 1, abort, p.status, site0 + 10))) break;
          tc_fence_after();
          if (elect_one()) {
            if constexpr (M::VT) {
              swa_scores_tmem<D, 64>(tmem + M::P0, tmem + M::V, gt, 64 * x);
              swa_extra_tmem<64>(tmem + M::P0, tmem + M::ONE + 8, 64 * x, ex);
            } else {
              swa_scores<D, 64>(tmem + M::P0, vt, gt, 64 * x);
              swa_extra<64>(tmem + M::P0, base + C::ONE_OFF + kSwaExtra, 64 * x, ex);
            }
            umma_commit(&bar.s_full[x]);
            if (!M::VT && x == 1 && t == w.t1 - 1) umma_commit(&bar.k_empty[ks]);
          }
          __syncwarp();
        }
      }
    }
    swa_issued(&bar.mma_done[0], p.status);
  } else if (warp == 2) {
    // ------------------------------------------------------------ dV += P^T dO, dK += dS^T Q
    const bool mute = swa_take_fault(p.status, 2);
    const uint32_t tK = tmem + M::ACC, tV = tK + D;
    uint32_t step = 0, an = 0;
    bool ok = true;
    for (int u = blockIdx.x; ok && u < nunits; u += gridDim.x) {
      SwaDkvUnit w;
      if (!swa_dkv_unit(p, u, w)) continue;
      for (int t = w.t0; ok && t < w.t1; ++t, ++step) {
        const uint32_t st = step % C::QS;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint32_t h = 2 * step + x;
          if (!(ok = mbar_wait_warp(&bar.ds_full[x][step & 1], (step >> 1) & 1, abort, p.status, site0 + 5))) break;
          if (x == 0 && t == w.t0) {
            if (!(ok = mbar_wait_warp(&bar.acc_empty[0], (an & 1) ^ 1, abort, p.status, site0 + 6))) break;
            ++an;
          }
          tc_fence_after();
          if (elect_one()) {
            const uint32_t qp = base + C::Q_OFF + st * T::TILE, gp = base + C::DO_OFF + st * T::TILE;
            const uint32_t tS = tmem + M::s_at(h);   // of 32 queries: P^T, then dS^T
            swa_acc<D, 16>(tV, tS, gp, x, x == 0 && t == w.t0);
            swa_acc<D, 16>(tK, tS + 16, qp, x, x == 0 && t == w.t0);
            if (!mute || step > 0) {
              umma_commit(&bar.slot_empty[h % M::S]);
              if (x == 1) {
                umma_commit(&bar.q_empty[st]);
                if (t == w.t1 - 1) umma_commit(&bar.acc_full[0]);
              }
            }
          }
          __syncwarp();
        }
      }
    }
    swa_issued(&bar.mma_done[1], p.status);
  } else {
    // ------------------------------------------------------------ P^T, dS^T; dK, dV out
    const int q4 = warp & 3, grp = (warp - 4) >> 2;
    const int r = 32 * q4 + lane;                   // key of the tile == TMEM lane
    const uint32_t lane_off = (uint32_t)(32 * q4) << 16;
    const int x = grp >> 1, sub = 32 * (grp & 1);   // half of the tile, its first column there
    const uint32_t tK = tmem + lane_off + M::ACC, tV = tK + D;
    const float sl2 = p.scale_log2;
    uint32_t sc = 0, an = 0;
    bool ok = true;
    SwaDkvUnit nw;
    auto seek = [&](int v) {
      while (v < nunits && !swa_dkv_unit(p, v, nw)) v += gridDim.x;
      return v;
    };
    uint32_t kn = 0;
    // A unit's K (groups 0, 1) and V (2, 3; D = 128: K alone, by all) from shared memory into
    // TMEM, 16 values of a row in turn to a group, once the last unit's products have read
    // what was there.
    auto stage_kv = [&]() {
      const uint32_t ks = kn % C::KS;
      if (sc > 0 && !mbar_wait_warp(&bar.s_full[1], (sc - 1) & 1, abort, p.status, site0 + 12)) return false;
      if (!mbar_wait_warp(&bar.k_full[ks], (kn / C::KS) & 1, abort, p.status, site0 + 13)) return false;
      tc_fence_after();
      const bool isv = M::VT && x == 1;
      const unsigned char *tile = sbase + (isv ? C::V_OFF : C::K_OFF) + ks * T::TILE;
#pragma unroll
      for (int j = 0; j < D / 16; ++j) {
        if (M::VT ? (j & 1) != (grp & 1) : (j & 3) != grp) continue;
        uint32_t v[8];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int c = 2 * j + e;
          const uint4 a = *reinterpret_cast<const uint4 *>(
              c < 8 ? tile + r * 128 + ((c ^ (r & 7)) << 4)
              : D == 128 ? tile + T::R0 + r * 128 + (((c - 8) ^ (r & 7)) << 4)
                         : tile + T::R0 + r * 32 + (((c - 8) ^ ((r >> 2) & 1)) << 4));
          v[4 * e] = a.x;
          v[4 * e + 1] = a.y;
          v[4 * e + 2] = a.z;
          v[4 * e + 3] = a.w;
        }
        tmem_st8(tmem + lane_off + (isv ? M::V : M::K) + 8 * j, v);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&bar.k_empty[ks]);
        mbar_arrive(&bar.kv_ready);
      }
      ++kn;
      return true;
    };
    int u = seek(blockIdx.x);
    if constexpr (M::VT) {
      if (grp == 0) {
        const uint32_t lse1[8] = {0x3F803F80u, 0x00003F80u, 0u, 0u, 0u, 0u, 0u, 0u};
        const uint32_t d1[8] = {0u, 0x3F800000u, 0x3F803F80u, 0u, 0u, 0u, 0u, 0u};
        tmem_st8(tmem + lane_off + M::ONE, lse1);
        tmem_st8(tmem + lane_off + M::ONE + 8, d1);
      }
    }
    if (u < nunits) ok = stage_kv();
    while (ok && u < nunits) {
      const SwaDkvUnit w = nw;
      const int key0 = w.kt * kTileKeys, key = key0 + r;
      int qt = w.first + w.t0 % w.len;
      for (int t = w.t0; t < w.t1; ++t, ++sc) {
        if (!(ok = mbar_wait_warp(&bar.s_full[x], sc & 1, abort, p.status, site0 + 8))) break;
        tc_fence_after();
        const int i0 = qt * kTileRows + 64 * x + sub;   // row of the group's first column
        const bool full = key0 + kTileKeys - 1 <= i0 && (i0 + 31 - key0 < p.window || key0 + kTileKeys <= p.sink);
        if (++qt == w.first + w.len) qt = w.first;
        const uint32_t tS = tmem + lane_off + M::s_at(2 * sc + x);
        uint32_t sv[32], pv[32];
        tmem_ld32(tS + sub, sv);
        tmem_ld32(tmem + lane_off + M::P0 + sub, pv);
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.p_empty[0]);
        uint32_t pp[16], dd[16];
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          float x0, x1, d0, d1;
          mul2(x0, x1, __uint_as_float(sv[e]), __uint_as_float(sv[e + 1]), sl2, sl2);
          x0 = ex2_approx(x0);
          x1 = ex2_approx(x1);
          mul2(d0, d1, __uint_as_float(pv[e]), __uint_as_float(pv[e + 1]), x0, x1);
          pp[e / 2] = pack_bf16x2(x0, x1);
          dd[e / 2] = pack_bf16x2(d0, d1);
        }
        if (!full) {
          // Rows that do not see the key: zero halves of the packed pairs.
          const uint32_t b = ~first_bits(key - i0) & (first_bits(key + p.window - i0) | (key < p.sink ? 0xFFFFFFFFu : 0u));
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const uint32_t keep = pair_mask(b, e);
            pp[e / 2] &= keep;
            dd[e / 2] &= keep;
          }
        }
        // Over the 32 columns of scores that this group has read itself: P^T, dS^T.
        tmem_st16(tS + sub, pp);
        tmem_st16(tS + sub + 16, dd);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.ds_full[x][sc & 1]);
      }
      if (!ok) break;
      u = seek(u + gridDim.x);
      if (u < nunits && !(ok = stage_kv())) break;
      if (!(ok = mbar_wait_warp(&bar.acc_full[0], an & 1, abort, p.status, site0 + 9))) break;
      ++an;
      tc_fence_after();
      // Groups 0 and 1 write dK, groups 2 and 3 dV, every other 16 columns each.
      const bool isk = x == 0;
      const uint32_t ta = isk ? tK : tV;
      const float scl = isk ? p.scale : 1.f;
      if (w.part < 0) {
        uint16_t *dst = isk ? p.dk + (int64_t)w.b * p.dk_sb + (int64_t)w.hk * p.dk_sh + (int64_t)key * p.dk_sn
                            : p.dv + (int64_t)w.b * p.dv_sb + (int64_t)w.hk * p.dv_sh + (int64_t)key * p.dv_sn;
#pragma unroll
        for (int c = 0; c < D; c += 16) {
          if ((c / 16 & 1) != (grp & 1)) continue;
          uint32_t o[16];
          tmem_ld16(ta + c, o);
          tmem_wait_ld();
          if (key < p.N) store16(dst + c, o, scl);
        }
      } else {
        float *dst = p.part + (((((int64_t)w.b * p.hkv + w.hk) * p.nst + w.kt) * (1 + p.nseg) + w.part) * 2 + x) *
                                  (kTileKeys * D) + r * D;
#pragma unroll
        for (int c = 0; c < D; c += 16) {
          if ((c / 16 & 1) != (grp & 1)) continue;
          uint32_t o[16];
          tmem_ld16(ta + c, o);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; e += 4)
            *reinterpret_cast<uint4 *>(dst + c + e) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.acc_empty[0]);
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------ join

// dK, dV of the sinks' key tiles: part 0 (the band) and the far parts in order.  A block
// per eight rows of one tile; 4 columns a thread.
template <int D>
__global__ void __launch_bounds__(256) swa_bwd_join_kernel(const SwaBwdParams p) {
  const int tile = blockIdx.x;                       // (b, hk, kt)
  const int kt = tile % p.nst, hk = tile / p.nst % p.hkv, b = tile / p.nst / p.hkv;
  const int far = p.nt - 1 - swa_last_tile(kt, p.window, p.nt);
  if (far <= 0) return;                              // written by the band's unit
  const int parts = 1 + (p.G * far + p.seg - 1) / p.seg;
  const int side = blockIdx.z;
  for (int i = threadIdx.x; i < 8 * (D / 4); i += 256) {
    const int r = blockIdx.y * 8 + i / (D / 4), c = (i % (D / 4)) * 4;
    const int key = kt * kTileKeys + r;
    if (key >= p.N) continue;
    const float *src = p.part + ((int64_t)tile * (1 + p.nseg) * 2 + side) * (kTileKeys * D) + r * D + c;
    float a[4] = {0.f, 0.f, 0.f, 0.f};
    for (int x = 0; x < parts; ++x) {
      const float4 y = *reinterpret_cast<const float4 *>(src + (int64_t)x * 2 * kTileKeys * D);
      a[0] += y.x; a[1] += y.y; a[2] += y.z; a[3] += y.w;
    }
    const float s = side == 0 ? p.scale : 1.f;
    uint16_t *dst = side == 0 ? p.dk + (int64_t)b * p.dk_sb + (int64_t)hk * p.dk_sh + (int64_t)key * p.dk_sn
                              : p.dv + (int64_t)b * p.dv_sb + (int64_t)hk * p.dv_sh + (int64_t)key * p.dv_sn;
    *reinterpret_cast<uint2 *>(dst + c) = make_uint2(pack_bf16x2(a[0] * s, a[1] * s), pack_bf16x2(a[2] * s, a[3] * s));
  }
}

// ------------------------------------------------------------------ launch

template <int D>
static cudaError_t launch_swa_bwd_d(const CUtensorMap *m, const SwaBwdParams &p, int nsm, cudaStream_t st) {
  const int groups = (p.nt * kTileRows + RowLanes<D>::RPW - 1) / RowLanes<D>::RPW, heads = p.batch * p.hq;
  const int nb = max(1, min((groups + 7) / 8, nsm * 16 / heads));
  swa_bwd_prep_kernel<D><<<(unsigned)heads * nb, 256, 0, st>>>(p, nb);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;

  e = cudaFuncSetAttribute(swa_bwd_dq_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, SwaDqCfg<D>::SMEM);
  if (e != cudaSuccess) return e;
  const long long items = (long long)p.batch * p.hq * p.nt;
  swa_bwd_dq_kernel<D><<<(int)(items < nsm ? items : nsm), kSwaBwdThreads, SwaDqCfg<D>::SMEM, st>>>(
      m[0], m[1], m[2], m[3], m[4], m[5], m[6], m[7], p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;

  e = cudaFuncSetAttribute(swa_bwd_dkdv_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, SwaDkvCfg<D>::SMEM);
  if (e != cudaSuccess) return e;
  const long long units = (long long)p.batch * p.hkv * (p.nst * p.nseg + p.nt);
  swa_bwd_dkdv_kernel<D><<<(int)(units < nsm ? units : nsm), kSwaBwdThreads, SwaDkvCfg<D>::SMEM, st>>>(
      m[0], m[1], m[2], m[3], m[4], m[5], m[6], m[7], p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;

  if (p.nst > 0) {
    swa_bwd_join_kernel<D><<<dim3(p.batch * p.hkv * p.nst, kTileKeys / 8, 2), 256, 0, st>>>(p);
    e = cudaGetLastError();
  }
  return e;
}

// maps: Q, dO, K, V, each with its column tail (D != 64).
cudaError_t launch_swa_bwd(const CUtensorMap *maps, const SwaBwdParams &p, int nsm, cudaStream_t st) {
  switch (p.d) {
    case 64: return launch_swa_bwd_d<64>(maps, p, nsm, st);
    case 80: return launch_swa_bwd_d<80>(maps, p, nsm, st);
    case 128: return launch_swa_bwd_d<128>(maps, p, nsm, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace moba
