// swa_fwd.cu -- sliding-window attention with sinks, forward, on sm_100a tensor cores.
//
// [SWA] = "SWA + MoE: 어텐션과 희소 전문가", Bit-Axon architecture page (§"어텐션 공식",
//         §"슬라이딩 윈도우 마스크").
//
// Query row i at position p = q_off + i attends the keys j <= p with p - j < window or
// j < sink: out = softmax(scale q K^T) V over them, in one pass with a running maximum and
// sum.  A work item is a 128-row tile of one head; it walks its chunks of 128 keys, the
// sinks' before the band, then the band's.
//
// A softmax is a chain (scores to registers, maximum, exponentials, write-back, product),
// and a chain that must end before its next scores can be issued leaves both the tensor core
// and the exponential unit idle.  So a chunk is split by keys between groups of four warps
// that share nothing but the query tile: a group has its own running maximum and sum and its
// own accumulator, and the next scores are there when it has written its probabilities.  The
// partial results of a row are joined when the item is read out, behind the first chunk of
// the next item.  (The two streams of attn.cu are query tiles of 128 keys; their scores and
// accumulators fill TMEM with one buffer each.)
//   D = 64, 80  four groups of 32 keys.  A warp of 64 keys leaves the exponential unit idle
//               while it reads, finds the maximum and writes back: two groups took 793 us
//               below, four 735.
//   D = 128     two groups of 64 keys (more accumulators do not fit).  Four groups in pairs
//               that exchange their maxima took 475 against 458 us (16 heads over 4, 16384
//               tokens, window 4096), and 869 us below.
// The halves' scores stand in a ring of three slots of 64 columns: a half's next scores wait
// for the other half's last product, which keeps the halves apart, so that one reads and
// writes while the other uses the exponential unit (four slots: 112.8 against 106.5 us at
// D = 64, 8192 tokens, window 2048; 461 against 457 us at D = 128).
//
// Per 128 x 128 keys 16384 exponentials at 16 a cycle are 1024 cycles; the products are 827
// cycles at D = 80 and 1291 at D = 128, where 64-key products are fed by shared memory (48
// cycles instead of 32).  At D = 128 that is the bound, so Q goes into TMEM as the left operand
// of S: 1034 cycles (451 -> 432 us as above; at D = 64, where the softmax bounds, the copy
// costs more than it gives, 106 -> 108 us; at D = 80 TMEM is full).
// Measured (32 heads, d = 80, N = 16384, window 4096, 4 sinks): 735 us, 820 TFLOP/s at a
// power-capped 1.4-1.6 GHz, against 811 us with the two streams over query tiles; one
// 1000-token prompt (4 heads) 10.5 against 16.7 us in a graph, since a walk's chain is half
// as long.
//
//   warp 0      TMA: K and V
//   warp 1      issues S = Q K^T (TMEM owner)
//   warp 2      issues O += P V
//   warp 3      TMA: Q
//   warps 4-    the groups; a thread owns one TMEM lane, a row
// Every wait is bounded.
#include <cuda.h>
#include <cuda_bf16.h>
#include <math.h>
#include <stdint.h>

#include "common.cuh"
#include "params.h"
#include "swa_tile.cuh"

namespace moba {

constexpr float kSwaRaise = 8.f;   // the running maximum is raised when it grows by 2^8

// Work item u: one 128-row query tile and its chunks: ns of sinks from key 0, then the
// band's from chunk c0.
struct SwaItem {
  int b, h, hk, qt, ns, c0, nc;
};

__device__ __forceinline__ SwaItem swa_item(const AttnParams &p, int u) {
  const int nt = (p.N + kTileRows - 1) / kTileRows;
  SwaItem w;
  w.qt = nt - 1 - u % nt;                        // later (longer) walks first
  const int bh = u / nt;
  w.b = bh / p.hq;
  w.h = bh % p.hq;
  w.hk = w.h / p.G;
  const int first = p.q_off + w.qt * kTileRows;  // position of the first row, of the last:
  const int last = p.q_off + min(p.N, (w.qt + 1) * kTileRows) - 1;
  w.c0 = max(0, first - p.window + 1) / kTileKeys;
  w.ns = min((p.sink + kTileKeys - 1) / kTileKeys, w.c0);
  w.nc = w.ns + last / kTileKeys - w.c0 + 1;
  return w;
}

__device__ __forceinline__ int swa_key(const SwaItem &w, int m) {
  return (m < w.ns ? m : w.c0 + m - w.ns) * kTileKeys;
}

template <int D>
struct SwaFwdCfg {
  static constexpr int GRP = D == 128 ? 2 : 4;                 // softmax groups
  static constexpr int W = 128 / GRP;                          // keys of a group
  static constexpr int THREADS = 128 + 128 * GRP;
  static constexpr int QS = 2;                                 // Q stages
  static constexpr int NK = D == 128 ? 2 : 4;                  // K and V stages
  static constexpr int NV = D == 128 ? 2 : 4;
  static constexpr int Q_OFF = 0;
  static constexpr int K_OFF = QS * SwaTile<D>::TILE;
  static constexpr int V_OFF = K_OFF + NK * SwaTile<D>::TILE;
  static constexpr int ML_OFF = V_OFF + NV * SwaTile<D>::TILE; // [item parity][group][128] (m, l)
  static constexpr int BAR_OFF = ML_OFF + 2 * GRP * 128 * 8;
  static constexpr int SMEM = BAR_OFF + 1024 + 1024;
  static_assert(SMEM <= 232448, "shared memory of a CTA");
  // TMEM: a ring of 64-column slots for the halves' scores (P is written back over them),
  // then the groups' accumulators.
  static constexpr int S = 3;
  static constexpr uint32_t O = 64 * S;
  static constexpr bool QT = D == 128;                         // Q in TMEM as a left operand
  static constexpr uint32_t Q = O + GRP * D;
  static_assert(Q + (QT ? D / 2 : 0) <= 512, "TMEM columns");
  static __device__ __forceinline__ uint32_t s_at(uint32_t h) { return 64 * (h % S); }
};

struct SwaFwdBars {
  uint64_t q_full[2], q_empty[2], k_full[4], k_empty[4], v_full[4], v_empty[4];
  uint64_t s_full[2][2], p_full[2][2], pv_done[2][2];   // per half, of even and odd chunks
  uint64_t o_full, o_empty, ml_full, qt_full;
  uint64_t mma_done[2];
  uint32_t tmem_base;
  int abort;
};

template <int D>
__global__ void __launch_bounds__(SwaFwdCfg<D>::THREADS, 1)
swa_fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmQ1,
               const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmK1,
               const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmV1,
               const AttnParams p) {
  using C = SwaFwdCfg<D>;
  using T = SwaTile<D>;
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  unsigned char *sbase = smem_raw + (base - raw);
  SwaFwdBars &bar = *reinterpret_cast<SwaFwdBars *>(sbase + C::BAR_OFF);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int site0 = (42 * 16 + (D == 64 ? 0 : (D == 80 ? 1 : 2))) * 256;
  constexpr uint32_t FULL = 0xffffffffu;
  const int nitems = p.ntiles;

  if (tid == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bar.q_full[s], 1);
      mbar_init(&bar.q_empty[s], C::QT ? 2 * C::GRP : 1);
    }
    for (int s = 0; s < 4; ++s) {
      mbar_init(&bar.k_full[s], 1);
      mbar_init(&bar.k_empty[s], 1);
      mbar_init(&bar.v_full[s], 1);
      mbar_init(&bar.v_empty[s], 1);
    }
    for (int x = 0; x < 2; ++x)
      for (int s = 0; s < 2; ++s) {
        mbar_init(&bar.s_full[x][s], 1);
        mbar_init(&bar.p_full[x][s], 2 * C::GRP);   // (a warp arrives once)
        mbar_init(&bar.pv_done[x][s], 1);
      }
    mbar_init(&bar.o_full, 1);
    mbar_init(&bar.qt_full, 2 * C::GRP);
    mbar_init(&bar.o_empty, 4 * C::GRP);
    mbar_init(&bar.ml_full, 4 * C::GRP);
    mbar_init(&bar.mma_done[0], 1);
    mbar_init(&bar.mma_done[1], 1);
    bar.abort = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmQ);
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
    uint32_t nk = 0, nv = 0;                        // issued
    bool ok = true;
    for (int u = blockIdx.x; ok && u < nitems; u += gridDim.x) {
      const SwaItem w = swa_item(p, u);
      for (int m = 0; m < w.nc; ++m) {
        const uint32_t ks = nk % C::NK, vs = nv % C::NV;
        if (!(ok = mbar_wait_warp(&bar.k_empty[ks], ((nk / C::NK) & 1) ^ 1, abort, p.status, site0 + 1))) break;
        if (elect_one()) {
          mbar_arrive_expect_tx(&bar.k_full[ks], T::BYTES);
          swa_load_tile<D>(sbase + C::K_OFF + ks * T::TILE, &tmK, &tmK1, &bar.k_full[ks], swa_key(w, m), w.hk, w.b);
        }
        __syncwarp();
        ++nk;
        if (!(ok = mbar_wait_warp(&bar.v_empty[vs], ((nv / C::NV) & 1) ^ 1, abort, p.status, site0 + 1))) break;
        if (elect_one()) {
          mbar_arrive_expect_tx(&bar.v_full[vs], T::BYTES);
          swa_load_tile<D>(sbase + C::V_OFF + vs * T::TILE, &tmV, &tmV1, &bar.v_full[vs], swa_key(w, m), w.hk, w.b);
        }
        __syncwarp();
        ++nv;
      }
    }
    drain_ring(bar.k_full, nk, C::NK, p.status);
    drain_ring(bar.v_full, nv, C::NV, p.status);
  } else if (warp == 3) {
    // ------------------------------------------------------------ Q
    uint32_t cnt = 0;
    for (int u = blockIdx.x; u < nitems; u += gridDim.x, ++cnt) {
      const SwaItem w = swa_item(p, u);
      const uint32_t st = cnt % C::QS;
      if (!mbar_wait_warp(&bar.q_empty[st], ((cnt / C::QS) & 1) ^ 1, abort, p.status, site0 + 2)) break;
      if (elect_one()) {
        mbar_arrive_expect_tx(&bar.q_full[st], T::BYTES);
        swa_load_tile<D>(sbase + C::Q_OFF + st * T::TILE, &tmQ, &tmQ1, &bar.q_full[st], w.qt * kTileRows, w.h, w.b);
      }
      __syncwarp();
    }
    drain_ring(bar.q_full, cnt, C::QS, p.status);
  } else if (warp == 1) {
    // ------------------------------------------------------------ S
    // Of each half chunk, once its slot's last probabilities have been consumed.
    uint32_t step = 0, qn = 0;
    bool ok = true;
    for (int u = blockIdx.x; ok && u < nitems; u += gridDim.x, ++qn) {
      const SwaItem w = swa_item(p, u);
      const uint32_t qs = qn % C::QS, qt = base + C::Q_OFF + qs * T::TILE;
      ok = C::QT ? mbar_wait_warp(&bar.qt_full, qn & 1, abort, p.status, site0 + 3)
                 : mbar_wait_warp(&bar.q_full[qs], (qn / C::QS) & 1, abort, p.status, site0 + 3);
      if (!ok) break;
      for (int m = 0; ok && m < w.nc; ++m, ++step) {
        const uint32_t ks = step % C::NK, kt = base + C::K_OFF + ks * T::TILE;
        if (!(ok = mbar_wait_warp(&bar.k_full[ks], (step / C::NK) & 1, abort, p.status, site0 + 4))) break;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          // The half that had the slot before, h - S: its chunk and half.
          const uint32_t h = 2 * step + x, chunk = (h - C::S) >> 1;
          if (h >= C::S && !(ok = mbar_wait_warp(&bar.pv_done[(h - C::S) & 1][chunk & 1], (chunk >> 1) & 1, abort,
                                                 p.status, site0 + 5)))
            break;
          tc_fence_after();
          if (elect_one()) {
            if constexpr (C::QT) swa_scores_tmem<D, 64>(tmem + C::s_at(h), tmem + C::Q, kt, 64 * x);
            else swa_scores<D, 64>(tmem + C::s_at(h), qt, kt, 64 * x);
            umma_commit(&bar.s_full[x][step & 1]);
            if (x == 1) {
              umma_commit(&bar.k_empty[ks]);
              if (!C::QT && m == w.nc - 1) umma_commit(&bar.q_empty[qs]);
            }
          }
          __syncwarp();
        }
      }
    }
    swa_issued(&bar.mma_done[0], p.status);
  } else if (warp == 2) {
    // ------------------------------------------------------------ O += P V
    const bool mute = swa_take_fault(p.status, 1);
    uint32_t step = 0, an = 0;
    bool ok = true;
    for (int u = blockIdx.x; ok && u < nitems; u += gridDim.x, ++an) {
      const SwaItem w = swa_item(p, u);
      for (int m = 0; ok && m < w.nc; ++m, ++step) {
        const uint32_t vs = step % C::NV, vt = base + C::V_OFF + vs * T::TILE, sl = step & 1;
        if (!(ok = mbar_wait_warp(&bar.v_full[vs], (step / C::NV) & 1, abort, p.status, site0 + 6))) break;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if (!(ok = mbar_wait_warp(&bar.p_full[x][sl], (step >> 1) & 1, abort, p.status, site0 + 7))) break;
          if (m == 0 && x == 0 && !(ok = mbar_wait_warp(&bar.o_empty, (an & 1) ^ 1, abort, p.status, site0 + 8))) break;
          tc_fence_after();
          if (elect_one()) {
            const uint32_t tP = tmem + C::s_at(2 * step + x);
            if constexpr (C::GRP == 2) {
              swa_acc<D>(tmem + C::O + D * x, tP, vt, x, m == 0);
            } else {
              swa_acc32<D>(tmem + C::O + D * (2 * x), tP, vt, 2 * x, m == 0);
              swa_acc32<D>(tmem + C::O + D * (2 * x + 1), tP + 32, vt, 2 * x + 1, m == 0);
            }
            if (!mute || step > 0) {
              umma_commit(&bar.pv_done[x][sl]);
              if (x == 1) {
                umma_commit(&bar.v_empty[vs]);
                if (m == w.nc - 1) umma_commit(&bar.o_full);
              }
            }
          }
          __syncwarp();
        }
      }
    }
    swa_issued(&bar.mma_done[1], p.status);
  } else {
    // ------------------------------------------------------------ softmax, and O out
    const int q4 = warp & 3, grp = (warp - 4) >> 2;
    const int x = grp * 2 / C::GRP, sub = grp * C::W - 64 * x;   // half, first column there
    const int r = 32 * q4 + lane;                   // row == TMEM lane
    const uint32_t lane_off = (uint32_t)(32 * q4) << 16;
    const uint32_t tO = tmem + lane_off + C::O, tOg = tO + D * grp;
    float2 *ml = reinterpret_cast<float2 *>(sbase + C::ML_OFF);
    const float sl2 = p.scale_log2;
    uint32_t sc = 0, an = 0;                        // chunks, items read out
    bool ok = true, pend = false, live = false;
    uint16_t *dst = nullptr;                        // the last item's row, its place in lse
    float *ldst = nullptr;
    auto read_out = [&]() {
      if (!mbar_wait_warp(&bar.ml_full, an & 1, abort, p.status, site0 + 9)) return false;
      if (!mbar_wait_warp(&bar.o_full, an & 1, abort, p.status, site0 + 10)) return false;
      tc_fence_after();
      float wgt[C::GRP], mx = -INFINITY, l = 0.f;
#pragma unroll
      for (int g = 0; g < C::GRP; ++g) mx = fmaxf(mx, ml[((an & 1) * C::GRP + g) * 128 + r].x);
      const float mu = mx == -INFINITY ? 0.f : mx;
#pragma unroll
      for (int g = 0; g < C::GRP; ++g) {
        const float2 a = ml[((an & 1) * C::GRP + g) * 128 + r];
        wgt[g] = ex2_approx(a.x - mu);
        l = fmaf(wgt[g], a.y, l);
      }
      ++an;
      const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
#pragma unroll
      for (int g = 0; g < C::GRP; ++g) wgt[g] *= inv;
#pragma unroll
      for (int c = 0; c < D; c += 16) {
        if (c / 16 % C::GRP != grp) continue;
        float o[16];
#pragma unroll
        for (int g = 0; g < C::GRP; g += 2) {
          uint32_t u[16], v[16];
          tmem_ld16(tO + D * g + c, u);
          tmem_ld16(tO + D * (g + 1) + c, v);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float t = g == 0 ? wgt[0] * __uint_as_float(u[e]) : fmaf(wgt[g], __uint_as_float(u[e]), o[e]);
            o[e] = fmaf(wgt[g + 1], __uint_as_float(v[e]), t);
          }
        }
        if (live) {                                 // one whole 32-byte sector of the row
          uint32_t u[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) u[e] = __float_as_uint(o[e]);
          store16(dst + c, u, 1.f);
        }
      }
      if (live && grp == 0) *ldst = (mu + log2f(l)) * 0.69314718055994530942f;
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.o_empty);
      return true;
    };
    // Q of the CTA's item n from shared memory into TMEM, by the groups of half 1 once the
    // last item's scores are complete (half 1's of its last chunk are the last).
    auto stage_q = [&](uint32_t n) {
      const uint32_t qs = n % C::QS;
      if (!mbar_wait_warp(&bar.q_full[qs], (n / C::QS) & 1, abort, p.status, site0 + 13)) return false;
      tc_fence_after();
      const unsigned char *tile = sbase + C::Q_OFF + qs * T::TILE;
#pragma unroll
      for (int j = 0; j < D / 16; ++j) {
        if (j % (C::GRP / 2) != grp % (C::GRP / 2)) continue;
        uint32_t v[8];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int c = 2 * j + e;
          const uint4 a = *reinterpret_cast<const uint4 *>(tile + (c >> 3) * T::R0 + r * 128 + (((c & 7) ^ (r & 7)) << 4));
          v[4 * e] = a.x;
          v[4 * e + 1] = a.y;
          v[4 * e + 2] = a.z;
          v[4 * e + 3] = a.w;
        }
        tmem_st8(tmem + lane_off + C::Q + 8 * j, v);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&bar.q_empty[qs]);
        mbar_arrive(&bar.qt_full);
      }
      return true;
    };
    if (C::QT && x == 1 && blockIdx.x < nitems) ok = stage_q(0);
    uint32_t in = 0;                                // items
    for (int u = blockIdx.x; ok && u < nitems; u += gridDim.x, ++in) {
      const SwaItem w = swa_item(p, u);
      const int i0 = p.q_off + w.qt * kTileRows, pos = i0 + r;
      float m_run = -INFINITY, l_run = 0.f;
      for (int m = 0; m < w.nc; ++m, ++sc) {
        const uint32_t sl = sc & 1;
        if (!(ok = mbar_wait_warp(&bar.s_full[x][sl], (sc >> 1) & 1, abort, p.status, site0 + 11))) break;
        tc_fence_after();
        const int key0 = swa_key(w, m) + C::W * grp;
        const bool full = key0 + C::W - 1 <= i0 && (i0 + kTileRows - 1 - key0 < p.window || key0 + C::W <= p.sink);
        const uint32_t tS = tmem + lane_off + C::s_at(2 * sc + x) + sub;
        uint32_t sv[C::W];
        float *s = reinterpret_cast<float *>(sv);
        if constexpr (C::W == 64) tmem_ld64(tS, sv);
        else tmem_ld32(tS, sv);
        tmem_wait_ld();
        if (C::QT && x == 1 && m == w.nc - 1 && u + (int)gridDim.x < nitems && !(ok = stage_q(in + 1))) break;
        if (!full) {
#pragma unroll
          for (int c = 0; c < C::W; c += 32) {
            const uint32_t b = first_bits(pos + 1 - key0 - c) &
                               (~first_bits(pos + 1 - p.window - key0 - c) | first_bits(p.sink - key0 - c));
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!((b >> e) & 1u)) s[c + e] = -INFINITY;
          }
        }
        float mx4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
        for (int e = 4; e < C::W; ++e) mx4[e & 3] = fmaxf(mx4[e & 3], s[e]);
        const float m_new = fmaxf(m_run, fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * sl2);
        const bool raise = m_new > m_run + kSwaRaise;        // (from -inf too)
        if (__any_sync(FULL, raise)) {
          const float alpha = raise && m_run != -INFINITY ? ex2_approx(m_run - m_new) : 1.f;
          if (raise) {
            l_run *= alpha;
            m_run = m_new;
          }
          // O holds the item's chunks before this one once the last product is done.
          if (__any_sync(FULL, alpha != 1.f)) {
            if (!(ok = mbar_wait_warp(&bar.pv_done[x][sl ^ 1], ((sc - 1) >> 1) & 1, abort, p.status, site0 + 12))) break;
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < D; c += 16) {
              uint32_t o[16];
              tmem_ld16(tOg + c, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              tmem_st16(tOg + c, o);
            }
          }
        }
        const float mu = m_run == -INFINITY ? 0.f : m_run;
        float ls[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < C::W; c += 32) {
          uint32_t pp[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            float x0, x1;
            fma2(x0, x1, s[c + e], s[c + e + 1], sl2, -mu, -mu);
            x0 = ex2_approx(x0);
            x1 = ex2_approx(x1);
            add2(ls[e & 2], ls[(e & 2) + 1], x0, x1);
            pp[e / 2] = pack_bf16x2(x0, x1);
          }
          tmem_st16(tS + c / 2, pp);
        }
        l_run += (ls[0] + ls[1]) + (ls[2] + ls[3]);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.p_full[x][sl]);
        if (pend) {
          pend = false;
          if (!(ok = read_out())) break;
        }
      }
      if (!ok) break;
      ml[((in & 1) * C::GRP + grp) * 128 + r] = make_float2(m_run, l_run);
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.ml_full);
      const int i = w.qt * kTileRows + r;
      live = i < p.N;
      dst = p.out + (int64_t)w.b * p.o_sb + (int64_t)w.h * p.o_sh + (int64_t)i * p.o_sn;
      ldst = p.lse + ((int64_t)w.b * p.hq + w.h) * p.N + i;
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

// ------------------------------------------------------------------ launch

template <int D>
static cudaError_t launch_swa_fwd_d(const CUtensorMap *m, const AttnParams &p, int nsm, cudaStream_t st) {
  cudaError_t e = cudaFuncSetAttribute(swa_fwd_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, SwaFwdCfg<D>::SMEM);
  if (e != cudaSuccess) return e;
  swa_fwd_kernel<D><<<p.ntiles < nsm ? p.ntiles : nsm, SwaFwdCfg<D>::THREADS, SwaFwdCfg<D>::SMEM, st>>>(
      m[0], m[1], m[2], m[3], m[4], m[5], p);
  return cudaGetLastError();
}

// maps: Q, K, V, each with its column tail (D != 64).
cudaError_t launch_swa_fwd(const CUtensorMap *maps, const AttnParams &p, int nsm, cudaStream_t st) {
  switch (p.d) {
    case 64: return launch_swa_fwd_d<64>(maps, p, nsm, st);
    case 80: return launch_swa_fwd_d<80>(maps, p, nsm, st);
    case 128: return launch_swa_fwd_d<128>(maps, p, nsm, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace moba
