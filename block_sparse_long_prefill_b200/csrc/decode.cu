// decode.cu -- attention of one new token per sequence over a paged key-value cache.
//
// Sequence b has len = seq_lens[b] positions; its query sits at the last one and sees the
// keys j < len with (window > 0) len - 1 - j < window or j < sink:
//     out = softmax(scale q K^T) V over these keys, lse = log sum exp(scale q k).
// Position j lies in slot j % page of page table[b, j / page].
//
// Every visible key and value is read once for each group of up to 16 of the G query heads of
// its KV head, so the work is HBM-bound (up to 16 flops a byte).  The keys of a (sequence, KV head,
// group of up to 16 query heads) -- an item -- are cut into tiles of 16, and the work of
// the batch is dealt out in equal runs to a grid of two or three CTAs per SM, whatever the
// sequences' lengths: a run may end inside an item, which then has partial results
// (normalised rows and their log-sum-exp) that a second, small kernel joins.  An item counts
// as its tiles and kDecItem more, about what filling the pipeline and joining the warps
// costs: by tiles alone a run of many one-tile items took six times as long as one of few
// long items (32 ragged sequences of 32 heads with a window of 4096: 237 against 88 us).
// Measured: one sequence of 2^20 tokens, 8 KV heads of 128, 683 us with the call, 6.3 TB/s
// (746 us, 5.8 TB/s on a card with a slower memory); 48 ragged sequences of up to 16384 tokens
// 90 us, 5.1 TB/s (fills and ends of 384 items; 95 us on the other card).
//
// A warp takes every fourth tile of its CTA's run and works alone: its tiles arrive by
// cp.async in a ring of its own (three stages of 16 keys and 16 values, about 9 KB each,
// so an SM has up to 140 KB in flight, several times what its share of the bandwidth
// needs over the memory's latency), page ids are read a tile ahead, and S = Q K^T and
// O += P V run on mma.sync m16n8k16 (query heads as the 16 rows; a tensor pipe at a few
// per cent, so the wider tcgen05 tiles would only idle).  The softmax is one pass with a
// running maximum and sum in fp32; P is rounded to bf16 for the product, as in the prefill (up
// to 2^-8 of each value, the same step as the output's own; the output is off by 0.0015 to
// 0.0022 of its norm, 0.0013 to 0.0016 of them its own rounding).  The four warps' results are
// joined through shared memory at the end of an item.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "common.cuh"
#include "params.h"

namespace moba {

constexpr int kDecThreads = 128;
constexpr int kDecWarps = 4;
constexpr int kDecKeys = 16;      // keys of a tile
constexpr int kDecStages = 3;
constexpr int kDecItem = 8;       // an item's fixed cost in tiles

template <int D>
struct DecCfg {
  static constexpr int CH = D / 8;                    // 16-byte chunks of a row
  static constexpr int RS = D * 2 + 16;               // row stride: ldmatrix without conflicts
  static constexpr int TILE = kDecKeys * RS;          // bytes of a K (or V) tile
  static constexpr int STAGE = 2 * TILE;
  static constexpr int WARP = kDecStages * STAGE;     // a warp's ring
  static constexpr int OROW = D + 4;                  // floats of a row of the joining buffer
  static constexpr int SMEM = kDecWarps * WARP;
  static constexpr int PER_SM = D == 128 ? 2 : 3;     // resident CTAs (shared memory, registers)
  static_assert(kDecWarps * 16 * OROW * 4 <= SMEM, "the joining buffer lies over the rings");
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t &a, uint32_t &b, uint32_t &c, uint32_t &d) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(a), "=r"(b), "=r"(c), "=r"(d) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t &a, uint32_t &b, uint32_t &c, uint32_t &d) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(a), "=r"(b), "=r"(c), "=r"(d) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// What a sequence's query sees: keys [0, s) and [w0, len), counted in one row v < n.
struct Seen {
  int n, s, w0;
};

__device__ __forceinline__ Seen seen_of(const DecodeParams &p, int b) {
  const long long cap = (long long)p.max_pages * p.page;
  const int len0 = __ldg(p.seq_lens + b);
  const int len = (int)min((long long)max(len0, 0), cap);
  Seen x;
  x.w0 = p.window > 0 ? max(0, len - p.window) : 0;
  x.s = min(p.sink, x.w0);
  x.n = x.s + len - x.w0;
  return x;
}

__device__ __forceinline__ int tiles_of(const Seen &x) { return (x.n + kDecKeys - 1) / kDecKeys; }

// Cost of an item of nt tiles, in tiles.
__device__ __forceinline__ int cost_of(int nt) { return nt > 0 ? nt + kDecItem : 0; }

// Length of a CTA's run: at least two tiles for each warp, so that small batches are not
// spread so thin that joining costs more than reading.
__host__ __device__ __forceinline__ int run_of(int total, int ctas) {
  const int r = (total + ctas - 1) / ctas;
  return r < 2 * kDecWarps ? 2 * kDecWarps : r;
}

template <int D>
__global__ void __launch_bounds__(kDecThreads, DecCfg<D>::PER_SM) paged_decode_kernel(const DecodeParams p) {
  using C = DecCfg<D>;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ int sh_sum[kDecWarps + 1];
  __shared__ int sh_at[2];                 // first sequence of the run, cost before it
  __shared__ float sh_m[kDecWarps][16], sh_l[kDecWarps][16];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr uint32_t FULL = 0xffffffffu;
  const int items = p.hkv * p.ngrp;        // items of one sequence

  // Where the CTA's run begins.  Thread i sums the tiles of sequences [i R, (i + 1) R).
  const int R = (p.batch + kDecThreads - 1) / kDecThreads;
  const int bt0 = min(tid * R, p.batch), bt1 = min(bt0 + R, p.batch);
  int mine = 0;
  for (int b = bt0; b < bt1; ++b) mine += cost_of(tiles_of(seen_of(p, b))) * items;
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(FULL, incl, o);
    if (lane >= o) incl += t;
  }
  if (lane == 31) sh_sum[warp] = incl;
  __syncthreads();
  int pre = incl - mine, total = 0;
#pragma unroll
  for (int w = 0; w < kDecWarps; ++w) {
    if (w < warp) pre += sh_sum[w];
    total += sh_sum[w];
  }
  const int run = run_of(total, gridDim.x);
  const int lo = min((long long)blockIdx.x * run, (long long)total);
  const int hi = min((long long)lo + run, (long long)total);
  if (lo < hi && pre <= lo && lo < pre + mine) {
    int at = pre;
    for (int b = bt0; b < bt1; ++b) {
      const int t = cost_of(tiles_of(seen_of(p, b))) * items;
      if (lo < at + t) {
        sh_at[0] = b;
        sh_at[1] = at;
        break;
      }
      at += t;
    }
  }
  if (blockIdx.x == 0) {
    int at = pre;
    for (int b = bt0; b < bt1; ++b) {
      p.before[b] = at;
      at += cost_of(tiles_of(seen_of(p, b))) * items;
      const long long cap = (long long)p.max_pages * p.page;
      const int len = __ldg(p.seq_lens + b);
      if (len < 0 || len > cap) record_index_error(p.status, (33 * 16) * 256);
    }
    if (tid == 0) p.before[p.batch] = total;
  }
  __syncthreads();
  if (lo >= hi) return;

  const uint32_t ring = smem_u32(smem) + warp * C::WARP;
  const bool one = p.kp.sb == p.vp.sb && p.kp.sn == p.vp.sn && p.kp.sh == p.vp.sh;
  const int qr = lane >> 2, qc = (lane & 3) * 2;       // fragment row and first column
  int b = sh_at[0], at = sh_at[1];                     // sequence, cost before it
  Seen sn = seen_of(p, b);
  int nt = tiles_of(sn), cost = cost_of(nt);
  for (int pos = lo, next; pos < hi; pos = next) {
    while (cost * items <= pos - at) {                 // next sequence with keys
      at += cost * items;
      ++b;
      sn = seen_of(p, b);
      nt = tiles_of(sn);
      cost = cost_of(nt);
    }
    const int item = (pos - at) / cost;
    const int begin = at + item * cost;                // the item is [begin, begin + cost)
    next = min(begin + cost, hi);
    const int t0 = max(0, pos - begin - kDecItem);     // tiles [t0, t1) of the item
    const int t1 = next - begin - kDecItem;
    if (t0 >= t1) continue;                            // its fixed cost alone
    const int hk = item / p.ngrp, h0 = hk * p.G + (item % p.ngrp) * kDecodeRows;
    const int rows = min(kDecodeRows, (hk + 1) * p.G - h0);
    const uint16_t *kb = p.kp.ptr + (int64_t)hk * p.kp.sh, *vb = p.vp.ptr + (int64_t)hk * p.vp.sh;
    const int32_t *tab = p.table + (int64_t)b * p.max_pages;

    // Place in the pages of the lane's row (lanes 0 - 15) of tile t: page and slot, then
    // element offsets, or -1 for a row behind the last visible key or on a page that is not
    // there.
    struct Place {
      int id, slot;            // id -2: no key
    };
    auto look = [&](int t) {
      Place x{-2, 0};
      const int v = t * kDecKeys + lane;
      if (lane < kDecKeys && t < t1 && v < sn.n) {
        const int key = v < sn.s ? v : v - sn.s + sn.w0;
        const int pg = key / p.page;
        x.slot = key - pg * p.page;
        x.id = max(-1, __ldg(tab + pg));
      }
      return x;
    };
    auto place = [&](const Place &x, int64_t &ko, int64_t &vo) {
      ko = vo = -1;
      if (x.id >= 0 && x.id < p.num_pages) {
        ko = (int64_t)x.id * p.kp.sb + (int64_t)x.slot * p.kp.sn;
        vo = one ? ko : (int64_t)x.id * p.vp.sb + (int64_t)x.slot * p.vp.sn;
      } else if (x.id != -2) {
        record_index_error(p.status, (33 * 16 + 1) * 256);
      }
    };
    auto issue = [&](int stage, int64_t ko, int64_t vo) {
      const uint32_t dst = ring + stage * C::STAGE;
#pragma unroll
      for (int i = 0; i < C::CH / 2; ++i) {
        const int c = i * 32 + lane, row = c / C::CH, col = c % C::CH;
        const int64_t k = __shfl_sync(FULL, ko, row);
        const int64_t w = one ? k : __shfl_sync(FULL, vo, row);
        const uint32_t d = dst + row * C::RS + col * 16;
        cp_async_16_zfill(d, k < 0 ? kb : kb + k + col * 8, k >= 0);
        cp_async_16_zfill(d + C::TILE, k < 0 ? vb : vb + w + col * 8, k >= 0);
      }
    };

    // The first tiles; then the query fragments (rows of heads, bf16 pairs).
    int64_t ko, vo;
    uint32_t okm[kDecStages];                          // visible keys of the stages' tiles
    int tl = t0 + warp;                                // next tile to load
    Place ahead[kDecStages];                           // (page ids of the first tiles together)
#pragma unroll
    for (int s = 0; s < kDecStages; ++s) ahead[s] = look(tl + s * kDecWarps);
#pragma unroll
    for (int s = 0; s < kDecStages - 1; ++s, tl += kDecWarps) {
      place(ahead[s], ko, vo);
      okm[s] = __ballot_sync(FULL, ko >= 0) & 0xffffu;
      if (tl < t1) issue(s, ko, vo);
      cp_async_commit();
    }
    Place nx = ahead[kDecStages - 1];
    uint32_t qa[D / 16][4];
    {
      const uint16_t *q0 = p.q + (int64_t)b * p.q_sb + (int64_t)(h0 + qr) * p.q_sh + qc;
      const uint16_t *q1 = q0 + 8 * p.q_sh;
      const bool r0 = qr < rows, r1 = qr + 8 < rows;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        qa[ks][0] = r0 ? __ldg(reinterpret_cast<const uint32_t *>(q0 + ks * 16)) : 0u;
        qa[ks][1] = r1 ? __ldg(reinterpret_cast<const uint32_t *>(q1 + ks * 16)) : 0u;
        qa[ks][2] = r0 ? __ldg(reinterpret_cast<const uint32_t *>(q0 + ks * 16 + 8)) : 0u;
        qa[ks][3] = r1 ? __ldg(reinterpret_cast<const uint32_t *>(q1 + ks * 16 + 8)) : 0u;
      }
    }
    float o[D / 8][4];
#pragma unroll
    for (int n = 0; n < D / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    int stage = 0;
    for (int t = t0 + warp; t < t1; t += kDecWarps) {
      // Load two tiles ahead (into the stage that the last turn read), with the place read
      // a turn ago; then read the place of the next one.
      {
        const int into = stage == 0 ? kDecStages - 1 : stage - 1;
        place(nx, ko, vo);
        const uint32_t ok = __ballot_sync(FULL, ko >= 0) & 0xffffu;
#pragma unroll
        for (int s = 0; s < kDecStages; ++s)
          if (s == into) okm[s] = ok;
        if (tl < t1) issue(into, ko, vo);
        cp_async_commit();
        tl += kDecWarps;
        nx = look(tl);
      }
      cp_async_wait_group<kDecStages - 1>();
      __syncwarp();
      uint32_t ok = okm[0];
#pragma unroll
      for (int s = 1; s < kDecStages; ++s)
        if (s == stage) ok = okm[s];
      const uint32_t ks0 = ring + stage * C::STAGE, vs0 = ks0 + C::TILE;
      float s0[4] = {0.f, 0.f, 0.f, 0.f}, s1[4] = {0.f, 0.f, 0.f, 0.f};
      {
        // Matrices: keys 0-7 and 8-15 at columns 0-7 and 8-15 of the k-step.
        const uint32_t a = ks0 + ((lane & 7) + (lane >> 4) * 8) * C::RS + ((lane >> 3) & 1) * 16;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          uint32_t b0, b1, b2, b3;
          ldsm4(a + ks * 32, b0, b1, b2, b3);
          mma_bf16(s0, qa[ks], b0, b1);
          mma_bf16(s1, qa[ks], b2, b3);
        }
      }
      const float sl = p.scale_log2;
      float z0[4] = {s0[0] * sl, s0[1] * sl, s1[0] * sl, s1[1] * sl};   // row qr
      float z1[4] = {s0[2] * sl, s0[3] * sl, s1[2] * sl, s1[3] * sl};   // row qr + 8
      if (ok != 0xffffu) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (!((ok >> (qc + (e & 1) + (e >> 1) * 8)) & 1u)) z0[e] = z1[e] = -INFINITY;
      }
      float x0 = fmaxf(fmaxf(z0[0], z0[1]), fmaxf(z0[2], z0[3]));
      float x1 = fmaxf(fmaxf(z1[0], z1[1]), fmaxf(z1[2], z1[3]));
      x0 = fmaxf(x0, __shfl_xor_sync(FULL, x0, 1));
      x1 = fmaxf(x1, __shfl_xor_sync(FULL, x1, 1));
      x0 = fmaxf(x0, __shfl_xor_sync(FULL, x0, 2));
      x1 = fmaxf(x1, __shfl_xor_sync(FULL, x1, 2));
      const bool up = x0 > m0 || x1 > m1;
      if (__any_sync(FULL, up)) {
        const float n0 = fmaxf(m0, x0), n1 = fmaxf(m1, x1);
        const float a0 = n0 == -INFINITY ? 1.f : ex2_approx(m0 - n0);
        const float a1 = n1 == -INFINITY ? 1.f : ex2_approx(m1 - n1);
        m0 = n0;
        m1 = n1;
        l0 *= a0;
        l1 *= a1;
#pragma unroll
        for (int n = 0; n < D / 8; ++n) {
          o[n][0] *= a0;
          o[n][1] *= a0;
          o[n][2] *= a1;
          o[n][3] *= a1;
        }
      }
      const float u0 = m0 == -INFINITY ? 0.f : m0, u1 = m1 == -INFINITY ? 0.f : m1;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        z0[e] = ex2_approx(z0[e] - u0);
        z1[e] = ex2_approx(z1[e] - u1);
      }
      l0 += (z0[0] + z0[1]) + (z0[2] + z0[3]);
      l1 += (z1[0] + z1[1]) + (z1[2] + z1[3]);
      const uint32_t pa[4] = {pack_bf16x2(z0[0], z0[1]), pack_bf16x2(z1[0], z1[1]),
                              pack_bf16x2(z0[2], z0[3]), pack_bf16x2(z1[2], z1[3])};
      {
        // Matrices: keys 0-7 and 8-15 of columns n and n + 8.
        const uint32_t a = vs0 + (lane & 15) * C::RS + (lane >> 4) * 16;
#pragma unroll
        for (int n = 0; n < D / 16; ++n) {
          uint32_t b0, b1, b2, b3;
          ldsm4_t(a + n * 32, b0, b1, b2, b3);
          mma_bf16(o[2 * n], pa, b0, b1);
          mma_bf16(o[2 * n + 1], pa, b2, b3);
        }
      }
      __syncwarp();      // the stage is read; the next turn loads into it
      stage = stage + 1 == kDecStages ? 0 : stage + 1;
    }
    cp_async_wait_all();
    l0 += __shfl_xor_sync(FULL, l0, 1);
    l1 += __shfl_xor_sync(FULL, l1, 1);
    l0 += __shfl_xor_sync(FULL, l0, 2);
    l1 += __shfl_xor_sync(FULL, l1, 2);

    // Join the warps: rows into shared memory (over the rings, which are drained).
    __syncthreads();
    float *orow = reinterpret_cast<float *>(smem);
    if ((lane & 3) == 0) {
      sh_m[warp][qr] = m0;
      sh_m[warp][qr + 8] = m1;
      sh_l[warp][qr] = l0;
      sh_l[warp][qr + 8] = l1;
    }
#pragma unroll
    for (int n = 0; n < D / 8; ++n) {
      if (qr < rows)
        *reinterpret_cast<float2 *>(orow + (warp * 16 + qr) * C::OROW + n * 8 + qc) = make_float2(o[n][0], o[n][1]);
      if (qr + 8 < rows)
        *reinterpret_cast<float2 *>(orow + (warp * 16 + qr + 8) * C::OROW + n * 8 + qc) = make_float2(o[n][2], o[n][3]);
    }
    __syncthreads();
    const bool whole = t0 == 0 && t1 == nt;
    const int64_t slot = (int64_t)blockIdx.x * 2 + (pos == lo ? 0 : 1);   // (lo >= begin: its first)
    for (int i = tid; i < rows * (D / 4); i += kDecThreads) {
      const int r = i / (D / 4), c = (i % (D / 4)) * 4;
      float mx = sh_m[0][r];
#pragma unroll
      for (int w = 1; w < kDecWarps; ++w) mx = fmaxf(mx, sh_m[w][r]);
      const float mu = mx == -INFINITY ? 0.f : mx;
      float l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < kDecWarps; ++w) {
        const float f = ex2_approx(sh_m[w][r] - mu);
        const float4 x = *reinterpret_cast<const float4 *>(orow + (w * 16 + r) * C::OROW + c);
        l = fmaf(f, sh_l[w][r], l);
        acc[0] = fmaf(f, x.x, acc[0]);
        acc[1] = fmaf(f, x.y, acc[1]);
        acc[2] = fmaf(f, x.z, acc[2]);
        acc[3] = fmaf(f, x.w, acc[3]);
      }
      const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);   // (a NaN stays)
      const float lse2 = mu + log2f(l);                              // no keys: -inf
      if (whole) {
        *reinterpret_cast<uint2 *>(p.out + (int64_t)b * p.o_sb + (int64_t)(h0 + r) * p.o_sh + c) =
            make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv));
        if (c == 0) p.lse[(int64_t)b * p.hq + h0 + r] = lse2 * 0.69314718055994530942f;
      } else {
        *reinterpret_cast<float4 *>(p.opart + (slot * kDecodeRows + r) * D + c) =
            make_float4(acc[0] * inv, acc[1] * inv, acc[2] * inv, acc[3] * inv);
        if (c == 0) p.lpart[slot * kDecodeRows + r] = lse2;
      }
    }
    __syncthreads();     // the buffer is read; the next item's loads may overwrite it
  }
}

// Joins the partial results of the items that several CTAs share, and writes the empty
// row of a sequence without visible keys.  One CTA per (sequence, item): the parts' weights
// first (all of their log-sum-exps are read at once), then the weighted sum.
// Its warps take a row each and, where there are fewer rows than warps, a share of the parts.
constexpr int kJoinWarps = 16;
template <int D>
__global__ void __launch_bounds__(32 * kJoinWarps) paged_decode_join_kernel(const DecodeParams p, int ctas) {
  __shared__ float wgt[kDecodeRows][kDecodeCtas + 1];
  __shared__ float inv[kDecodeRows], lse[kDecodeRows];
  __shared__ float4 sum[kJoinWarps][D / 4];
  constexpr uint32_t FULL = 0xffffffffu;
  // The partial results are the previous launch's: wait until it has completed.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x, items = p.hkv * p.ngrp;
  const int b = blockIdx.x / items, item = blockIdx.x % items;
  const int hk = item / p.ngrp, h0 = hk * p.G + (item % p.ngrp) * kDecodeRows;
  const int rows = min(kDecodeRows, (hk + 1) * p.G - h0);
  const int before = p.before[b], cost = (p.before[b + 1] - before) / items, total = p.before[p.batch];
  if (cost == 0) {
    for (int i = tid; i < rows * (D / 4); i += 32 * kJoinWarps) {
      const int r = i / (D / 4), c = (i % (D / 4)) * 4;
      *reinterpret_cast<uint2 *>(p.out + (int64_t)b * p.o_sb + (int64_t)(h0 + r) * p.o_sh + c) = make_uint2(0u, 0u);
      if (c == 0) p.lse[(int64_t)b * p.hq + h0 + r] = -INFINITY;
    }
    return;
  }
  const int run = run_of(total, ctas);
  const int a = before + item * cost;                   // the item is [a, a + cost)
  const int c0 = (a + kDecItem) / run, c1 = (a + cost - 1) / run;
  if (c0 == c1) return;                                 // whole in one CTA
  const int n = c1 - c0 + 1;
  auto slot = [&](int x) { return (int64_t)(c0 + x) * 2 + ((int64_t)(c0 + x) * run >= a ? 0 : 1); };
  for (int i = tid; i < rows * n; i += 32 * kJoinWarps) {
    const int r = i / n, x = i - r * n;
    wgt[r][x] = p.lpart[slot(x) * kDecodeRows + r];
  }
  __syncthreads();
  for (int r = tid >> 5; r < rows; r += kJoinWarps) {
    const int lane = tid & 31;
    float mx = -INFINITY, l = 0.f;
    for (int x = lane; x < n; x += 32) mx = fmaxf(mx, wgt[r][x]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, o));
    const float u = mx == -INFINITY ? 0.f : mx;
    for (int x = lane; x < n; x += 32) {
      const float f = ex2_approx(wgt[r][x] - u);
      wgt[r][x] = f;
      l += f;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(FULL, l, o);
    if (lane == 0) {
      inv[r] = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
      lse[r] = (u + log2f(l)) * 0.69314718055994530942f;
    }
  }
  __syncthreads();
  const int warp = tid >> 5, lane = tid & 31;
  const int shares = kJoinWarps / rows, r = warp % rows, share = warp / rows;
  if (share < shares && lane < D / 4) {
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int x = share; x < n; x += shares) {
      const float4 y = *reinterpret_cast<const float4 *>(p.opart + (slot(x) * kDecodeRows + r) * D + lane * 4);
      const float f = wgt[r][x];
      acc.x = fmaf(f, y.x, acc.x);
      acc.y = fmaf(f, y.y, acc.y);
      acc.z = fmaf(f, y.z, acc.z);
      acc.w = fmaf(f, y.w, acc.w);
    }
    sum[warp][lane] = acc;
  }
  __syncthreads();
  if (share == 0 && lane < D / 4) {
    float4 acc = sum[warp][lane];
    for (int x = 1; x < shares; ++x) {
      const float4 y = sum[warp + x * rows][lane];
      acc.x += y.x;
      acc.y += y.y;
      acc.z += y.z;
      acc.w += y.w;
    }
    const float v = inv[r];
    *reinterpret_cast<uint2 *>(p.out + (int64_t)b * p.o_sb + (int64_t)(h0 + r) * p.o_sh + lane * 4) =
        make_uint2(pack_bf16x2(acc.x * v, acc.y * v), pack_bf16x2(acc.z * v, acc.w * v));
    if (lane == 0) p.lse[(int64_t)b * p.hq + h0 + r] = lse[r];
  }
}

// ------------------------------------------------------------------ launch

template <int D>
static cudaError_t launch_decode_d(const DecodeParams &p, int nsm, cudaStream_t st) {
  const int ctas = min(DecCfg<D>::PER_SM * nsm, kDecodeCtas);
  cudaError_t e = cudaFuncSetAttribute(paged_decode_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       DecCfg<D>::SMEM);
  if (e != cudaSuccess) return e;
  paged_decode_kernel<D><<<ctas, kDecThreads, DecCfg<D>::SMEM, st>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  // The join may be set up while the main kernel runs; it waits for its completion.
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(p.batch * p.hkv * p.ngrp));
  cfg.blockDim = dim3(32 * kJoinWarps);
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_decode_join_kernel<D>, p, ctas);
}

cudaError_t launch_decode(const DecodeParams &p, int d, int nsm, cudaStream_t st) {
  switch (d) {
    case 64: return launch_decode_d<64>(p, nsm, st);
    case 80: return launch_decode_d<80>(p, nsm, st);
    case 128: return launch_decode_d<128>(p, nsm, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace moba
