// rope.cu -- norms of queries and keys per head with the position rotation in the same
// pass (forward and backward), and the paged append that does both on the way into the
// cache.
//
// A row x of d values (one head of one token at position p) becomes
//     xn = x rstd w,  rstd = 1 / sqrt(mean(x^2) + eps)      (no norm: xn = x)
//     (u_i, u_j) = (xn_i cos - xn_j sin, xn_j cos + xn_i sin)
// for the pairs (i, j) of its first `rot` columns at the angles of position p (halves:
// j = i + rot / 2; interleaved: j = i + 1); the other columns pass.  The backward is
//     g = R^T dy,  dw += g x rstd,  dx = rstd (g w - x rstd mean(g w x rstd)).
// Everything between the bf16 loads and stores is fp32.
//
// The work is one read and one write of every row, so it is HBM-bound.  A lane holds one
// 16-byte vector (8 columns) of a row, d / 8 lanes a row, so a warp carries 32 / (d / 8)
// tokens; it takes a run of heads of these tokens, all of their rows in flight (cp.async into
// slots of its own: registers as the buffer spilled, and fewer rows in flight took 178
// against 133 us below), and keeps the angles times the weights of its columns in registers.
// In the half layout a column's partner sits in another lane's vector: four shuffles of
// packed bf16 pairs fetch it, and the row sums are a butterfly of the same lanes.
// Measured: forward of 32768 tokens, 32 and 8 heads of 128, 125 us (5.4 TB/s); append of
// 4 ragged chunks of up to 4096 tokens, 32 KV heads of 80, 37.5 us (5.5 TB/s), of one token of
// 64 sequences, 32 and 8 heads of 128, 3.5 us in a graph; backward of 2 x 8191 tokens, 32 and
// 8 heads of 128, 122 us (4.1 TB/s): its arithmetic, 230 instructions a warp and row group,
// and its registers (2 CTAs an SM; 3 spill, 297 us) bound it as much as HBM does.  Without
// norms (all 128 columns turned, halves) 80 us, 4.3 TB/s.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "params.h"
#include "rows.cuh"

namespace moba {

constexpr int kRopeHeads = 8;   // most heads of a warp's task, their rows in flight together
constexpr int kRopeThreads = 256;
constexpr int kRopeWarps = kRopeThreads / 32;

__device__ __forceinline__ void load_weight(const RopeWeight &w, int c0, float (&x)[8]) {
  if (!w.ptr) {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = 1.f;
  } else if (w.f32) {
    const float *p = static_cast<const float *>(w.ptr) + c0;
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = __ldg(p + e);
  } else {
    const uint16_t *p = static_cast<const uint16_t *>(w.ptr) + c0;
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = __uint_as_float((uint32_t)__ldg(p + e) << 16);
  }
}

// A vector's eight values as pairs for the packed fp32 instructions (each half rounded as
// the scalar instruction would).
struct Vec8 {
  float2 v[4];
};
__device__ __forceinline__ Vec8 unpack_v(const uint4 &a) {
  Vec8 x;
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int e = 0; e < 4; ++e)
    x.v[e] = make_float2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xFFFF0000u));
  return x;
}
__device__ __forceinline__ uint4 pack_v(const Vec8 &x) {
  return make_uint4(pack_bf16x2(x.v[0].x, x.v[0].y), pack_bf16x2(x.v[1].x, x.v[1].y),
                    pack_bf16x2(x.v[2].x, x.v[2].y), pack_bf16x2(x.v[3].x, x.v[3].y));
}
__device__ __forceinline__ Vec8 to_v(const float (&x)[8]) {
  Vec8 y;
#pragma unroll
  for (int e = 0; e < 4; ++e) y.v[e] = make_float2(x[2 * e], x[2 * e + 1]);
  return y;
}
__device__ __forceinline__ Vec8 mul_v(const Vec8 &a, const Vec8 &b) {
  Vec8 c;
#pragma unroll
  for (int e = 0; e < 4; ++e) c.v[e] = __fmul2_rn(a.v[e], b.v[e]);
  return c;
}
__device__ __forceinline__ Vec8 mul_v(const Vec8 &a, float b) {
  Vec8 c;
#pragma unroll
  for (int e = 0; e < 4; ++e) c.v[e] = __fmul2_rn(a.v[e], make_float2(b, b));
  return c;
}
__device__ __forceinline__ Vec8 fma_v(const Vec8 &a, const Vec8 &b, const Vec8 &c) {
  Vec8 d;
#pragma unroll
  for (int e = 0; e < 4; ++e) d.v[e] = __ffma2_rn(a.v[e], b.v[e], c.v[e]);
  return d;
}
__device__ __forceinline__ float dot_v(const Vec8 &a, const Vec8 &b) {
  float2 s = __fmul2_rn(a.v[0], b.v[0]), t = __fmul2_rn(a.v[1], b.v[1]);
  s = __ffma2_rn(a.v[2], b.v[2], s);
  t = __ffma2_rn(a.v[3], b.v[3], t);
  s = __fadd2_rn(s, t);
  return s.x + s.y;
}

// A lane's place in the rotation: the lane that holds its columns' partners, and the
// first pair of its angles.  Columns outside the rotation have themselves as partners.
struct Place {
  int mate;    // lane of the partner vector (the lane itself: within the vector, or none)
  int a0;      // first pair
  int kind;    // 0 passes, 1 the lower half (x c - y s), 2 the upper half, 3 interleaved
};

__device__ __forceinline__ Place place_of(int v, int lane, int rot, int interleaved) {
  Place p;
  const int hv = rot / 16;  // vectors per half
  p.mate = lane;
  p.a0 = 0;
  p.kind = 0;
  if (v < 2 * hv) {
    if (interleaved) {
      p.kind = 3;
      p.a0 = v * 4;
    } else {
      const bool low = v < hv;
      p.kind = low ? 1 : 2;
      p.mate = low ? lane + hv : lane - hv;
      p.a0 = (low ? v : v - hv) * 8;
    }
  }
  return p;
}

// The lane's factors at one position: y = x c + partner s.
__device__ __forceinline__ void load_angles(const Place &pl, const float *cosp, const float *sinp,
                                            int rot, int pos, float (&c)[8], float (&s)[8]) {
  const int64_t off = (int64_t)pos * (rot / 2) + pl.a0;
  if (pl.kind == 0) {
#pragma unroll
    for (int e = 0; e < 8; ++e) { c[e] = 1.f; s[e] = 0.f; }
  } else if (pl.kind == 3) {
    const float4 a = __ldg(reinterpret_cast<const float4 *>(cosp + off));
    const float4 b = __ldg(reinterpret_cast<const float4 *>(sinp + off));
    const float ca[4] = {a.x, a.y, a.z, a.w}, sa[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      c[2 * e] = c[2 * e + 1] = ca[e];
      s[2 * e] = -sa[e];
      s[2 * e + 1] = sa[e];
    }
  } else {
    const float sg = pl.kind == 1 ? -1.f : 1.f;
#pragma unroll
    for (int e = 0; e < 8; e += 4) {
      const float4 a = __ldg(reinterpret_cast<const float4 *>(cosp + off + e));
      const float4 b = __ldg(reinterpret_cast<const float4 *>(sinp + off + e));
      c[e] = a.x; c[e + 1] = a.y; c[e + 2] = a.z; c[e + 3] = a.w;
      s[e] = sg * b.x; s[e + 1] = sg * b.y; s[e + 2] = sg * b.z; s[e + 3] = sg * b.w;
    }
  }
}

// The partner's values of a packed row vector x = unpack_v(a).  (Where a column has none
// its factor is zero, and so is this, so that infinities pass.)
__device__ __forceinline__ Vec8 mate_v(const Place &pl, int interleaved, const uint4 &a, const Vec8 &x) {
  Vec8 y;
  if (interleaved) {
#pragma unroll
    for (int e = 0; e < 4; ++e) y.v[e] = make_float2(x.v[e].y, x.v[e].x);
  } else {
    uint4 b;
    b.x = __shfl_sync(kFull, a.x, pl.mate);
    b.y = __shfl_sync(kFull, a.y, pl.mate);
    b.z = __shfl_sync(kFull, a.z, pl.mate);
    b.w = __shfl_sync(kFull, a.w, pl.mate);
    y = unpack_v(b);
  }
  if (pl.kind == 0) {
#pragma unroll
    for (int e = 0; e < 4; ++e) y.v[e] = make_float2(0.f, 0.f);
  }
  return y;
}

// Normalise and rotate one row vector: y = (x cw + partner sw) rstd, cw and sw the lane's
// angles times the weights of its own and of its partners' columns.
template <int D>
__device__ __forceinline__ uint4 turn_row(const uint4 &a, bool norm, const Place &pl, int interleaved,
                                          int base, int v, float eps, const Vec8 &cw, const Vec8 &sw) {
  const Vec8 x = unpack_v(a);
  Vec8 u = fma_v(mate_v(pl, interleaved, a, x), sw, mul_v(x, cw));
  if (norm) u = mul_v(u, rsqrtf(row_sum<D>(dot_v(x, x), base, v) * (1.f / D) + eps));
  return pack_v(u);
}

// The weights of a lane's columns and of its partners' columns.
__device__ __forceinline__ void load_weights(const RopeWeight &wt, const Place &pl, int v, int lane,
                                             float (&w)[8], float (&wm)[8]) {
  load_weight(wt, v * 8, w);
  if (pl.kind == 3) {
#pragma unroll
    for (int e = 0; e < 8; ++e) wm[e] = w[e ^ 1];
  } else {
    load_weight(wt, (v + pl.mate - lane) * 8, wm);
  }
}

// Angles times weights.
__device__ __forceinline__ void load_factors(const Place &pl, const float *cosp, const float *sinp, int rot,
                                             int pos, const RopeWeight &wt, int v, int lane, Vec8 &cw, Vec8 &sw) {
  float c[8], s[8];
  load_angles(pl, cosp, sinp, rot, pos, c, s);
  cw = to_v(c);
  sw = to_v(s);
  if (wt.ptr) {
    float w[8], wm[8];
    load_weights(wt, pl, v, lane, w, wm);
    cw = mul_v(cw, to_v(w));
    sw = mul_v(sw, to_v(wm));
  }
}

// A lane's slots in shared memory: it copies its own vectors there and reads them back, so
// rows in flight cost no registers and need no barrier.
__device__ __forceinline__ uint32_t lane_slot(const uint4 *buf, int i) {
  return smem_u32(buf + i * 32 + (threadIdx.x & 31));
}

// ------------------------------------------------------------------ forward

// hpt: heads of a warp's task.
template <int D>
__global__ void __launch_bounds__(kRopeThreads, 4) qk_norm_rope_fwd_kernel(const RopeParams p, int hpt) {
  constexpr int LPR = RowLanes<D>::LPR, RPW = RowLanes<D>::RPW;
  __shared__ uint4 slots[kRopeWarps][kRopeHeads * 32];
  const int lane = threadIdx.x & 31;
  const int sub = min(lane / LPR, RPW - 1), v = lane - sub * LPR, base = sub * LPR;
  const bool in = v < LPR;
  const int cq = (p.hq + hpt - 1) / hpt, ck = (p.hkv + hpt - 1) / hpt;
  const int groups = (p.N + RPW - 1) / RPW;
  // The block's warps take neighbouring tokens of the same heads, so that head-major rows are
  // written in runs of kRopeWarps warps.
  const int hc = (int)(blockIdx.x % (unsigned)(cq + ck));
  const long long tg = (long long)(blockIdx.x / (unsigned)(cq + ck)) * kRopeWarps + (threadIdx.x >> 5);
  const int b = (int)(tg / groups);
  if (b >= p.batch) return;
  const int n = (int)(tg % groups) * RPW + sub;
  const bool isq = hc < cq;
  const RopeTensor src = isq ? p.q : p.k, dst = isq ? p.qo : p.ko;
  const RopeWeight wt = isq ? p.qw : p.kw;
  const int h0 = (isq ? hc : hc - cq) * hpt;
  const int nh = min(hpt, (isq ? p.hq : p.hkv) - h0);
  bool live = in && n < p.N;
  int pos = n;
  if (live && p.positions) pos = __ldg(p.positions + (int64_t)b * p.N + n);
  if (live && (pos < 0 || pos >= p.max_pos)) {
    live = false;
    record_index_error(p.status, (32 * 16 + 1) * 256);
  }
  const int vv = in ? v : 0;
  const Place pl = place_of(vv, lane, p.rot, p.interleaved);
  uint16_t *out = dst.ptr + b * dst.sb + (int64_t)n * dst.sn + vv * 8 + h0 * dst.sh;
  // (A lane without a row of its own reads the tensor's first.)
  const uint16_t *row = src.ptr + (live ? b * src.sb + (int64_t)n * src.sn + vv * 8 : 0) + h0 * src.sh;
  uint4 *buf = slots[threadIdx.x >> 5];
  for (int h = 0; h < nh; ++h) cp_async_16(lane_slot(buf, h), row + h * src.sh);
  cp_async_commit();
  Vec8 cw, sw;
  load_factors(pl, p.cosp, p.sinp, p.rot, live ? pos : 0, wt, vv, lane, cw, sw);
  cp_async_wait_all();
#pragma unroll 2
  for (int h = 0; h < nh; ++h) {
    const uint4 o = turn_row<D>(buf[h * 32 + lane], wt.ptr != nullptr, pl, p.interleaved, base, vv, p.eps, cw, sw);
    if (live) *reinterpret_cast<uint4 *>(out + h * dst.sh) = o;
  }
}

// ------------------------------------------------------------------ backward

constexpr int kRopeRound = 4;   // heads of a round of the backward

// Persistent: a lane's columns are the same in all of its rows, so it sums their weight
// gradients in registers; the CTA's lanes of equal columns add up in one order and leave
// one partial row, which qk_norm_rope_dw_kernel sums over the CTAs (no atomics).  A round is
// four heads of a warp's tokens; the next round's rows are in flight while one is worked on,
// and two rounds in a row share a token's angles.
template <int D>
__global__ void __launch_bounds__(kRopeThreads, 2) qk_norm_rope_bwd_kernel(const RopeParams p) {
  constexpr int LPR = RowLanes<D>::LPR, RPW = RowLanes<D>::RPW, R = kRopeRound;
  extern __shared__ __align__(16) unsigned char rope_smem[];   // [warp][buffer][g, x][R][32] vectors
  __shared__ float part[kRopeWarps * RPW][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = min(lane / LPR, RPW - 1), v = lane - sub * LPR, base = sub * LPR;
  const bool in = v < LPR;
  const int vv = in ? v : 0;
  uint4 *ring = reinterpret_cast<uint4 *>(rope_smem) + warp * (2 * 2 * R * 32);
  const int groups = (p.N + RPW - 1) / RPW;
  const Place pl = place_of(vv, lane, p.rot, p.interleaved);
  const int gw = blockIdx.x * kRopeWarps + warp, nw = gridDim.x * kRopeWarps;
  for (int side = 0; side < 2; ++side) {
    const bool isq = side == 0;
    const RopeTensor src = isq ? p.q : p.k, dst = isq ? p.qo : p.ko, up = isq ? p.gq : p.gk;
    const RopeWeight wt = isq ? p.qw : p.kw;
    const bool norm = wt.ptr != nullptr;
    const int heads = isq ? p.hq : p.hkv, chunks = (heads + R - 1) / R;
    Vec8 w, dw, c, s;                  // (s: the sines of R^T, their sign turned)
    {
      float x[8];
      load_weight(wt, vv * 8, x);
      w = to_v(x);
#pragma unroll
      for (int e = 0; e < 4; ++e) dw.v[e] = make_float2(0.f, 0.f);
    }
    // Rounds in pairs: a warp takes the rounds 2 k, 2 k + 1 for k = gw, gw + nw, ...
    // (Below 2^32 - 2^14 by the call's check, so that the steps cannot pass the end.)
    const unsigned rounds = (unsigned)chunks * (unsigned)groups * (unsigned)p.batch;
    auto after = [&](unsigned k) { return (k & 1) ? k + 2u * nw - 1u : k + 1u; };
    struct Round {
      int b, n, h0, nh, pos;
      bool live;
      unsigned tg;
    };
    auto decode = [&](unsigned k) {
      Round x;
      x.tg = k / (unsigned)chunks;
      x.h0 = (int)(k - x.tg * chunks) * R;
      x.nh = min(R, heads - x.h0);
      x.b = (int)(x.tg / (unsigned)groups);
      x.n = (int)(x.tg - (unsigned)x.b * groups) * RPW + sub;
      x.live = in && x.n < p.N;
      x.pos = x.n;
      if (x.live && p.positions) x.pos = __ldg(p.positions + (int64_t)x.b * p.N + x.n);
      if (x.live && (x.pos < 0 || x.pos >= p.max_pos)) {
        x.live = false;
        record_index_error(p.status, (32 * 16 + 2) * 256);
      }
      return x;
    };
    auto issue = [&](const Round &x, int buf) {
      const uint16_t *g = up.ptr + (x.live ? x.b * up.sb + (int64_t)x.n * up.sn + vv * 8 : 0) + x.h0 * up.sh;
      const uint16_t *r = src.ptr + (x.live ? x.b * src.sb + (int64_t)x.n * src.sn + vv * 8 : 0) + x.h0 * src.sh;
      uint4 *to = ring + buf * (2 * R * 32);
      for (int i = 0; i < x.nh; ++i) {
        cp_async_16_zfill(lane_slot(to, i), g + i * up.sh, x.live);
        if (norm) cp_async_16_zfill(lane_slot(to, R + i), r + i * src.sh, x.live);
      }
    };
    unsigned k = 2u * gw, tg = 0xFFFFFFFFu;
    Round cur{};
    if (k < rounds) {
      cur = decode(k);
      issue(cur, 0);
    }
    cp_async_commit();
    for (int buf = 0; k < rounds; buf ^= 1) {
      const unsigned kn = after(k);
      Round nx{};
      if (kn < rounds) {
        nx = decode(kn);
        issue(nx, buf ^ 1);
      }
      cp_async_commit();
      if (cur.tg != tg) {
        float x[8], y[8];
        load_angles(pl, p.cosp, p.sinp, p.rot, cur.live ? cur.pos : 0, x, y);
        c = to_v(x);
        s = mul_v(to_v(y), -1.f);
        tg = cur.tg;
      }
      cp_async_wait_group<1>();
      uint16_t *out = dst.ptr + cur.b * dst.sb + (int64_t)cur.n * dst.sn + vv * 8 + cur.h0 * dst.sh;
      const uint4 *from = ring + buf * (2 * R * 32) + lane;
      for (int i = 0; i < cur.nh; ++i) {
        const uint4 ga = from[i * 32];
        const Vec8 dy = unpack_v(ga);
        Vec8 g = fma_v(mate_v(pl, p.interleaved, ga, dy), s, mul_v(dy, c));
        if (norm) {
          const Vec8 x = unpack_v(from[(R + i) * 32]), gw = mul_v(g, w);
          const float ss = row_sum<D>(dot_v(x, x), base, vv);
          const float gx = row_sum<D>(dot_v(gw, x), base, vv);
          // (A lane without a row has zeros, which eps = 0 would turn into 0 times infinity.)
          const float r = cur.live ? rsqrtf(ss * (1.f / D) + p.eps) : 0.f;
          const Vec8 xn = mul_v(x, r);
          dw = fma_v(g, xn, dw);
          const float m = -gx * (1.f / D) * r;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            g.v[e] = __fmul2_rn(__ffma2_rn(xn.v[e], make_float2(m, m), gw.v[e]), make_float2(r, r));
        }
        if (cur.live) *reinterpret_cast<uint4 *>(out + i * dst.sh) = pack_v(g);
      }
      k = kn;
      cur = nx;
    }
    cp_async_wait_all();
    if (!norm) continue;   // (uniform over the grid)
    __syncthreads();
    if (in) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        part[warp * RPW + sub][vv * 8 + 2 * e] = dw.v[e].x;
        part[warp * RPW + sub][vv * 8 + 2 * e + 1] = dw.v[e].y;
      }
    }
    __syncthreads();
    if (threadIdx.x < D) {
      float t = 0.f;
#pragma unroll
      for (int i = 0; i < kRopeWarps * RPW; ++i) t += part[i][threadIdx.x];
      p.dw[((int64_t)blockIdx.x * 2 + side) * D + threadIdx.x] = t;
    }
  }
}

// Weight gradients: the sum of the CTAs' partial rows, one block per 32 columns of one
// side; 8 row threads a column, joined in one order.
template <int D>
__global__ void __launch_bounds__(256) qk_norm_rope_dw_kernel(const RopeParams p, int nparts) {
  __shared__ float part[8][33];
  const int side = blockIdx.y, col = blockIdx.x * 32 + (threadIdx.x & 31), r = threadIdx.x >> 5;
  float *dst = side == 0 ? p.dqw : p.dkw;
  if (!dst) return;
  float t = 0.f;
  if (col < D)
    for (int i = r; i < nparts; i += 8) t += p.dw[((int64_t)i * 2 + side) * D + col];
  part[r][threadIdx.x & 31] = t;
  __syncthreads();
  if (r == 0 && col < D) {
#pragma unroll
    for (int i = 1; i < 8; ++i) t += part[i][threadIdx.x];
    dst[col] = t;
  }
}

// ------------------------------------------------------------------ paged append

// Sequence of the token of the lane's row (token `first` + the row): the last s with
// cu[s] <= token (empty sequences are passed over), or -1 when the token lies behind the
// last sequence or before the first.  The warp's lanes read the offsets together.
__device__ __forceinline__ int sequence_of(const int32_t *cu, int batch, int lane, int rpw, int lpr,
                                           int first) {
  int mine = -1;
  for (int j0 = 0; j0 <= batch; j0 += 32) {
    const int c = j0 + lane <= batch ? __ldg(cu + j0 + lane) : 0x7fffffff;
    bool beyond = false;
    for (int r = 0; r < rpw; ++r) {
      const unsigned m = __ballot_sync(kFull, c <= first + r);
      if (r == min(lane / lpr, rpw - 1)) mine += __popc(m);
      beyond |= m == kFull;
    }
    if (!beyond) break;   // every later offset is above all of the warp's tokens
  }
  return mine < batch ? mine : -1;
}

// Heads of a token in the order queries, keys, values; a warp takes hpt of one of the three
// and the tokens of its rows.
template <int D>
__global__ void __launch_bounds__(kRopeThreads, 4) kv_append_kernel(const AppendParams p, int hpt) {
  constexpr int LPR = RowLanes<D>::LPR, RPW = RowLanes<D>::RPW;
  __shared__ uint4 slots[kRopeWarps][kRopeHeads * 32];
  const int lane = threadIdx.x & 31;
  const int sub = min(lane / LPR, RPW - 1), v = lane - sub * LPR, base = sub * LPR;
  const bool in = v < LPR;
  const int vv = in ? v : 0;
  const int cq = p.q.ptr ? (p.hq + hpt - 1) / hpt : 0;
  const int ck = (p.hkv + hpt - 1) / hpt;
  const int hc = (int)(blockIdx.x % (unsigned)(cq + 2 * ck));
  const long long t0 = ((long long)(blockIdx.x / (unsigned)(cq + 2 * ck)) * kRopeWarps + (threadIdx.x >> 5)) * RPW;
  if (t0 >= p.T) return;
  const int t = (int)t0 + sub;
  const int which = hc < cq ? 0 : (hc < cq + ck ? 1 : 2);   // q, k, v
  const RopeTensor src = which == 0 ? p.q : (which == 1 ? p.k : p.v);
  const RopeWeight wt = which == 0 ? p.qw : p.kw;
  const int h0 = (which == 0 ? hc : (which == 1 ? hc - cq : hc - cq - ck)) * hpt;
  const int nh = min(hpt, (which == 0 ? p.hq : p.hkv) - h0);
  bool live = in && t < p.T;
  {
    // (A lane without a token of its own reads the tensor's first.)
    const uint16_t *row = src.ptr + (live ? (int64_t)t * src.sn + vv * 8 : 0) + h0 * src.sh;
    for (int h = 0; h < nh; ++h) cp_async_16(lane_slot(slots[threadIdx.x >> 5], h), row + h * src.sh);
    cp_async_commit();
  }
  // The token's sequence and position, and its place in the pages (queries have none there,
  // but a token without one is left out whole).
  int seq = t, pos = 0, pid = -1, slot = 0;
  if (p.cu) seq = sequence_of(p.cu, p.batch, lane, RPW, LPR, (int)t0);
  live = live && seq >= 0 && seq < p.batch;
  if (live) {
    const int len = __ldg(p.seq_lens + seq);
    pos = p.cu ? len - __ldg(p.cu + seq + 1) + t : len - 1;
    if (pos >= 0 && pos < len && (!p.cosp || pos < p.max_pos)) {
      const int pg = pos / p.page;
      slot = pos - pg * p.page;
      if (pg < p.max_pages) pid = __ldg(p.table + (int64_t)seq * p.max_pages + pg);
    } else {
      pos = 0;
    }
  }
  // The angles are read while the page id is on its way.
  const Place pl = place_of(vv, lane, p.cosp ? p.rot : 0, p.interleaved);
  Vec8 cw, sw;
  if (which != 2) load_factors(pl, p.cosp, p.sinp, p.rot, pos, wt, vv, lane, cw, sw);
  if (live && (pid < 0 || pid >= p.num_pages)) {
    live = false;
    record_index_error(p.status, (32 * 16 + 3) * 256);
  }
  uint16_t *out;
  int64_t osh;
  if (which == 0) {
    out = p.qo.ptr + (int64_t)t * p.qo.sn;
    osh = p.qo.sh;
  } else {
    const RopeTensor dst = which == 1 ? p.kp : p.vp;
    out = dst.ptr + (int64_t)pid * dst.sb + (int64_t)slot * dst.sn;
    osh = dst.sh;
  }
  out += vv * 8 + h0 * osh;
  const uint4 *buf = slots[threadIdx.x >> 5];
  if (which == 2) {
    cp_async_wait_all();
    for (int h = 0; h < nh; ++h)
      if (live) *reinterpret_cast<uint4 *>(out + h * osh) = buf[h * 32 + lane];
    return;
  }
  cp_async_wait_all();
#pragma unroll 2
  for (int h = 0; h < nh; ++h) {
    const uint4 o = turn_row<D>(buf[h * 32 + lane], wt.ptr != nullptr, pl, p.interleaved, base, vv, p.eps, cw, sw);
    if (live) *reinterpret_cast<uint4 *>(out + h * osh) = o;
  }
}

// ------------------------------------------------------------------ launch

static unsigned rope_blocks(long long tasks) {
  return (unsigned)((tasks + kRopeWarps - 1) / kRopeWarps);
}

// Heads of a task: kRopeHeads, so that the angles serve as many rows; fewer where the whole
// call would not fill the GPU (148 SMs, 32 warps each) otherwise.
static int rope_heads(long long rows_per_head, int heads) {
  for (int hpt = kRopeHeads; hpt > 1; hpt /= 2)
    if (rows_per_head * ((heads + hpt - 1) / hpt) >= 148 * 32) return hpt;
  return 1;
}

template <int D>
static cudaError_t launch_rope_fwd_d(const RopeParams &p, cudaStream_t st) {
  const long long groups = (long long)((p.N + RowLanes<D>::RPW - 1) / RowLanes<D>::RPW) * p.batch;
  const int hpt = rope_heads(groups, p.hq + p.hkv);
  const long long chunks = (p.hq + hpt - 1) / hpt + (p.hkv + hpt - 1) / hpt;
  qk_norm_rope_fwd_kernel<D><<<(unsigned)(chunks * rope_blocks(groups)), kRopeThreads, 0, st>>>(p, hpt);
  return cudaGetLastError();
}

cudaError_t launch_rope_fwd(const RopeParams &p, int d, cudaStream_t st) {
  switch (d) {
    case 64: return launch_rope_fwd_d<64>(p, st);
    case 80: return launch_rope_fwd_d<80>(p, st);
    case 128: return launch_rope_fwd_d<128>(p, st);
  }
  return cudaErrorInvalidValue;
}

// CTAs of the backward, each with one partial row of weight gradients per side.
int rope_bwd_ctas(int batch, int hq, int hkv, int N, int d) {
  const long long rpw = 32 / (d / 8);
  const long long chunks = (hq > hkv ? hq : hkv) / (2 * kRopeRound) + 1;   // pairs of rounds of the larger side
  const long long blocks = (chunks * ((N + rpw - 1) / rpw) * batch + kRopeWarps - 1) / kRopeWarps;
  return (int)(blocks < kRopeBwdCtas ? blocks : kRopeBwdCtas);
}

template <int D>
static cudaError_t launch_rope_bwd_d(const RopeParams &p, int grid, cudaStream_t st) {
  constexpr int smem = kRopeWarps * 2 * 2 * kRopeRound * 32 * 16;
  cudaError_t e = cudaFuncSetAttribute(qk_norm_rope_bwd_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  qk_norm_rope_bwd_kernel<D><<<grid, kRopeThreads, smem, st>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess || (!p.dqw && !p.dkw)) return e;
  qk_norm_rope_dw_kernel<D><<<dim3((D + 31) / 32, 2), 256, 0, st>>>(p, grid);
  return cudaGetLastError();
}

cudaError_t launch_rope_bwd(const RopeParams &p, int d, int grid, cudaStream_t st) {
  switch (d) {
    case 64: return launch_rope_bwd_d<64>(p, grid, st);
    case 80: return launch_rope_bwd_d<80>(p, grid, st);
    case 128: return launch_rope_bwd_d<128>(p, grid, st);
  }
  return cudaErrorInvalidValue;
}

template <int D>
static cudaError_t launch_append_d(const AppendParams &p, cudaStream_t st) {
  const long long groups = (p.T + RowLanes<D>::RPW - 1) / RowLanes<D>::RPW;
  const int hpt = rope_heads(groups, (p.q.ptr ? p.hq : 0) + 2 * p.hkv);
  const long long ck = (p.hkv + hpt - 1) / hpt;
  const long long cq = p.q.ptr ? (p.hq + hpt - 1) / hpt : 0;
  kv_append_kernel<D><<<(unsigned)((cq + 2 * ck) * rope_blocks(groups)), kRopeThreads, 0, st>>>(p, hpt);
  return cudaGetLastError();
}

cudaError_t launch_append(const AppendParams &p, int d, cudaStream_t st) {
  switch (d) {
    case 64: return launch_append_d<64>(p, st);
    case 80: return launch_append_d<80>(p, st);
    case 128: return launch_append_d<128>(p, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace moba
