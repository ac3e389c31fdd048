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
// tokens; it walks a run of heads of these tokens with several rows in flight and keeps
// the angles (and weights) of its columns in registers meanwhile.  In the half layout a
// column's partner sits in another lane's vector: four shuffles of packed bf16 pairs fetch
// it, and the row sums are a butterfly of the same lanes.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "params.h"
#include "rows.cuh"

namespace moba {

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

// The partner's values of a packed row vector (zero where a column has none, so that
// infinities pass).
__device__ __forceinline__ void mate8(const Place &pl, int interleaved, const uint4 &a,
                                      const float (&x)[8], float (&y)[8]) {
  if (interleaved) {
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = x[e ^ 1];
  } else {
    uint4 b;
    b.x = __shfl_sync(kFull, a.x, pl.mate);
    b.y = __shfl_sync(kFull, a.y, pl.mate);
    b.z = __shfl_sync(kFull, a.z, pl.mate);
    b.w = __shfl_sync(kFull, a.w, pl.mate);
    unpack8(b, y);
  }
  if (pl.kind == 0) {
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = 0.f;
  }
}

// Normalise and rotate one row vector; w, wm: the weights of the lane's and of its
// partners' columns.
template <int D>
__device__ __forceinline__ uint4 turn_row(const uint4 &a, bool norm, const Place &pl, int interleaved,
                                          int base, int v, float eps, const float (&c)[8],
                                          const float (&s)[8], const float (&w)[8],
                                          const float (&wm)[8]) {
  float x[8], y[8], u[8];
  unpack8(a, x);
  mate8(pl, interleaved, a, x, y);
  if (norm) {
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
    const float r = rsqrtf(row_sum<D>(ss, base, v) * (1.f / D) + eps);
#pragma unroll
    for (int e = 0; e < 8; ++e) u[e] = fmaf(y[e] * wm[e], s[e], x[e] * w[e] * c[e]) * r;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) u[e] = fmaf(y[e], s[e], x[e] * c[e]);
  }
  return pack8(u);
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

// ------------------------------------------------------------------ forward

constexpr int kRopeHeads = 4;   // heads a warp walks, their rows in flight together

template <int D>
__global__ void __launch_bounds__(kRopeThreads) qk_norm_rope_fwd_kernel(const RopeParams p) {
  constexpr int LPR = RowLanes<D>::LPR, RPW = RowLanes<D>::RPW;
  const int lane = threadIdx.x & 31;
  const int sub = min(lane / LPR, RPW - 1), v = lane - sub * LPR, base = sub * LPR;
  const bool in = v < LPR;
  const int cq = (p.hq + kRopeHeads - 1) / kRopeHeads, ck = (p.hkv + kRopeHeads - 1) / kRopeHeads;
  const int groups = (p.N + RPW - 1) / RPW;
  const long long task = (long long)blockIdx.x * kRopeWarps + (threadIdx.x >> 5);
  const int hc = (int)(task % (cq + ck));
  const long long tg = task / (cq + ck);
  const int b = (int)(tg / groups);
  if (b >= p.batch) return;
  const int n = (int)(tg % groups) * RPW + sub;
  const bool isq = hc < cq;
  const RopeTensor src = isq ? p.q : p.k, dst = isq ? p.qo : p.ko;
  const RopeWeight wt = isq ? p.qw : p.kw;
  const int h0 = (isq ? hc : hc - cq) * kRopeHeads;
  const int nh = min(kRopeHeads, (isq ? p.hq : p.hkv) - h0);
  bool live = in && n < p.N;
  int pos = n;
  if (live && p.positions) pos = __ldg(p.positions + (int64_t)b * p.N + n);
  if (live && (pos < 0 || pos >= p.max_pos)) {
    live = false;
    record_index_error(p.status, (32 * 16 + 1) * 256);
  }
  const int vv = in ? v : 0;
  const Place pl = place_of(vv, lane, p.rot, p.interleaved);
  const uint16_t *row = src.ptr + b * src.sb + (int64_t)n * src.sn + vv * 8;
  uint16_t *out = dst.ptr + b * dst.sb + (int64_t)n * dst.sn + vv * 8;
  uint4 a[kRopeHeads];
#pragma unroll
  for (int i = 0; i < kRopeHeads; ++i) {
    a[i] = make_uint4(0, 0, 0, 0);
    if (live && i < nh) a[i] = __ldg(reinterpret_cast<const uint4 *>(row + (int64_t)(h0 + i) * src.sh));
  }
  float c[8], s[8], w[8], wm[8];
  load_angles(pl, p.cosp, p.sinp, p.rot, live ? pos : 0, c, s);
  const bool norm = wt.ptr != nullptr;
  load_weights(wt, pl, vv, lane, w, wm);
#pragma unroll
  for (int i = 0; i < kRopeHeads; ++i) {
    const uint4 o = turn_row<D>(a[i], norm, pl, p.interleaved, base, vv, p.eps, c, s, w, wm);
    if (live && i < nh) *reinterpret_cast<uint4 *>(out + (int64_t)(h0 + i) * dst.sh) = o;
  }
}

// ------------------------------------------------------------------ backward

// Persistent: a lane's columns are the same in all of its rows, so it sums their weight
// gradients in registers; the CTA's lanes of equal columns add up in one order and leave
// one partial row, which qk_norm_rope_dw_kernel sums over the CTAs (no atomics).
template <int D>
__global__ void __launch_bounds__(kRopeThreads, 2) qk_norm_rope_bwd_kernel(const RopeParams p) {
  constexpr int LPR = RowLanes<D>::LPR, RPW = RowLanes<D>::RPW;
  __shared__ float part[kRopeWarps * RPW][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = min(lane / LPR, RPW - 1), v = lane - sub * LPR, base = sub * LPR;
  const bool in = v < LPR;
  const int vv = in ? v : 0;
  const int cq = (p.hq + kRopeHeads - 1) / kRopeHeads, ck = (p.hkv + kRopeHeads - 1) / kRopeHeads;
  const int groups = (p.N + RPW - 1) / RPW;
  const Place pl = place_of(vv, lane, p.rot, p.interleaved);
  for (int side = 0; side < 2; ++side) {
    const bool isq = side == 0;
    const RopeTensor src = isq ? p.q : p.k, dst = isq ? p.qo : p.ko, up = isq ? p.gq : p.gk;
    const RopeWeight wt = isq ? p.qw : p.kw;
    const bool norm = wt.ptr != nullptr;
    const int heads = isq ? p.hq : p.hkv, chunks = isq ? cq : ck;
    float w[8], wm[8], dw[8];
    load_weights(wt, pl, vv, lane, w, wm);
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[e] = 0.f;
    const long long tasks = (long long)chunks * groups * p.batch;
    for (long long task = (long long)blockIdx.x * kRopeWarps + warp; task < tasks;
         task += (long long)gridDim.x * kRopeWarps) {
      const int h0 = (int)(task % chunks) * kRopeHeads;
      const long long tg = task / chunks;
      const int b = (int)(tg / groups), n = (int)(tg % groups) * RPW + sub;
      const int nh = min(kRopeHeads, heads - h0);
      bool live = in && n < p.N;
      int pos = n;
      if (live && p.positions) pos = __ldg(p.positions + (int64_t)b * p.N + n);
      if (live && (pos < 0 || pos >= p.max_pos)) {
        live = false;
        record_index_error(p.status, (32 * 16 + 2) * 256);
      }
      const uint16_t *grow = up.ptr + b * up.sb + (int64_t)n * up.sn + vv * 8;
      const uint16_t *xrow = src.ptr + b * src.sb + (int64_t)n * src.sn + vv * 8;
      uint16_t *out = dst.ptr + b * dst.sb + (int64_t)n * dst.sn + vv * 8;
      uint4 ga[kRopeHeads], xa[kRopeHeads];
#pragma unroll
      for (int i = 0; i < kRopeHeads; ++i) {
        ga[i] = xa[i] = make_uint4(0, 0, 0, 0);
        if (live && i < nh) {
          ga[i] = __ldg(reinterpret_cast<const uint4 *>(grow + (int64_t)(h0 + i) * up.sh));
          if (norm) xa[i] = __ldg(reinterpret_cast<const uint4 *>(xrow + (int64_t)(h0 + i) * src.sh));
        }
      }
      float c[8], s[8];
      load_angles(pl, p.cosp, p.sinp, p.rot, live ? pos : 0, c, s);
#pragma unroll
      for (int i = 0; i < kRopeHeads; ++i) {
        float dy[8], ym[8], g[8], x[8];
        unpack8(ga[i], dy);
        mate8(pl, p.interleaved, ga[i], dy, ym);
        // R^T: the sines turn their sign.
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] = fmaf(ym[e], -s[e], dy[e] * c[e]);
        if (norm) {
          unpack8(xa[i], x);
          float ss = 0.f, gx = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            ss = fmaf(x[e], x[e], ss);
            gx = fmaf(g[e] * w[e], x[e], gx);
          }
          ss = row_sum<D>(ss, base, vv);
          gx = row_sum<D>(gx, base, vv);
          const float r = rsqrtf(ss * (1.f / D) + p.eps);
          const float m = gx * (1.f / D) * r * r;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            dw[e] = fmaf(g[e] * r, x[e], dw[e]);
            g[e] = r * fmaf(-m, x[e], g[e] * w[e]);
          }
        }
        if (live && i < nh) *reinterpret_cast<uint4 *>(out + (int64_t)(h0 + i) * dst.sh) = pack8(g);
      }
    }
    if (!norm) continue;   // (uniform over the grid)
    __syncthreads();
    if (in) {
#pragma unroll
      for (int e = 0; e < 8; ++e) part[warp * RPW + sub][vv * 8 + e] = dw[e];
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

// Heads of a token in the order queries, keys, values; a warp takes kRopeHeads of one of
// the three and the tokens of its rows.
template <int D>
__global__ void __launch_bounds__(kRopeThreads) kv_append_kernel(const AppendParams p) {
  constexpr int LPR = RowLanes<D>::LPR, RPW = RowLanes<D>::RPW;
  const int lane = threadIdx.x & 31;
  const int sub = min(lane / LPR, RPW - 1), v = lane - sub * LPR, base = sub * LPR;
  const bool in = v < LPR;
  const int vv = in ? v : 0;
  const int cq = p.q.ptr ? (p.hq + kRopeHeads - 1) / kRopeHeads : 0;
  const int ck = (p.hkv + kRopeHeads - 1) / kRopeHeads;
  const long long task = (long long)blockIdx.x * kRopeWarps + (threadIdx.x >> 5);
  const int hc = (int)(task % (cq + 2 * ck));
  const long long t0 = task / (cq + 2 * ck) * RPW;
  if (t0 >= p.T) return;
  const int t = (int)t0 + sub;
  const int which = hc < cq ? 0 : (hc < cq + ck ? 1 : 2);   // q, k, v
  const RopeTensor src = which == 0 ? p.q : (which == 1 ? p.k : p.v);
  const RopeWeight wt = which == 0 ? p.qw : p.kw;
  const int h0 = (which == 0 ? hc : (which == 1 ? hc - cq : hc - cq - ck)) * kRopeHeads;
  const int nh = min(kRopeHeads, (which == 0 ? p.hq : p.hkv) - h0);
  bool live = in && t < p.T;
  uint4 a[kRopeHeads];
  {
    const uint16_t *row = src.ptr + (int64_t)t * src.sn + vv * 8;
#pragma unroll
    for (int i = 0; i < kRopeHeads; ++i) {
      a[i] = make_uint4(0, 0, 0, 0);
      if (live && i < nh) a[i] = __ldg(reinterpret_cast<const uint4 *>(row + (int64_t)(h0 + i) * src.sh));
    }
  }
  // The token's sequence and position, and its place in the pages.
  int seq = t, pos = 0, pid = 0, slot = 0;
  if (p.cu) seq = sequence_of(p.cu, p.batch, lane, RPW, LPR, (int)t0);
  live = live && seq >= 0 && seq < p.batch;
  if (live) {
    const int len = __ldg(p.seq_lens + seq);
    pos = p.cu ? len - __ldg(p.cu + seq + 1) + t : len - 1;
    bool ok = pos >= 0 && pos < len && (!p.cosp || pos < p.max_pos);
    if (ok && which != 0) {
      const int pg = pos / p.page;
      slot = pos - pg * p.page;
      ok = pg < p.max_pages;
      if (ok) {
        pid = __ldg(p.table + (int64_t)seq * p.max_pages + pg);
        ok = pid >= 0 && pid < p.num_pages;
      }
    }
    if (!ok) {
      live = false;
      record_index_error(p.status, (32 * 16 + 3) * 256);
    }
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
  if (which == 2) {
#pragma unroll
    for (int i = 0; i < kRopeHeads; ++i)
      if (live && i < nh) *reinterpret_cast<uint4 *>(out + i * osh) = a[i];
    return;
  }
  const Place pl = place_of(vv, lane, p.cosp ? p.rot : 0, p.interleaved);
  float c[8], s[8], w[8], wm[8];
  load_angles(pl, p.cosp, p.sinp, p.rot, live ? pos : 0, c, s);
  load_weights(wt, pl, vv, lane, w, wm);
#pragma unroll
  for (int i = 0; i < kRopeHeads; ++i) {
    const uint4 o = turn_row<D>(a[i], wt.ptr != nullptr, pl, p.interleaved, base, vv, p.eps, c, s, w, wm);
    if (live && i < nh) *reinterpret_cast<uint4 *>(out + i * osh) = o;
  }
}

// ------------------------------------------------------------------ launch

static unsigned rope_blocks(long long tasks) {
  return (unsigned)((tasks + kRopeWarps - 1) / kRopeWarps);
}

template <int D>
static cudaError_t launch_rope_fwd_d(const RopeParams &p, cudaStream_t st) {
  const long long chunks = (p.hq + kRopeHeads - 1) / kRopeHeads + (p.hkv + kRopeHeads - 1) / kRopeHeads;
  const long long groups = (p.N + RowLanes<D>::RPW - 1) / RowLanes<D>::RPW;
  qk_norm_rope_fwd_kernel<D><<<rope_blocks(chunks * groups * p.batch), kRopeThreads, 0, st>>>(p);
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
  const long long chunks = (hq + kRopeHeads - 1) / kRopeHeads + (hkv + kRopeHeads - 1) / kRopeHeads;
  const long long blocks = (chunks * ((N + rpw - 1) / rpw) * batch + kRopeWarps - 1) / kRopeWarps;
  return (int)(blocks < kRopeBwdCtas ? blocks : kRopeBwdCtas);
}

template <int D>
static cudaError_t launch_rope_bwd_d(const RopeParams &p, int grid, cudaStream_t st) {
  qk_norm_rope_bwd_kernel<D><<<grid, kRopeThreads, 0, st>>>(p);
  cudaError_t e = cudaGetLastError();
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
  const long long ck = (p.hkv + kRopeHeads - 1) / kRopeHeads;
  const long long cq = p.q.ptr ? (p.hq + kRopeHeads - 1) / kRopeHeads : 0;
  const long long groups = (p.T + RowLanes<D>::RPW - 1) / RowLanes<D>::RPW;
  kv_append_kernel<D><<<rope_blocks((cq + 2 * ck) * groups), kRopeThreads, 0, st>>>(p);
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
