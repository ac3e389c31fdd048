// params.h -- problem description, workspace layout and kernel parameter blocks
// shared by the host-side ABI and the kernels.
#pragma once

#include <stddef.h>
#include <stdint.h>
#include <vector_types.h>

namespace moba {

constexpr int kTileRows = 128;   // query rows per attention tile (tcgen05 M)
constexpr int kUnitRows = 256;   // list entries per gathered work unit (two tiles)
constexpr int kTileKeys = 128;   // keys per attention chunk (tcgen05 N of S = QK^T)
constexpr size_t kPartialCapBytes = size_t(4) << 30;  // partial outputs kept per pass

// Block-major dispatch lists and partial outputs, carved out of the caller's workspace.
// List L = ((chunk * batch + b) * hkv + hk) * nblk + j holds the (row, q-head, slot)
// triples of the rows of query chunk `chunk` that picked past block j.
struct WorkspaceLayout {
  int nblk;         // ceil((q_off + N) / block): a partial last block when block does not
                    // divide the key count
  int G;            // hq / hkv
  int npast;        // topk - 1: partial slots per row
  int chunk_rows;   // query rows per pass (multiple of 128)
  int nchunks;
  int nlists;       // nchunks * batch * hkv * nblk
  size_t off_counts;   // int32 [nlists + 2]   entries per list (atomic counts), then the
                       //                      gate's tile counter and finished-CTA count
  size_t off_cursor;   // int32 [nlists]       scatter cursors
  size_t off_listoff;  // int32 [nlists + 1]   exclusive prefix of counts
  size_t off_tileoff;  // int32 [nlists + 1]   exclusive prefix of ceil(count / 256)
  size_t off_entries;  // uint32 [max_entries] entry = (i * G + g) * npast + slot
  size_t off_tiles;    // int4 [max_tiles]      per 256-entry unit: list, first entry, rows
  size_t off_opart;    // bf16 [batch, hq, chunk_rows, topk, d]: slots 0..npast-1 past
                       //      blocks, slot npast the own block
  size_t off_lpart;    // f32  [batch, hq, chunk_rows, topk]
  size_t total;
  long long max_entries;
  long long max_tiles;
};

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// N query rows; the keys run over q_off + N positions (q_off > 0: a chunk of a longer
// prefill whose queries are the last N positions).
inline WorkspaceLayout make_layout(int batch, int hq, int hkv, int N, int d, int block,
                                   int topk, int q_off = 0) {
  WorkspaceLayout w{};
  w.nblk = (q_off + N + block - 1) / block;
  w.G = hq / hkv;
  w.npast = topk - 1;
  // Partials exist only when a row can attend past blocks: topk slots per row then.
  const size_t nslots = w.npast > 0 ? size_t(topk) : 0;
  const size_t per_row = nslots * (size_t(d) * 2 + 4) * size_t(batch) * size_t(hq);
  long long rows = N;
  if (per_row > 0 && per_row * size_t(N) > kPartialCapBytes) {
    rows = static_cast<long long>(kPartialCapBytes / per_row) / kTileRows * kTileRows;
    if (rows < kTileRows) rows = kTileRows;
  }
  w.chunk_rows = static_cast<int>(rows);
  w.nchunks = static_cast<int>((N + w.chunk_rows - 1) / w.chunk_rows);
  w.nlists = w.nchunks * batch * hkv * w.nblk;
  w.max_entries = static_cast<long long>(batch) * hq * N * w.npast;
  w.max_tiles = w.max_entries / kUnitRows + w.nlists + 1;
  size_t off = 0;
  w.off_counts = off;  off = align_up(off + sizeof(int) * size_t(w.nlists + 2), 256);
  w.off_cursor = off;  off = align_up(off + sizeof(int) * size_t(w.nlists), 256);
  w.off_listoff = off; off = align_up(off + sizeof(int) * size_t(w.nlists + 1), 256);
  w.off_tileoff = off; off = align_up(off + sizeof(int) * size_t(w.nlists + 1), 256);
  w.off_entries = off; off = align_up(off + sizeof(uint32_t) * size_t(w.max_entries), 256);
  w.off_tiles = off;   off = align_up(off + 16 * size_t(w.max_tiles), 256);
  const size_t prow = size_t(batch) * hq * size_t(w.chunk_rows) * nslots;
  w.off_opart = off;   off = align_up(off + prow * size_t(d) * 2, 256);
  w.off_lpart = off;   off = align_up(off + prow * sizeof(float), 256);
  w.total = off;
  return w;
}

// Parameters of the gate / top-k kernel.
struct SelectParams {
  const uint16_t *q;     // bf16 bits
  int64_t q_sb, q_sh, q_sn;
  const uint16_t *kbar_split;  // [batch, hkv, 2, nblk, d]
  int32_t *idx;          // [batch, hq, N, topk]
  int *counts;           // workspace list counts
  int batch, hq, hkv, N, d, block, topk, nblk, G, chunk_rows;
  int q_off;             // position of query row 0 among the keys
  int minmax;            // 1: the planes are block maxima and minima (min/max pooling), and
                         // the score is q+ . kmax + q- . kmin; 0: hi + lo of the means
};

// Parameters of the tensor-core gate / top-k kernel (q and the pooled keys arrive
// through TMA maps).
struct GateParams {
  int *status;           // device status words
  int32_t *idx;          // [batch, hq, N, topk]
  int *counts;           // workspace list counts
  int batch, hq, hkv, N, d, block, topk, nblk, G, chunk_rows;
  int q_off;             // position of query row 0 among the keys
  int qstages;           // query tile ring depth (set by the launcher)
  int kslots;            // pooled-key staging slots, 1 or 2 (set by the launcher)
  int *sched;            // tile counter, zero at launch (the word after the list counts)
  int chunk_tiles;       // tiles per chunk taken from it (set by the launcher)
  // When done is set (zero at launch, the second word after the counts), the last
  // CTA to finish writes the list offsets (cursor, listoff, tileoff over nlists).
  int *done;
  int *cursor, *listoff, *tileoff;
  int nlists;
};

struct ScatterParams {
  const int32_t *idx;
  int *cursor;
  uint32_t *entries;
  int batch, hq, hkv, N, block, topk, nblk, G, chunk_rows;
  int q_off;               // position of query row 0 among the keys
  // Unit table (written by the scatter grid from the scanned offsets).
  const int *counts;
  const int *listoff;
  const int *tileoff;
  int4 *tiles;
  int nlists;
  int cache_rows;          // 1: the CTA's block choices are staged in shared memory
};

// Attention kernel modes.
enum AttnMode : int {
  kQueryMajor = 0,  // contiguous 128-row query tiles: own block (MoBA) or band (SWA)
  kGathered = 1,    // gathered rows of one block-major list against one whole block
};

struct AttnParams {
  int *status;             // device status words (see common.cuh)
  // Tensors (bf16 bits) and strides in elements.
  const uint16_t *q;
  int64_t q_sb, q_sh, q_sn;
  uint16_t *out;
  int64_t o_sb, o_sh, o_sn;
  float *lse;              // [batch, hq, N]
  const int32_t *idx;      // [batch, hq, N, topk] (MoBA) or null (SWA)
  // Problem: N query rows; keys and values run over q_off + N positions, query row i
  // sits at position q_off + i.
  int batch, hq, hkv, N, d, block, topk, window, G;
  int sink;                // swa_fwd.cu: keys [0, sink) stay visible behind the window
  int q_off;
  float scale_log2;        // scale * log2(e)
  int is_moba;             // 0: sliding window only (swa_attn_fwd)
  // Gathered pass: 1 when the query rows are fetched by TMA gather4 through a 2-D map
  // over q (row ((b * hq + h) * N + i)); 0 when by cp.async (q's strides admit no
  // single row stride, or the row count exceeds int32).
  int q_gather_tma;
  // Query-major pass: row range of this pass.
  int row_begin, row_end;  // multiples of 128 except row_end == N (any N)
  int ntiles;              // query-major work units in this pass
  // Block-major lists and partials (MoBA).
  const int *listoff;
  const int *tileoff;
  const int4 *tiles;       // per gathered unit: list, first entry, rows (<= 256)
  const uint32_t *entries;
  uint16_t *opart;         // [batch, hq, chunk_rows, topk, d]
  float *lpart;            // [batch, hq, chunk_rows, topk]
  int chunk, chunk_rows, npast, nblk, lists_per_chunk;
};

// Parameters of the merge pass (one query chunk).
struct MergeParams {
  const uint16_t *opart;   // [batch, hq, chunk_rows, topk, d]
  const float *lpart;      // [batch, hq, chunk_rows, topk]
  const int32_t *idx;      // [batch, hq, N, topk]
  uint16_t *out;
  int64_t o_sb, o_sh, o_sn;
  float *lse;              // [batch, hq, N]
  int batch, hq, N, d, block, topk, chunk_rows, row_begin, row_end;
  int q_off;               // position of query row 0 among the keys
};

// Parameters of the backward kernels (bwd.cu).
struct BwdParams {
  int *status;             // device status words
  const uint16_t *q, *out, *dout;
  int64_t q_sb, q_sh, q_sn, o_sb, o_sh, o_sn, do_sb, do_sh, do_sn;
  const float *lse;        // [batch, hq, N] (natural log)
  uint16_t *dq, *dk, *dv;
  int64_t dq_sb, dq_sh, dq_sn, dk_sb, dk_sh, dk_sn, dv_sb, dv_sh, dv_sn;
  float2 *rowstat;         // [batch, hq, N]: lse * log2(e), D = dO . o
  float *dqp;              // [batch, hq, N, topk, d] fp32 partial dQ per block slot
  int batch, hq, hkv, N, d, block, topk, npast, nblk, G, nchunks, nlists;
  float scale, scale_log2;
  // Dispatch lists of the forward's selection step (its workspace).
  const uint32_t *entries;
  const int4 *tiles;
  const int *tileoff, *listoff;
};

// Bytes of the backward's own workspace: the row statistics, then the dQ partials.
inline size_t bwd_workspace_bytes(int batch, int hq, int N, int d, int topk, size_t *off_dqp) {
  const size_t rows = size_t(batch) * hq * size_t(N);
  const size_t a = align_up(rows * 8, 256);
  if (off_dqp) *off_dqp = a;
  return a + align_up(rows * size_t(topk) * size_t(d) * 4, 256);
}

constexpr int kRopeBwdCtas = 296;  // most CTAs (partial weight-gradient rows) of the norm + rotary backward

// Parameters of the per-head norm + rotary kernels (rope.cu).  Rows are (b, head, n);
// strides in elements.
struct RopeTensor {
  uint16_t *ptr;           // bf16 bits
  int64_t sb, sh, sn;
};

// A per-head weight of D values, bf16 or float32 (null: no norm).
struct RopeWeight {
  const void *ptr;
  int f32;
};

struct RopeParams {
  int *status;
  RopeTensor q, k;         // inputs (the forward's x)
  RopeTensor qo, ko;       // outputs: the rotated rows, or (backward) dq, dk
  RopeTensor gq, gk;       // backward: upstream gradients of the rotated rows
  RopeWeight qw, kw;
  const float *cosp, *sinp;  // [max_pos, rot / 2]
  const int32_t *positions;  // [batch, N], or null: position n
  int batch, hq, hkv, N;
  int rot, max_pos, interleaved;
  float eps;
  float *dw;               // backward: partial weight gradients [grid, 2, D]
  float *dqw, *dkw;        // backward: weight gradients [D] (null where there is no norm)
};

// Parameters of the paged append (rope.cu): tokens t of sequence s are
// cu[s] .. cu[s + 1] - 1 and sit at the last positions below seq_lens[s].
struct AppendParams {
  int *status;
  RopeTensor q, k, v;      // new tokens [T, heads, D] (sb unused); q.ptr may be null
  RopeTensor qo;           // rotated queries
  RopeTensor kp, vp;       // pages: sb page, sh KV head, sn slot
  RopeWeight qw, kw;
  const float *cosp, *sinp;  // null: no rotation
  const int32_t *cu;       // [batch + 1], or null: one token per sequence
  const int32_t *seq_lens; // [batch]
  const int32_t *table;    // [batch, max_pages]
  int batch, T, hq, hkv;
  int rot, max_pos, interleaved;
  int page, num_pages, max_pages;
  float eps;
};

// Parameters of the paged decode (decode.cu).  One query token per sequence, at the last
// of its seq_lens[b] positions.
constexpr int kDecodeCtas = 444;      // most CTAs of the main kernel (three per SM)
constexpr int kDecodeRows = 16;       // query heads of one KV head a CTA takes together
struct DecodeParams {
  int *status;
  const uint16_t *q;       // [batch, hq, D]
  int64_t q_sb, q_sh;
  uint16_t *out;
  int64_t o_sb, o_sh;
  float *lse;              // [batch, hq]
  RopeTensor kp, vp;       // pages: sb page, sh KV head, sn slot
  const int32_t *seq_lens; // [batch]
  const int32_t *table;    // [batch, max_pages]
  int batch, hq, hkv, G, ngrp;   // ngrp: groups of kDecodeRows query heads per KV head
  int page, num_pages, max_pages;
  int window, sink;
  float scale_log2;
  // Workspace: work (in tiles) before each sequence [batch + 1], then the partial results: per CTA
  // two slots (its first and its last item) of kDecodeRows rows of D values and their LSE.
  int *before;
  float *opart;            // [ctas, 2, kDecodeRows, D]
  float *lpart;            // [ctas, 2, kDecodeRows]
};

inline size_t decode_workspace_bytes(int batch, int d, size_t *off_o, size_t *off_l) {
  size_t off = align_up(sizeof(int) * (size_t(batch) + 1), 256);
  const size_t rows = size_t(kDecodeCtas) * 2 * kDecodeRows;
  if (off_o) *off_o = off;
  off = align_up(off + rows * size_t(d) * 4, 256);
  if (off_l) *off_l = off;
  return align_up(off + rows * 4, 256);
}

// Parameters of the sliding-window backward (swa_bwd.cu).
struct SwaBwdParams {
  int *status;
  const uint16_t *out, *dout;
  int64_t o_sb, o_sh, o_sn, do_sb, do_sh, do_sn;
  const float *lse;        // [batch, hq, N] (natural log)
  uint16_t *dq, *dk, *dv;
  int64_t dq_sb, dq_sh, dq_sn, dk_sb, dk_sh, dk_sn, dv_sb, dv_sh, dv_sn;
  float *stat;             // [batch, hq, nt, 2, 128]: -lse * log2(e), -D = -dO . o of a tile's
                           // rows (behind row N: -inf, 0)
  uint16_t *extra;         // [batch, hq, nt, 128, 16]: the same statistics as bf16 columns of
                           // the products (swizzled rows of 32 bytes)
  float *part;             // dK, dV of the sinks' key tiles in parts:
                           // [batch, hkv, nst, 1 + nseg, 2, 128, D]
  int batch, hq, hkv, N, d, window, sink, G;
  int nt;                  // 128-row tiles of N
  int nst;                 // key tiles that hold sinks, 0 when no row sees one behind its band
  int seg, nseg;           // query tiles of a far part, most far parts of a key tile
  float scale, scale_log2;
};

// Query tiles of one head that a key tile's band reaches: kt .. swa_last_tile.
__host__ __device__ inline int swa_last_tile(int kt, int window, int nt) {
  const long long last = ((long long)kt * kTileKeys + kTileKeys - 1 + window - 1) / kTileRows;
  return last < nt - 1 ? (int)last : nt - 1;
}

// Split of the sinks' walks and the workspace of the sliding-window backward.  A key tile
// with sinks is attended by the query tiles of its band, like every key tile, and by all
// later ones; these are cut into parts of `seg` query tiles (of all G heads) so that no
// part is much longer than a band's walk.
struct SwaBwdPlan {
  int nt, nst, seg, nseg;
  size_t off_extra, off_part, total;
};

inline SwaBwdPlan swa_bwd_plan(int batch, int hq, int hkv, int N, int d, int window, int sink) {
  SwaBwdPlan w{};
  w.nt = (N + kTileRows - 1) / kTileRows;
  const int G = hq / hkv;
  const long long far0 = (long long)G * (w.nt - 1 - swa_last_tile(0, window, w.nt));
  if (sink > 0 && far0 > 0) {
    const int s = sink < N ? sink : N;
    w.nst = (s + kTileKeys - 1) / kTileKeys;
    // At least a band's walk (or 16 tiles) a part, and about eight parts per SM at most.
    long long seg = (long long)G * (window / kTileRows + 2);
    if (seg < 16) seg = 16;
    const long long all = far0 * w.nst * hkv * batch;
    if (seg < all / 1184) seg = all / 1184;
    if (seg > far0) seg = far0;
    w.seg = (int)seg;
    w.nseg = (int)((far0 + seg - 1) / seg);
  }
  size_t off = align_up(size_t(batch) * hq * w.nt * 2 * kTileRows * 4, 1024);
  w.off_extra = off;
  off = align_up(off + size_t(batch) * hq * w.nt * kTileRows * 32, 1024);
  w.off_part = off;
  off += size_t(batch) * hkv * w.nst * (1 + w.nseg) * 2 * kTileKeys * d * 4;
  w.total = align_up(off, 256);
  return w;
}

}  // namespace moba
