// The line of key tiles that attention over the paged cache works through, and
// the end of its pieces (see attn_tree_kernel.cuh).
#pragma once

#include "attn_tree_kernel.cuh"

namespace attn {
namespace tree {

// The work of a launch as one line of key tiles, cut into equal shares: for
// sequence after sequence, for each group of its key heads and row tile (a
// segment), its key tiles.  Every unit (`heads` warps, one to a head of the
// group) takes `share` consecutive tiles, whatever segments they fall in, so
// ragged lengths leave no SM idle at the end.  A segment inside one share is
// written as the result; the pieces of a segment that shares cut go to the
// workspace, two slots a unit (slot 0: a piece that begins with the unit's share,
// slot 1: one that begins inside it) for each of its heads, and the join kernel
// finds them again by the same arithmetic.
struct Work {
  int rows;       // query rows of a segment's tile
  int heads;      // key heads of a segment
  int log_tile;   // log2 of the keys of a tile
  int min_share;  // tiles
  int units;
};

__device__ __forceinline__ int seq_tiles(const Seq& s, const Work& w) {
  return (int)(((int64_t)s.len + (1 << w.log_tile) - 1) >> w.log_tile);
}
__device__ __forceinline__ int seq_segments(const Params& p, const Seq& s, const Work& w) {
  return (s.n * p.G + w.rows - 1) / w.rows * (p.H / w.heads);
}
// Tiles of sequence b in the line; 0 if it has no new token or impossible lengths.
__device__ __forceinline__ int64_t line_tiles(const Params& p, const Work& w, int b, bool report) {
  Seq s;
  if (!load_seq(p, b, s)) {
    if (report) atomicOr(p.err, rows::kBadSeqlens);
    return 0;
  }
  return (int64_t)seq_segments(p, s, w) * seq_tiles(s, w);
}
__device__ __forceinline__ int64_t share_of(int64_t total, const Work& w) {
  const int64_t even = (total + w.units - 1) / w.units;
  return even > w.min_share ? even : w.min_share;
}

// Where a unit is in the line: sequence b (lengths in s), segment seg of it, tile
// of that, and how many tiles of its share are left.
struct Walk {
  int b, seg, segs, tile, tiles;
  int64_t left;
  Seq s;
  __device__ __forceinline__ void enter(const Params& p, const Work& w) {
    if (load_seq(p, b, s)) {
      segs = seq_segments(p, s, w);
      tiles = seq_tiles(s, w);
    } else {
      segs = tiles = 0;
    }
  }
  // tiles of the current segment that belong to the share
  __device__ __forceinline__ int piece() const { return (int)(tiles - tile < left ? tiles - tile : left); }
  // behind the piece; false at the end of the share
  __device__ __forceinline__ bool next(const Params& p, const Work& w) {
    left -= piece();
    if (left <= 0) return false;
    tile = 0;
    if (++seg < segs) return true;
    seg = 0;
    do {
      if (++b >= p.B) return false;
      enter(p, w);
    } while (segs == 0 || tiles == 0);
    return true;
  }
};

// A unit's place in the line, found by each of its warps: lane t sums the tiles
// of its block of sequences, the sums are scanned, and the lane whose block holds
// the first tile of the share walks to it.  False: nothing to do.
__device__ __forceinline__ bool find_place(const Params& p, const Work& w, int unit, bool report, Walk& walk) {
  const int t = threadIdx.x % 32, per = (p.B + 31) / 32;
  const int b0 = (int)min((int64_t)t * per, (int64_t)p.B), b1 = min(p.B - b0, per) + b0;
  int64_t mine = 0;
  for (int b = b0; b < b1; ++b) mine += line_tiles(p, w, b, report);
  int64_t upto = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, upto, off);
    if (t >= off) upto += v;
  }
  const int64_t total = __shfl_sync(0xffffffffu, upto, 31), before = upto - mine;
  const int64_t share = share_of(total, w), first = share * unit;
  if (first >= total) return false;
  walk = Walk{};
  int64_t at = 0;
  const bool here = first >= before && first < upto;
  if (here) {
    at = first - before;
    for (walk.b = b0;; ++walk.b) {
      const int64_t n = line_tiles(p, w, walk.b, false);
      if (at < n) break;
      at -= n;
    }
  }
  const int src = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
  walk.b = __shfl_sync(0xffffffffu, walk.b, src);
  at = __shfl_sync(0xffffffffu, at, src);
  walk.enter(p, w);
  walk.seg = (int)(at / walk.tiles);
  walk.tile = (int)(at - (int64_t)walk.seg * walk.tiles);
  walk.left = min(share, total - first);
  return true;
}

// The end of a piece: a warp writes kCols columns from col0 on of its kRows query
// rows (sums at buf[r pad], maximum and sum at sm_m, sm_l[r]), as the result where
// the piece is the whole segment (slot < 0), else into its slot of the workspace.
template <int D, bool kCodes, int kRows, int kCols>
__device__ __forceinline__ void write_piece(const Params& p, const Seq& sq, int b, int h, int row0, int slot,
                                            const float* buf, int pad, int col0, const float* sm_m,
                                            const float* sm_l, uint64_t hid, bool poison, int lane) {
  const int ctx = sq.len - sq.n, M = sq.n * p.G;
  constexpr int kVec = kCols / 4;  // lanes of a row, four columns each
  for (int i = lane; i < kRows * kVec; i += 32) {
    const int r = i / kVec, at_col = 4 * (i % kVec), col = col0 + at_col;
    if (row0 + r >= M) continue;
    const int tok = (row0 + r) / p.G, head = h * p.G + (row0 + r) - tok * p.G;
    const float mm = sm_m[r], ls = mm == -INFINITY ? 0.f : sm_l[r];
    const float4 x = *reinterpret_cast<const float4*>(buf + r * pad + at_col);
    float f[4] = {x.x, x.y, x.z, x.w};
    // a row of NaN sums keeps them; one that saw nothing is 0
    const float inv = ls != 0.f ? 1.f / ls : 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) f[k] = ls != 0.f ? f[k] * inv : 0.f;
    float lse = ls != 0.f ? (mm + lg2(ls)) * 0.69314718055994531f : -INFINITY;
    if (hid) {
      uint64_t todo = hid & mask_word(p.mask, sq.q0 + tok, tok);
      while (todo) {
        const int t = __ffsll((long long)todo) - 1;
        todo &= todo - 1;
        const int pos = ctx + t;
        const int id = p.table[(int64_t)b * p.stride + (pos >> p.log_page)];
        if ((unsigned)id >= (unsigned)p.pages) continue;
        const int64_t at = ((((int64_t)id << p.log_page) + (pos & ((1 << p.log_page) - 1))) * p.H + h) * D + col;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (kCodes) {
            const uint8_t x = reinterpret_cast<const uint8_t*>(p.v)[at + k];
            if ((x & 0x7f) == 0x7f) f[k] = NAN;
          } else {
            const float x = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p.v)[at + k]);
            if (!isfinite(x)) f[k] += x;
          }
        }
      }
    }
    if (poison) {  // a NaN row; +inf makes the merge of the pieces one
      f[0] = f[1] = f[2] = f[3] = NAN;
      lse = slot < 0 ? NAN : INFINITY;
    }
    if (slot < 0) {
      const int64_t out = (int64_t)(sq.q0 + tok) * p.Hq + head;
      *reinterpret_cast<uint2*>(p.o + out * D + col) =
          make_uint2(rows::pack2(f[0], f[1]), rows::pack2(f[2], f[3]));
      if (col == 0) p.lse[out] = lse;
    } else {
      const int64_t at = (int64_t)slot * kRows + r;
      *reinterpret_cast<float4*>(p.o_part + at * D + col) = make_float4(f[0], f[1], f[2], f[3]);
      if (col == 0) p.lse_part[at] = lse;
    }
  }
}

// Pieces of a row joined: weights e^(LSE - max), as for split keys elsewhere in
// the library.  kPerRow warps for each (new token, query head): one, or eight
// where segments are cut into many pieces; warp k takes pieces k, k + kPerRow, ..
// Rows whose segment lies in one share (or whose sequence the attention refused)
// are left as they are.
template <int D, int kPerRow>
__global__ void __launch_bounds__(256) tree_join_kernel(const __grid_constant__ Params p, const __grid_constant__ Work w) {
  constexpr int kPer = D / 32;
  __shared__ float sm_sum[8], sm_acc[8][D];
  grid_dep_wait();
  grid_dep_launch();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, k = warp % kPerRow;
  const int64_t rowi = ((int64_t)blockIdx.x * 8 + warp) / kPerRow;
  if (rowi >= (int64_t)p.total * p.Hq) return;  // with eight warps to a row, the whole CTA
  const int t = (int)(rowi / p.Hq), head = (int)(rowi - (int64_t)t * p.Hq);
  const int b = rows::find_sequence(p.cu, p.B, t);
  if (b >= p.B) return;
  Seq sq;
  if (!load_seq(p, b, sq) || t < sq.q0 || t >= sq.q0 + sq.n) return;
  int64_t total = 0, before = 0;
  for (int i = lane; i < p.B; i += 32) {
    const int64_t n = line_tiles(p, w, i, false);
    total += n;
    before += i < b ? n : 0;
  }
#pragma unroll
  for (int off = 16; off; off >>= 1) {
    total += __shfl_xor_sync(0xffffffffu, total, off);
    before += __shfl_xor_sync(0xffffffffu, before, off);
  }
  const int h = head / p.G, row = (t - sq.q0) * p.G + head - h * p.G;
  const int group = h / w.heads, sub = h - group * w.heads;
  const int mtiles = (sq.n * p.G + w.rows - 1) / w.rows, mt = row / w.rows, r = row - mt * w.rows;
  const int64_t share = share_of(total, w), tiles = seq_tiles(sq, w);
  const int64_t first = before + ((int64_t)group * mtiles + mt) * tiles;
  const int c0 = (int)(first / share), c1 = (int)((first + tiles - 1) / share);
  if (c0 == c1) return;
  const bool inside = first % share != 0;  // the first piece begins inside its share
  auto at = [&](int c) { return (((int64_t)2 * c + (c == c0 && inside)) * w.heads + sub) * w.rows + r; };
  float top = -INFINITY;
  for (int c = c0 + lane; c <= c1; c += 32) top = fmaxf(top, p.lse_part[at(c)]);
#pragma unroll
  for (int off = 16; off; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
  float acc[kPer], sum = 0.f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) acc[i] = 0.f;
#pragma unroll 4
  for (int c = c0 + k; c <= c1; c += kPerRow) {
    const float ls = p.lse_part[at(c)];
    float x[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) x[i] = p.o_part[at(c) * D + lane * kPer + i];
    if (ls == -INFINITY) continue;
    const float wt = __expf(ls - top);  // a NaN stays one: fmaxf has passed it over
    sum += wt;
#pragma unroll
    for (int i = 0; i < kPer; ++i) acc[i] = fmaf(wt, x[i], acc[i]);
  }
  if (kPerRow > 1) {  // the row's warps are the CTA's
    if (lane == 0) sm_sum[k] = sum;
#pragma unroll
    for (int i = 0; i < kPer; ++i) sm_acc[k][lane * kPer + i] = acc[i];
    __syncthreads();
    if (k != 0) return;
    for (int j = 1; j < kPerRow; ++j) {
      sum += sm_sum[j];
#pragma unroll
      for (int i = 0; i < kPer; ++i) acc[i] += sm_acc[j][lane * kPer + i];
    }
  }
  const float inv = sum != 0.f ? 1.f / sum : 0.f;
  __nv_bfloat16* dst = p.o + rowi * D + lane * kPer;
#pragma unroll
  for (int i = 0; i < kPer; i += 2)
    *reinterpret_cast<uint32_t*>(dst + i) =
        sum != 0.f ? rows::pack2(acc[i] * inv, acc[i + 1] * inv) : 0u;
  if (lane == 0) p.lse[rowi] = sum != 0.f ? top + __logf(sum) : -INFINITY;
}

}  // namespace tree
}  // namespace attn
