// The line of key tiles that attention over the paged cache works through, and
// the end of its pieces.
#pragma once

#include "attn_tree_common.cuh"

namespace attn {
namespace tree {

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// One arrive on the barrier once this thread's cp.async copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

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

template <bool kShared>
__device__ __forceinline__ int seq_tiles(const Seq<kShared>& s, const Work& w) {
  return (s.len + (1 << w.log_tile) - 1) >> w.log_tile;  // lengths end 256 below 2^31
}
template <bool kShared>
__device__ __forceinline__ int seq_segments(const Params& p, const Seq<kShared>& s, const Work& w) {
  return (s.n * p.G + w.rows - 1) / w.rows * (p.H / w.heads);
}
// Tiles of sequence b in the line; 0 if it has no new token, impossible lengths, or is
// the first and does not begin at 0.  falls is set where the offsets decrease: then they
// place no row at all (a row could belong to two sequences).
__device__ __forceinline__ int line_tiles(const Params& p, const Work& w, int b, bool report, Seq<false>& s, bool& falls) {
  const bool fits = load_seq(p, b, s);
  falls |= (int)((uint32_t)s.q0 + (uint32_t)s.n) < s.q0;
  if (!fits || (b == 0 && s.q0 != 0)) {
    if (report) atomicOr(p.err, rows::kBadSeqlens);
    return 0;
  }
  return seq_segments(p, s, w) * seq_tiles(s, w);  // the whole line is below 2^31 (checked on the host)
}
__device__ __forceinline__ int share_of(int total, const Work& w) {
  const int even = (total - 1) / w.units + 1;
  return even > w.min_share ? even : w.min_share;
}

// Where a unit is in the line: item b (lengths in s), segment seg of it, tile
// of that, and how many tiles of its share are left.
template <bool kShared>
struct Walk {
  int b, seg, segs, tile, tiles, left;
  Seq<kShared> s;
  __device__ __forceinline__ void enter(const Params& p, const Work& w) {
    if (load_seq(p, b, s)) {
      segs = seq_segments(p, s, w);
      tiles = seq_tiles(s, w);
    } else {
      segs = tiles = 0;
    }
  }
  // tiles of the current segment that belong to the share
  __device__ __forceinline__ int piece() const { return min(tiles - tile, left); }
  // behind the piece; false at the end of the share
  __device__ __forceinline__ bool next(const Params& p, const Work& w) {
    left -= piece();
    if (left <= 0) return false;
    tile = 0;
    if (++seg < segs) return true;
    seg = 0;
    do {
      if (++b >= (kShared ? p.n_items : p.B)) return false;
      enter(p, w);
    } while (segs == 0 || tiles == 0);
    return true;
  }
};

// A unit's place in the line, found by each of its warps: lane t sums the tiles
// of its block of sequences, the sums are scanned, and the lane whose block holds
// the first tile of the share walks to it.  False: nothing to do.
__device__ __forceinline__ bool find_place(const Params& p, const Work& w, int unit, bool report, Walk<false>& walk) {
  const int t = threadIdx.x % 32, per = (p.B + 31) / 32;
  const int b0 = (int)min((int64_t)t * per, (int64_t)p.B), b1 = min(p.B - b0, per) + b0;
  Seq<false> s{};
  int mine = 0;
  bool falls = false;
  for (int b = b0; b < b1; ++b) mine += line_tiles(p, w, b, report, s, falls);
  if (__any_sync(0xffffffffu, falls)) return false;
  int upto = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, upto, off);
    if (t >= off) upto += v;
  }
  const int total = __shfl_sync(0xffffffffu, upto, 31), before = upto - mine;
  if (total == 0) return false;
  const int share = share_of(total, w);
  if ((int64_t)share * unit >= total) return false;
  const int first = share * unit;
  int at = first - before;
  int b = b0;
  const bool here = first >= before && first < upto;
  if (here && per > 1)  // else s is the one it has read
    for (;; ++b) {
      const int n = line_tiles(p, w, b, false, s, falls);
      if (at < n) break;
      at -= n;
    }
  const int src = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
  walk.b = __shfl_sync(0xffffffffu, b, src);
  walk.s.q0 = __shfl_sync(0xffffffffu, s.q0, src);
  walk.s.n = __shfl_sync(0xffffffffu, s.n, src);
  walk.s.len = __shfl_sync(0xffffffffu, s.len, src);
  at = __shfl_sync(0xffffffffu, at, src);
  walk.segs = seq_segments(p, walk.s, w);
  walk.tiles = seq_tiles(walk.s, w);
  walk.seg = at / walk.tiles;
  walk.tile = at - walk.seg * walk.tiles;
  walk.left = min(share, total - first);
  return true;
}

// n / d for n >= 0, d > 0, by an fp32 reciprocal and its correction: a chain of some ten
// divisions leads to a row's pieces, and the compiler's takes three times as long.
__device__ __forceinline__ int quotient(int n, int d) {
  int q = (int)(__int2float_rn(n) * __frcp_rn(__int2float_rn(d)));
  int r = n - q * d;
  if (r < 0) --q, r += d;
  if (r >= d) ++q, r -= d;
  return (unsigned)r < (unsigned)d ? q : n / d;  // quotients beyond 2^22 or so
}
__device__ __forceinline__ int padded(int tiles, int pad) { return pad > 1 ? quotient(tiles + pad - 1, pad) * pad : tiles; }
// The same over a line that is laid out: the last item whose first tile is not behind the
// share's, by 32 probes a step, the first of them on their way beside the line's numbers.
__device__ __forceinline__ bool find_place(const Params& p, const Work& w, int unit, bool, Walk<true>& walk) {
  const int lane = threadIdx.x % 32;
  const int4 line = *reinterpret_cast<const int4*>(p.line);
  int lo = 0, n = p.n_items;  // items 0 .. lo - 1 begin at or in front of it, lo + n .. behind
  int step = (n + 31) / 32, before;
  const Item* probe = p.items + (int)min((int64_t)(lane + 1) * step, (int64_t)n) - 1;
  if (p.n_items <= 32)
    load_item(probe, walk.s, before);
  else
    before = probe->first;
  const int total = line.x, share = line.y, pad = line.z;
  if (total == 0) return false;
  if ((int64_t)share * unit >= total) return false;
  const int first = share * unit;
  for (;;) {
    const int cnt = __popc(__ballot_sync(0xffffffffu, (int64_t)lane * step < n && before <= first));
    const int skip = (int)min((int64_t)cnt * step, (int64_t)n);
    lo += skip;
    n = min(step, n - skip);
    if (step == 1 || n == 0) break;
    step = (n + 31) / 32;
    before = p.items[lo + min((lane + 1) * step, n) - 1].first;
  }
  walk.b = lo - 1;  // items without tiles lie in front of it
  if (p.n_items <= 32) {  // a lane has it
    before = __shfl_sync(0xffffffffu, before, walk.b);
    walk.s.q0 = __shfl_sync(0xffffffffu, walk.s.q0, walk.b);
    walk.s.n = __shfl_sync(0xffffffffu, walk.s.n, walk.b);
    walk.s.len = __shfl_sync(0xffffffffu, walk.s.len, walk.b);
    walk.s.masked = __shfl_sync(0xffffffffu, walk.s.masked, walk.b);
    walk.s.at = __shfl_sync(0xffffffffu, walk.s.at, walk.b);
    walk.s.page0 = __shfl_sync(0xffffffffu, walk.s.page0, walk.b);
  } else {
    load_item(p.items + walk.b, walk.s, before);
  }
  walk.segs = seq_segments(p, walk.s, w);
  walk.tiles = seq_tiles(walk.s, w);
  const int room = padded(walk.tiles, pad);
  walk.seg = quotient(first - before, room);
  walk.tile = first - before - walk.seg * room;
  walk.left = min(share, total - first);
  if (pad > 1) walk.left = min(walk.left, walk.tiles - walk.tile);  // a share lies in one segment
  return true;
}

// The end of a piece: what a warp writes of its kRows query rows, as the result
// where the piece is the whole segment (slot < 0; or with shared prefixes into the
// rows that are kept for the join), else into its slot of the workspace.  Lane i takes columns 4 (i % 8) .. of rows i / 8, i / 8 + 4, ..
template <int D, bool kCodes, int kRows>
struct PieceEnd {
  static constexpr int kN = kRows / 4;
  int64_t at[kN];      // row of the output, or of the workspace
  float inv[kN];
  uint64_t hid[kN];    // new tokens with values that are not finite, seen by the row
  bool live[kN], direct, poison;
  float* part;

  template <bool kShared>
  __device__ __forceinline__ void rows_of(const Params& p, const Seq<kShared>& sq, int h, int row0, int slot, const float* sm_m,
                                          const float* sm_l, uint64_t hidden, bool bad, int lane) {
    const int M = sq.n * p.G;
    direct = slot < 0 && sq.whole();
    poison = bad;
#pragma unroll
    for (int j = 0; j < kN; ++j) {
      const int r = lane / 8 + 4 * j;
      live[j] = row0 + r < M;
      if (!live[j]) continue;
      const int tok = (row0 + r) / p.G, head = h * p.G + (row0 + r) - tok * p.G;
      const float m = sm_m[r], l = m == -INFINITY ? 0.f : sm_l[r];
      // a row of NaN sums keeps them; one that saw nothing is 0
      inv[j] = l != 0.f ? 1.f / l : 0.f;
      hid[j] = hidden ? hidden & mask_word(p.mask, sq.q0 + tok, tok) : 0;  // (none of a prefix)
      at[j] = slot < 0 ? (int64_t)(sq.q0 + tok) * p.Hq + head : (int64_t)slot * kRows + r;
      float lse = l != 0.f ? (m + lg2(l)) * 0.69314718055994531f : -INFINITY;
      if (poison) lse = direct ? NAN : INFINITY;  // +inf makes the join of the pieces a NaN row
      part = kShared && slot < 0 ? p.o_row : p.o_part;
      if (lane % 8 == 0) (direct ? p.lse : kShared && slot < 0 ? p.lse_row : p.lse_part)[at[j]] = lse;
    }
  }

  // 32 columns from col0 on; buf[r pad]: the rows' sums
  template <bool kShared>
  __device__ __forceinline__ void columns(const Params& p, const Seq<kShared>& sq, int b, int h, const float* buf,
                                          int pad, int col0, int lane) {
#pragma unroll
    for (int j = 0; j < kN; ++j) {
      if (!live[j]) continue;
      const float4 x = *reinterpret_cast<const float4*>(buf + (lane / 8 + 4 * j) * pad + 4 * (lane % 8));
      float f[4] = {x.x, x.y, x.z, x.w};
      const int col = col0 + 4 * (lane % 8);
#pragma unroll
      for (int k = 0; k < 4; ++k) f[k] = inv[j] != 0.f ? f[k] * inv[j] : 0.f;
      uint64_t todo = hid[j];
      while (todo) {
        const int t = __ffsll((long long)todo) - 1;
        todo &= todo - 1;
        const int pos = sq.len - sq.drafts() + t;
        const int id = p.table[sq.table(p, b) + (pos >> p.log_page)];
        if ((unsigned)id >= (unsigned)p.pages) continue;
        const int64_t v = ((((int64_t)id << p.log_page) + (pos & ((1 << p.log_page) - 1))) * p.H + h) * D + col;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (kCodes) {
            if ((reinterpret_cast<const uint8_t*>(p.v)[v + k] & 0x7f) == 0x7f) f[k] = NAN;
          } else {
            const float y = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p.v)[v + k]);
            if (!isfinite(y)) f[k] += y;
          }
        }
      }
      if (poison) f[0] = f[1] = f[2] = f[3] = NAN;
      if (direct)
        *reinterpret_cast<uint2*>(p.o + at[j] * D + col) =
            make_uint2(rows::pack2(f[0], f[1]), rows::pack2(f[2], f[3]));
      else
        *reinterpret_cast<float4*>(part + at[j] * D + col) = make_float4(f[0], f[1], f[2], f[3]);
    }
  }
};

// Pieces of a row joined: weights e^(LSE - max), as for split keys elsewhere in
// the library.  A row, (new token, query head), has one warp, or eight where segments
// are cut into many pieces (warp k takes pieces k, k + kPerRow, ..); a warp takes
// `run` rows one after the other, and looks a segment's place in the line up once
// (trees of 64 drafts, 30000 rows: 292 us in all with a row to a warp, 284 so).
// Rows whose segment lies in one share (or whose sequence the attention refused)
// are left as they are.
template <int D, int kPerRow>
__global__ void __launch_bounds__(256, kPerRow == 1 ? 4 : 3)
tree_join_kernel(const __grid_constant__ Params p, const __grid_constant__ Work w, int run) {
  constexpr int kPer = D / 32;
  __shared__ float sm_sum[8], sm_acc[8][D];
  grid_dep_wait();
  grid_dep_launch();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, k = warp % kPerRow;
  const int64_t all = (int64_t)p.total * p.Hq, row0 = ((int64_t)blockIdx.x * 8 + warp) / kPerRow * run;
  Seq<false> sq{};
  int total = 0, before = 0;
  // The sequence of token t and its place in the line: a lane reads sequences lane,
  // lane + 32, ..  The first that holds t has it.
  auto find = [&](int t) {
    Seq<false> other;
    int n = 0, b = p.B;
    bool falls = false;
    total = before = 0;
    for (int i = lane; i < p.B; i += 32) {
      n = line_tiles(p, w, i, false, other, falls);
      total += n;
      if (n && b == p.B && t >= other.q0 && t < other.q0 + other.n) b = i, sq = other;
    }
    if (falls) b = -1;  // no row has a sequence
    const int mine = b;
    b = __reduce_min_sync(0xffffffffu, b);
    const int src = __ffs(__ballot_sync(0xffffffffu, mine == b)) - 1;
    sq.q0 = __shfl_sync(0xffffffffu, sq.q0, src);
    sq.n = __shfl_sync(0xffffffffu, sq.n, src);
    sq.len = __shfl_sync(0xffffffffu, sq.len, src);
    const bool found = (unsigned)b < (unsigned)p.B;
    if (!found) sq.n = 0;
    if (p.B <= 32)
      before = lane < b ? n : 0;
    else
      for (int i = lane; i < b; i += 32) before += line_tiles(p, w, i, false, other, falls);
    total = __reduce_add_sync(0xffffffffu, total);
    before = __reduce_add_sync(0xffffffffu, before);
    return found;
  };
  int left = 0, r = 0, c0 = 0, c1 = 0, sub = 0;  // rows that follow in the same segment; row of it, its pieces
  bool inside = false, cut = false;
  const int64_t end = min(row0 + run, all);
#pragma unroll 1
  for (int64_t rowi = row0; rowi < end; ++rowi, ++r, --left) {
    if (left <= 0) {
      const int t = (int)(rowi / p.Hq), head = (int)(rowi - (int64_t)t * p.Hq);
      const int h = head / p.G, g = head - h * p.G;
      left = p.G - g;
      cut = t >= sq.q0 && t < sq.q0 + sq.n;
      if (!cut) cut = find(t);
      if (cut) {
        const int row = (t - sq.q0) * p.G + g, group = h / w.heads;
        sub = h - group * w.heads;
        const int mtiles = (sq.n * p.G + w.rows - 1) / w.rows, mt = row / w.rows;
        r = row - mt * w.rows;
        left = min(left, w.rows - r);
        const int share = share_of(total, w), tiles = seq_tiles(sq, w);
        const int first = before + (group * mtiles + mt) * tiles;
        c0 = first / share, c1 = (first + tiles - 1) / share;
        inside = first != c0 * share;  // the first piece begins inside its share
        cut = c0 != c1;
      }
    }
    if (!cut) continue;
    auto at = [&](int c) { return (((int64_t)2 * c + (c == c0 && inside)) * w.heads + sub) * w.rows + r; };
    // kBatch pieces on their way at a time, the first of them beside the maxima
    constexpr int kBatch = kPerRow == 1 ? 4 : 8;
    float x[kBatch][kPer], ls[kBatch];
    auto load = [&](int from) {
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int c = from + j * kPerRow;
        ls[j] = -INFINITY;
        if (c > c1) continue;
        ls[j] = p.lse_part[at(c)];
        const float* from_part = p.o_part + at(c) * D + lane * kPer;
        if (kPer == 4) {
          const float4 y = *reinterpret_cast<const float4*>(from_part);
          x[j][0] = y.x, x[j][1] = y.y, x[j][kPer - 2] = y.z, x[j][kPer - 1] = y.w;
        } else {
          const float2 y = *reinterpret_cast<const float2*>(from_part);
          x[j][0] = y.x, x[j][1] = y.y;
        }
      }
    };
    load(c0 + k);
    float top = -INFINITY;
    for (int c = c0 + lane; c <= c1; c += 32) top = fmaxf(top, p.lse_part[at(c)]);
#pragma unroll
    for (int off = 16; off; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    float acc[kPer], sum = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) acc[i] = 0.f;
    for (int c = c0 + k;;) {
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        if (ls[j] == -INFINITY) continue;
        const float wt = __expf(ls[j] - top);  // a NaN stays one: fmaxf has passed it over
        sum += wt;
#pragma unroll
        for (int i = 0; i < kPer; ++i) acc[i] = fmaf(wt, x[j][i], acc[i]);
      }
      c += kBatch * kPerRow;
      if (c > c1) break;
      load(c);
    }
    if (kPerRow > 1) {  // the row's warps are the CTA's
      if (lane == 0) sm_sum[k] = sum;
#pragma unroll
      for (int i = 0; i < kPer; ++i) sm_acc[k][lane * kPer + i] = acc[i];
      __syncthreads();
      if (k != 0) return;  // (run is 1)
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
}

}  // namespace tree
}  // namespace attn
