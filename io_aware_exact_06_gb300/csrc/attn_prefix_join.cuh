// The join of attention over shared prefixes: a row's pieces from the line of groups
// (its group's shared pages) and from the line of sequences (the pages that are its
// sequence's own), weighed by e^(LSE - max) as the pieces of one line are.
#pragma once

#include "attn_tree_work.cuh"

namespace attn {
namespace tree {

// The pieces of a row in one line: none, one that is the whole segment (in the line's
// rows), or those that shares cut (in slots).
struct Pieces {
  int c0, n;      // first share, how many
  bool inside;    // the first begins inside its share
  bool rows;      // n is 1: in the line's rows
  int sub, r;     // head of the segment, row of its tile
  __device__ __forceinline__ int64_t slot(const Work& w, int k) const {
    return (((int64_t)2 * (c0 + k) + (k == 0 && inside)) * w.heads + sub) * w.rows + r;
  }
};

// Row `row` of key head h, of an item (sq) with `before` tiles in front of it of `total`.
__device__ __forceinline__ Pieces find_pieces(const Params& p, const Work& w, const Seq<true>& sq, int total, int before,
                                              int h, int row) {
  Pieces x{};
  const int tiles = seq_tiles(sq, w);
  if (tiles == 0) return x;
  const int group = h / w.heads;
  x.sub = h - group * w.heads;
  const int mtiles = (sq.n * p.G + w.rows - 1) / w.rows, mt = row / w.rows;
  x.r = row - mt * w.rows;
  const int share = share_of(total, w), first = before + (group * mtiles + mt) * tiles;
  x.c0 = first / share;
  x.n = (first + tiles - 1) / share - x.c0 + 1;
  x.inside = first != x.c0 * share;
  x.rows = x.n == 1;
  return x;
}

// A row, (new token, query head), has one warp, or eight (warp k takes pieces k,
// k + kPerRow, ..); a warp takes `run` rows one after the other, and looks their
// sequence and group up once for a token.  Rows of a sequence that the attention
// refused, and rows that the line of sequences wrote as results, are left as they are.
template <int D, int kPerRow>
__global__ void __launch_bounds__(256, kPerRow == 1 ? 4 : 3)
prefix_join_kernel(const __grid_constant__ Params pg, const __grid_constant__ Work wg, const __grid_constant__ Params p,
                   const __grid_constant__ Work w, int run) {
  constexpr int kPer = D / 32;
  __shared__ float sm_sum[8], sm_acc[8][D];
  grid_dep_wait();
  grid_dep_launch();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, k = warp % kPerRow;
  const int64_t all = (int64_t)p.total * p.Hq, row0 = ((int64_t)blockIdx.x * 8 + warp) / kPerRow * run;
  if (groups_fall(p, false)) return;  // no row has a group
  Seq<true> sq{}, gq{};               // the token's sequence, its group
  int total = 0, before = 0, g_total = 0, g_before = 0;
  // Tiles in front of item b, and in all.
  auto count = [&](const Params& q, const Work& v, int b, int& sum, int& front) {
    Seq<true> other;
    bool falls = false;
    sum = front = 0;
    for (int i = lane; i < line_items<true>(q); i += 32) {
      const int n = line_tiles(q, v, i, false, other, falls);
      sum += n;
      if (i < b) front += n;
    }
    sum = __reduce_add_sync(0xffffffffu, sum);
    front = __reduce_add_sync(0xffffffffu, front);
    return !__any_sync(0xffffffffu, falls);
  };
  // The sequence of token t, what the line has of it, and the same for its group.
  auto find = [&](int t) {
    Seq<true> other;
    int b = p.B;
    bool falls = false;
    for (int i = lane; i < p.B; i += 32) {
      const int n = line_tiles(p, w, i, false, other, falls);
      if (n && b == p.B && t >= other.q0 && t < other.q0 + other.n) b = i;
    }
    b = __reduce_min_sync(0xffffffffu, b);
    if (b == p.B || !count(p, w, b, total, before)) return false;
    load_seq(p, b, sq);
    gq.n = gq.len = 0;
    if (sq.page0 > 0) {
      const int g = find_group(p, b);
      count(pg, wg, g, g_total, g_before);
      load_seq(pg, g, gq);
    }
    return true;
  };
  bool found = false;
  int at = -1;  // the token looked up
  const int64_t end = min(row0 + run, all);
#pragma unroll 1
  for (int64_t rowi = row0; rowi < end; ++rowi) {
    const int t = (int)(rowi / p.Hq), head = (int)(rowi - (int64_t)t * p.Hq);
    const int h = head / p.G, g = head - h * p.G;
    if (t != at) found = find(t), at = t;
    if (!found) continue;
    const Pieces a = find_pieces(pg, wg, gq, g_total, g_before, h, (t - gq.q0) * p.G + g);
    const Pieces b = find_pieces(p, w, sq, total, before, h, (t - sq.q0) * p.G + g);
    if (b.rows && sq.whole()) continue;  // the result
    const int n = a.n + b.n;
    auto part = [&](int c, const float*& o) {  // piece c: its LSE, and where its row is
      const Params& q = c < a.n ? pg : p;
      const Pieces& x = c < a.n ? a : b;
      const int64_t i = x.rows ? rowi : x.slot(c < a.n ? wg : w, c < a.n ? c : c - a.n);
      o = (x.rows ? q.o_row : q.o_part) + i * D;
      return (x.rows ? q.lse_row : q.lse_part) + i;
    };
    constexpr int kBatch = kPerRow == 1 ? 4 : 8;
    float x[kBatch][kPer], ls[kBatch];
    auto load = [&](int from) {
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int c = from + j * kPerRow;
        ls[j] = -INFINITY;
        if (c >= n) continue;
        const float* o;
        ls[j] = *part(c, o);
        o += lane * kPer;
        if (kPer == 4) {
          const float4 y = *reinterpret_cast<const float4*>(o);
          x[j][0] = y.x, x[j][1] = y.y, x[j][kPer - 2] = y.z, x[j][kPer - 1] = y.w;
        } else {
          const float2 y = *reinterpret_cast<const float2*>(o);
          x[j][0] = y.x, x[j][1] = y.y;
        }
      }
    };
    load(k);
    float top = -INFINITY;
    for (int c = lane; c < n; c += 32) {
      const float* o;
      top = fmaxf(top, *part(c, o));
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    float acc[kPer], sum = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) acc[i] = 0.f;
    for (int c = k;;) {
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        if (ls[j] == -INFINITY) continue;
        const float wt = __expf(ls[j] - top);  // a NaN stays one: fmaxf has passed it over
        sum += wt;
#pragma unroll
        for (int i = 0; i < kPer; ++i) acc[i] = fmaf(wt, x[j][i], acc[i]);
      }
      c += kBatch * kPerRow;
      if (c >= n) break;
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
      *reinterpret_cast<uint32_t*>(dst + i) = sum != 0.f ? rows::pack2(acc[i] * inv, acc[i + 1] * inv) : 0u;
    if (lane == 0) p.lse[rowi] = sum != 0.f ? top + __logf(sum) : -INFINITY;
  }
}

}  // namespace tree
}  // namespace attn
