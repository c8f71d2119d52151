// Attention over shared prefixes: the layout of its two lines of work, and the join of
// a row's pieces from both.
#pragma once

#include "attn_tree_work.cuh"

namespace attn {
namespace tree {

// ---------------------------------------------------------------------- plan --
// Every warp of the kernels behind it needs its place in a line, and every row of the
// join its sequence and its group: found from offsets, groups and lengths each time, that
// is a chain of some eight dependent loads and a scan over the batch (64 samples of one
// prompt: 122 us in all so, ...).
struct Plan {
  const int *lens, *cu, *groups, *prefix;
  Item *group_items, *seq_items;
  int* lines;  // tiles of both
  int B, total, n_groups, H, G, stride, log_page;
  int max_new, max_len, max_group, max_prefix;
  Work group_work, seq_work;
  int* err;
};

constexpr int kPlanThreads = 1024;

// The group of sequence b, or -1: the last whose offset is not above b.
__device__ __forceinline__ int find_group(const Plan& p, int b) {
  int lo = 0, hi = p.n_groups;  // groups[0 .. lo-1] <= b < groups[hi ..]
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (p.groups[mid] <= b) lo = mid + 1; else hi = mid;
  }
  return lo > 0 && b < p.groups[lo] ? lo - 1 : -1;
}

// Shared pages of group g; false if its offsets or its prefix are not what the caller's
// bounds allow (its sequences are refused then).
__device__ __forceinline__ bool load_group(const Plan& p, int g, int& pages) {
  const int s0 = p.groups[g], s1 = p.groups[g + 1], prefix = p.prefix[g];
  pages = prefix >> p.log_page;
  if (s0 < 0 || s1 < s0 || s1 > p.B || prefix < 0 || prefix > p.max_prefix || pages > p.stride) return false;
  return (int64_t)p.cu[s1] - p.cu[s0] <= p.max_group;
}

// Its rows are all its sequences' (of one that is refused they are computed and not used).
__device__ __forceinline__ bool group_item(const Plan& p, int g, Item& x) {
  int pages = 0;
  if (!load_group(p, g, pages)) return false;
  x.at = p.groups[g];
  x.q0 = max(p.cu[x.at], 0);
  x.n = max(min(p.cu[p.groups[g + 1]], p.total) - x.q0, 0);
  x.len = pages << p.log_page;
  x.page0 = -1;
  return true;
}

__device__ __forceinline__ bool seq_item(const Plan& p, int b, Item& x) {
  const int q0 = p.cu[b], end = p.cu[b + 1], len = p.lens[b];
  const int64_t n = (int64_t)end - q0;
  bool fits = (b == 0 ? q0 == 0 : q0 >= 0) && n >= 0 && end <= p.total && n <= p.max_new && len >= n && len <= p.max_len &&
              len <= (int64_t)p.stride << p.log_page;
  int pages = 0;
  x.group = find_group(p, b);
  if (x.group >= 0) fits &= load_group(p, x.group, pages);
  if (!fits || (int64_t)pages << p.log_page > len - n) return false;
  x.q0 = q0, x.n = x.masked = (int)n, x.len = len - (pages << p.log_page), x.at = b, x.page0 = pages;
  return true;
}

__global__ void __launch_bounds__(kPlanThreads) prefix_plan_kernel(const __grid_constant__ Plan p) {
  __shared__ int warps[kPlanThreads / 32];
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const bool cu_falls = rows::offsets_fall(p.cu, p.B, threadIdx.x, kPlanThreads);
  const bool falls = __syncthreads_or(cu_falls || rows::offsets_fall(p.groups, p.n_groups, threadIdx.x, kPlanThreads));
  bool bad = falls;
  for (int line = 0; line < 2; ++line) {
    const int items = line ? p.B : p.n_groups;
    const Work& w = line ? p.seq_work : p.group_work;
    int at = 0;
    for (int from = 0; from < items && !falls; from += kPlanThreads) {
      const int i = from + threadIdx.x;
      Item x{};
      int tiles = 0;
      if (i < items) {
        if (line ? seq_item(p, i, x) : group_item(p, i, x))
          tiles = (x.n * p.G + w.rows - 1) / w.rows * (p.H / w.heads) * ((x.len + (1 << w.log_tile) - 1) >> w.log_tile);
        else
          x.n = x.len = 0, bad = true;
      }
      int upto = tiles;  // the whole line is below 2^31 (checked on the host)
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, off);
        if (lane >= off) upto += v;
      }
      __syncthreads();
      if (lane == 31) warps[warp] = upto;
      __syncthreads();
      const int mine = warps[lane];
      const int before = __reduce_add_sync(0xffffffffu, lane < warp ? mine : 0);
      x.first = at + before + upto - tiles;
      at += __reduce_add_sync(0xffffffffu, mine);
      if (i < items) {
        int4* to = reinterpret_cast<int4*>((line ? p.seq_items : p.group_items) + i);
        to[0] = make_int4(x.q0, x.n, x.len, x.masked);
        to[1] = make_int4(x.at, x.page0, x.first, x.group);
      }
    }
    if (threadIdx.x == 0) p.lines[line] = at;
  }
  if (bad) atomicOr(p.err, rows::kBadSeqlens);
}

// ---------------------------------------------------------------------- join --
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
// sequence and group up once for a token.  Weights are e^(LSE - max), as for the pieces
// of one line.  Rows of a sequence that the attention refused, and rows that the line of
// sequences wrote as results, are left as they are.
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
  const int total = *p.line, g_total = *pg.line;
  if (total == 0) return;  // no sequence has rows (offsets that decrease among them)
  Seq<true> sq{}, gq{};    // the token's sequence, its group
  int before = 0, g_before = 0;
  auto find = [&](int t) {
    const int b = rows::find_sequence(p.cu, p.B, t);
    if (b >= p.B) return false;
    int group, none;
    load_item(p.items + b, sq, before, group);
    if (t < sq.q0 || t >= sq.q0 + sq.n) return false;
    gq.n = gq.len = 0;
    if (sq.page0 > 0) load_item(pg.items + group, gq, g_before, none);
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
