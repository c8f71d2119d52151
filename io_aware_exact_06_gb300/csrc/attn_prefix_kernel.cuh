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
// prompt, 16384 keys and up to 1024 of their own: 122 us in all so, 106 with this kernel;
// 78 with the lines side by side, which it gives their SMs).  One CTA: 6 us, its chain of
// loads, scans and barriers.
struct Plan {
  const int *lens, *cu, *groups, *prefix;
  Item *group_items, *seq_items;
  int* lines;  // of both, four words each: as Params::line
  int B, total, n_groups, H, G, stride, log_page;
  int max_new, max_len, max_group, max_prefix;
  Work group_work, seq_work;
  int group_cta, seq_cta;      // units of a CTA; negative: CTAs of a unit
  float group_cost, seq_cost;  // of a tile, as time of a CTA
  int* err;
};

constexpr int kPlanThreads = 256;
constexpr int kSms = 152;  // GB300

// Offsets and prefixes as a plan reads them: from shared memory where they fit.
struct Offsets {
  const int *cu, *groups, *prefix;
};

// The group of sequence b, or -1: the last whose offset is not above b.
__device__ __forceinline__ int find_group(const Plan& p, const Offsets& of, int b) {
  int lo = 0, hi = p.n_groups;  // groups[0 .. lo-1] <= b < groups[hi ..]
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (of.groups[mid] <= b) lo = mid + 1; else hi = mid;
  }
  return lo > 0 && b < of.groups[lo] ? lo - 1 : -1;
}

// Shared pages of group g; false if its offsets or its prefix are not what the caller's
// bounds allow (its sequences are refused then).
__device__ __forceinline__ bool load_group(const Plan& p, const Offsets& of, int g, int& pages) {
  const int s0 = of.groups[g], s1 = of.groups[g + 1], prefix = of.prefix[g];
  if (s0 < 0 || s1 < s0 || s1 > p.B) return false;
  const int64_t n = (int64_t)of.cu[s1] - of.cu[s0];
  pages = n > 0 ? prefix >> p.log_page : 0;  // nobody reads them else
  return n == 0 || (prefix >= 0 && prefix <= p.max_prefix && pages <= p.stride && n <= p.max_group);
}

// Its rows are all its sequences' (of one that is refused they are computed and not used).
__device__ __forceinline__ bool group_item(const Plan& p, const Offsets& of, int g, Item& x) {
  int pages = 0;
  if (!load_group(p, of, g, pages)) return false;
  const int end = of.groups[g + 1];
  x.at = of.groups[g];
  x.q0 = max(of.cu[x.at], 0);
  x.n = max(min(of.cu[end], p.total) - x.q0, 0);
  while (x.at + 1 < end && of.cu[x.at + 1] == of.cu[x.at]) ++x.at;  // the first with new tokens
  x.len = pages << p.log_page;
  x.page0 = -1;
  return true;
}

__device__ __forceinline__ bool seq_item(const Plan& p, const Offsets& of, int b, int len, Item& x, int& g) {
  const int q0 = of.cu[b], end = of.cu[b + 1];
  const int64_t n = (int64_t)end - q0;
  bool fits = (b == 0 ? q0 == 0 : q0 >= 0) && n >= 0 && end <= p.total && n <= p.max_new && len >= n && len <= p.max_len &&
              len <= (int64_t)p.stride << p.log_page;
  int pages = 0;
  g = find_group(p, of, b);
  if (g >= 0) fits &= load_group(p, of, g, pages);
  if (n == 0) pages = 0;  // no row reads them
  if (!fits || (int64_t)pages << p.log_page > len - n) return false;
  x.q0 = q0, x.n = x.masked = (int)n, x.len = len - (pages << p.log_page), x.at = b, x.page0 = pages;
  return true;
}

// A line whose segments are padded to whole shares has no share with pieces of two of
// them: the end of one and the beginning of another (queries, the pipeline's filling, the
// piece's end) cost about what kCross tiles do.  So it is padded where the units then suffice
// for shares of at most so many tiles more than even ones.
constexpr int kCross = 4;

__global__ void __launch_bounds__(kPlanThreads) prefix_plan_kernel(const __grid_constant__ Plan p) {
  __shared__ int warps[2][kPlanThreads / 32], shares[2][kCross + 1];
  __shared__ int sm_cu[kPlanThreads + 1], sm_groups[kPlanThreads + 1], sm_prefix[kPlanThreads];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  if (threadIdx.x < 2 * (kCross + 1)) (&shares[0][0])[threadIdx.x] = 0;
  prefetch(threadIdx.x == 0   ? p.cu
           : threadIdx.x == 1 ? p.lens
           : threadIdx.x == 2 ? p.groups
           : threadIdx.x == 3 ? p.prefix
           : threadIdx.x == 4 ? p.lines
                              : nullptr);
  grid_dep_wait();
  grid_dep_launch();
  Offsets of{p.cu, p.groups, p.prefix};
  const int first_len = (int)threadIdx.x < p.B ? p.lens[threadIdx.x] : 0;
  if (p.B <= kPlanThreads) {
    for (int i = threadIdx.x; i <= p.B; i += kPlanThreads) sm_cu[i] = p.cu[i];
    of.cu = sm_cu;
  }
  if (p.n_groups <= kPlanThreads) {
    for (int i = threadIdx.x; i <= p.n_groups && p.n_groups > 0; i += kPlanThreads) sm_groups[i] = p.groups[i];
    if ((int)threadIdx.x < p.n_groups) sm_prefix[threadIdx.x] = p.prefix[threadIdx.x];
    of.groups = sm_groups, of.prefix = sm_prefix;
  }
  __syncthreads();
  const bool cu_falls = rows::offsets_fall(of.cu, p.B, threadIdx.x, kPlanThreads);
  const bool falls = __syncthreads_or(cu_falls || rows::offsets_fall(of.groups, p.n_groups, threadIdx.x, kPlanThreads));
  bool bad = falls;
  // Places of this thread's counts behind those in front, in both lines; `at` moves on.
  auto scan = [&](int2 count, int2& at) {
    int2 upto = count;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, upto.x, off), y = __shfl_up_sync(0xffffffffu, upto.y, off);
      if (lane >= off) upto.x += x, upto.y += y;
    }
    __syncthreads();
    if (lane == 31) warps[0][warp] = upto.x, warps[1][warp] = upto.y;
    __syncthreads();
    const bool has = lane < kPlanThreads / 32;
    const int x = has ? warps[0][lane] : 0, y = has ? warps[1][lane] : 0;
    const int2 first = make_int2(at.x + __reduce_add_sync(0xffffffffu, lane < warp ? x : 0) + upto.x - count.x,
                                 at.y + __reduce_add_sync(0xffffffffu, lane < warp ? y : 0) + upto.y - count.y);
    at.x += __reduce_add_sync(0xffffffffu, x), at.y += __reduce_add_sync(0xffffffffu, y);
    return first;
  };
  auto segments = [&](const Item& x, const Work& w) {
    return quotient(x.n * p.G + w.rows - 1, w.rows) * (p.H >> (w.heads / 2));
  };
  auto tiles_of = [&](const Item& x, const Work& w) { return (x.len + (1 << w.log_tile) - 1) >> w.log_tile; };
  // Thread i has group i and sequence i, and those kPlanThreads further on.  (Lines of up
  // to kPlanThreads items may be padded; their items stay in registers.)
  const int most = max(p.B, p.n_groups);
  int2 at = make_int2(0, 0), pad = make_int2(1, 1);
  Item gi{}, si{};
  int2 segs{}, tiles{}, first{};
  int g = -1;
  auto load = [&](int i) {
    gi = Item{}, si = Item{};
    segs = tiles = make_int2(0, 0);
    if (i < p.n_groups) {
      if (group_item(p, of, i, gi))
        segs.x = segments(gi, p.group_work), tiles.x = tiles_of(gi, p.group_work);
      else
        gi.n = gi.len = 0, bad = true;
    }
    if (i < p.B) {
      if (seq_item(p, of, i, i < kPlanThreads ? first_len : p.lens[i], si, g))
        segs.y = segments(si, p.seq_work), tiles.y = tiles_of(si, p.seq_work);
      else
        si.n = si.len = 0, bad = true;
    }
  };
  for (int from = 0; from < most && !falls; from += kPlanThreads) {  // (the whole lines are below 2^31: checked on the host)
    load(from + threadIdx.x);
    scan(make_int2(segs.x * tiles.x, segs.y * tiles.y), at);
  }
  // The SMs go to the lines as their tiles cost.
  const float group_all = at.x * p.group_cost, seq_all = at.y * p.seq_cost;
  int sms = 0;  // of the line of groups
  if (at.x > 0) {
    const int team = max(-p.group_cta, 1);
    sms = at.y > 0 ? (int)(kSms * (group_all / (group_all + seq_all)) + 0.5f) : kSms;
    sms = min(max(sms / team * team, team), at.y > 0 ? kSms - 1 : kSms);
  }
  auto units_of = [&](int ctas, int per_cta, const Work& w) {
    return max(1, min(w.units, per_cta < 0 ? ctas / -per_cta : ctas * per_cta));
  };
  const int2 units = make_int2(units_of(sms, p.group_cta, p.group_work), units_of(kSms - sms, p.seq_cta, p.seq_work));
  int2 share = make_int2(at.x > 0 ? max((at.x - 1) / units.x + 1, p.group_work.min_share) : 1,
                         at.y > 0 ? max((at.y - 1) / units.y + 1, p.seq_work.min_share) : 1);
  if (most <= kPlanThreads) {
    if (32 * warp < most) {
#pragma unroll 1
      for (int c = 0; c <= kCross; c += 2) {
        // (segments beyond the units need not be counted: they are too many already)
        const int x = tiles.x > 0 ? min(segs.x, units.x + 1) * (quotient(tiles.x - 1, share.x + c) + 1) : 0;
        const int y = tiles.y > 0 ? min(segs.y, units.y + 1) * (quotient(tiles.y - 1, share.y + c) + 1) : 0;
        const int sx = __reduce_add_sync(0xffffffffu, min(x, 1 << 20)), sy = __reduce_add_sync(0xffffffffu, min(y, 1 << 20));
        if (lane == 0 && sx) atomicAdd(&shares[0][c], sx);
        if (lane == 0 && sy) atomicAdd(&shares[1][c], sy);
      }
    }
    __syncthreads();
    for (int c = kCross; c >= 0; c -= 2) {
      if (shares[0][c] <= units.x) pad.x = share.x + c;
      if (shares[1][c] <= units.y) pad.y = share.y + c;
    }
    if (pad.x > 1) share.x = pad.x;
    if (pad.y > 1) share.y = pad.y;
  }
  at = make_int2(0, 0);
  for (int from = 0; from < most && !falls; from += kPlanThreads) {
    const int i = from + threadIdx.x;
    if (most > kPlanThreads) load(i);
    first = scan(make_int2(segs.x * padded(tiles.x, pad.x), segs.y * padded(tiles.y, pad.y)), at);
    auto write = [&](Item* to, const Item& x, int front) {
      reinterpret_cast<int4*>(to)[0] = make_int4(x.q0, x.n, x.len, x.masked);
      reinterpret_cast<int4*>(to)[1] = make_int4(x.at, x.page0, front, 0);
    };
    if (i < p.n_groups) write(p.group_items + i, gi, first.x);
    if (i < p.B) write(p.seq_items + i, si, first.y);
  }
  __syncthreads();  // all groups are laid out: their sequences' items take them up
  for (int i = threadIdx.x; i < p.B && !falls; i += kPlanThreads) {
    if (most > kPlanThreads) load(i);
    if (si.page0 <= 0) continue;
    const int4 *of_group = reinterpret_cast<const int4*>(p.group_items + g), a = of_group[0], b = of_group[1];
    reinterpret_cast<int4*>(p.seq_items + i)[2] = make_int4(a.x, a.y, a.z, b.z);
  }
  if (threadIdx.x == 0) {
    reinterpret_cast<int4*>(p.lines)[0] = make_int4(at.x, share.x, pad.x, 0);
    reinterpret_cast<int4*>(p.lines)[1] = make_int4(at.y, share.y, pad.y, 0);
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

// Row `row` of key head h, of an item (sq) with `before` tiles in front of it; line as in
// Params.
__device__ __forceinline__ Pieces find_pieces(const Params& p, const Work& w, const Seq<true>& sq, int share, int pad,
                                              int before, int h, int row) {
  Pieces x{};
  const int tiles = seq_tiles(sq, w);
  if (tiles == 0) return x;
  const int group = h >> (w.heads / 2);  // 1, 2 or 4 heads
  x.sub = h - group * w.heads;
  const int mtiles = quotient(sq.n * p.G + w.rows - 1, w.rows), mt = quotient(row, w.rows);
  x.r = row - mt * w.rows;
  const int first = before + (group * mtiles + mt) * padded(tiles, pad);
  x.c0 = quotient(first, share);
  x.n = quotient(first + tiles - 1, share) - x.c0 + 1;
  x.inside = first != x.c0 * share;
  x.rows = x.n == 1;
  return x;
}

// A row, (new token, query head), has one warp; a warp takes `run` rows one after the
// other, and looks their sequence up once for a token, the first before it waits for the
// lines' ends (four samples of 1000 keys: 25.0 -> 22.8 us).  Weights are e^(LSE - max), as
// for the pieces of one line.  Rows of a sequence that the attention refused, and rows that
// the line of sequences wrote as results, are left as they are.  Latency bounds it, of
// offsets -> item -> pieces -> rows, 6 to 8 us with the launch.  A row's pieces loaded while
// the row before is joined spill registers (16 samples of 8 prompts: 90.8 -> 105.2).
template <int D>
__global__ void __launch_bounds__(256, 2)
prefix_join_kernel(const __grid_constant__ Params pg, const __grid_constant__ Work wg, const __grid_constant__ Params p,
                   const __grid_constant__ Work w, int run) {
  constexpr int kPer = D / 32, kBatch = 8;  // pieces on their way at a time
  prefetch_line(p);
  if (threadIdx.x >= 32 && threadIdx.x < 40) {
    const int t = threadIdx.x - 32;
    prefetch(t == 0 ? (const void*)pg.o_part : t == 1 ? (const void*)pg.lse_part : t == 2 ? (const void*)pg.o_row
             : t == 3 ? (const void*)pg.lse_row : t == 4 ? (const void*)p.cu : t == 5 ? (const void*)p.lse : nullptr);
  }
  __threadfence();  // as at the second line's start: what is read up to the wait was there before the lines began
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int all = p.total * p.Hq;  // a 32-bit number (checked on the host)
  const int row0 = (int)min(((int64_t)blockIdx.x * 8 + warp) * run, (int64_t)all), end = (int)min((int64_t)row0 + run, (int64_t)all);
  const int4 line = *reinterpret_cast<const int4*>(p.line), g_line = *reinterpret_cast<const int4*>(pg.line);
  Seq<true> sq{}, gq{};  // the token's sequence, its group
  int before = 0, g_before = 0;
  auto find = [&](int t) {
    const int b = rows::find_sequence<true>(p.cu, p.B, t);
    if (b >= p.B) return false;
    load_item(p.items + b, sq, before);
    const int4 g = reinterpret_cast<const int4*>(p.items + b)[2];
    if (t < sq.q0 || t >= sq.q0 + sq.n) return false;
    gq.n = gq.len = 0;
    if (sq.page0 > 0) gq.q0 = g.x, gq.n = g.y, gq.len = g.z, g_before = g.w;
    return true;
  };
  bool found = false;
  int at = -1, head_at = -1;  // the token looked up, the key head whose pieces a and b are
  Pieces a{}, b{};
  int t = quotient(row0, p.Hq), head = row0 - t * p.Hq;
  auto look = [&]() {
    if (t != at) found = find(t), at = t, head_at = -1;
    if (!found) return;
    if (head_at < 0 || head >= (head_at + 1) * p.G || (a.n > 0 && a.r + 1 == wg.rows) || b.r + 1 == w.rows) {
      const int h = quotient(head, p.G), g = head - h * p.G;
      head_at = h;
      a = find_pieces(pg, wg, gq, g_line.y, g_line.z, g_before, h, (t - gq.q0) * p.G + g);
      b = find_pieces(p, w, sq, line.y, line.z, before, h, (t - sq.q0) * p.G + g);
    } else {
      ++a.r, ++b.r;
    }
  };
  const bool some_row = row0 < end && line.x != 0;  // (offsets that decrease: no sequence has rows)
  if (some_row) look();
  grid_dep_wait();  // every thread: the kernel behind this one counts on both lines' end
  grid_dep_launch();
  if (!some_row) return;
#pragma unroll 1
  for (int rowi = row0; rowi < end; ++rowi) {
    if (rowi > row0) {
      if (++head == p.Hq) head = 0, ++t;
      look();
    }
    if (!found) continue;
    if (b.rows && sq.whole()) continue;  // the result
    const int n = a.n + b.n;
    auto part = [&](int c, const float*& o) {  // piece c: its LSE, and where its row is
      const Params& q = c < a.n ? pg : p;
      const Pieces& x = c < a.n ? a : b;
      const int64_t i = x.rows ? rowi : x.slot(c < a.n ? wg : w, c < a.n ? c : c - a.n);
      o = (x.rows ? q.o_row : q.o_part) + i * D;
      return (x.rows ? q.lse_row : q.lse_part) + i;
    };
    // 32 pieces at a time: lane c has the weight of piece c
    float top = -INFINITY, sum = 0.f, acc[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) acc[i] = 0.f;
    for (int c0 = 0; c0 < n; c0 += 32) {
      const int here = min(n - c0, 32);
      const float* o;
      const float* mine = part(min(c0 + lane, n - 1), o);
      const uint64_t where = reinterpret_cast<uint64_t>(o);
      float x[kBatch][kPer];
      auto load = [&](int from) {
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          const int c = min(from + j, here - 1);
          const float* row = reinterpret_cast<const float*>(__shfl_sync(0xffffffffu, where, c)) + lane * kPer;
          if (kPer == 4) {
            const float4 y = *reinterpret_cast<const float4*>(row);
            x[j][0] = y.x, x[j][1] = y.y, x[j][kPer - 2] = y.z, x[j][kPer - 1] = y.w;
          } else {
            const float2 y = *reinterpret_cast<const float2*>(row);
            x[j][0] = y.x, x[j][1] = y.y;
          }
        }
      };
      load(0);
      const float ls = lane < here ? *mine : -INFINITY;
      float most = ls;  // a NaN is passed over
#pragma unroll
      for (int off = 16; off; off >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, off));
      most = fmaxf(most, top);
      // (a first +inf, of a row that is to be NaN, makes every weight 0 or NaN)
      const float shrink = top == -INFINITY ? 0.f : __expf(top - most);
      float wt = ls == -INFINITY ? 0.f : __expf(ls - most);
      top = most;
      sum *= shrink;
#pragma unroll
      for (int i = 0; i < kPer; ++i) acc[i] *= shrink;
      const uint32_t some = __ballot_sync(0xffffffffu, ls != -INFINITY);
      for (int from = 0;;) {
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          const float f = __shfl_sync(0xffffffffu, wt, (from + j) & 31);
          if (from + j >= here || !((some >> (from + j)) & 1)) continue;  // (what an empty piece holds counts for nothing)
          sum += f;
#pragma unroll
          for (int i = 0; i < kPer; ++i) acc[i] = fmaf(f, x[j][i], acc[i]);
        }
        from += kBatch;
        if (from >= here) break;
        load(from);
      }
    }
    const float inv = sum != 0.f ? 1.f / sum : 0.f;
    __nv_bfloat16* dst = p.o + (int64_t)rowi * D + lane * kPer;
#pragma unroll
    for (int i = 0; i < kPer; i += 2)
      *reinterpret_cast<uint32_t*>(dst + i) = sum != 0.f ? rows::pack2(acc[i] * inv, acc[i + 1] * inv) : 0u;
    if (lane == 0) p.lse[rowi] = sum != 0.f ? top + __logf(sum) : -INFINITY;
  }
}

}  // namespace tree
}  // namespace attn
