// Host side of attn_fwd_prefix (include/attn_cache.h): attention over the paged cache
// for sequences whose first pages are shared.  Two lines of work at a time, each on SMs of
// its own: every sequence's rows over its own pages, and every group's over its shared
// ones.  A first kernel lays them out, a last one joins the rows' parts.  It keeps no workspace in the library.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
#include <climits>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "../../include/attn_cache.h"
#include "attn_prefix_kernel.cuh"
#include "attn_prefix_rows_kernel.cuh"
#include "attn_serve_host.h"
#include "attn_tree_plan.h"

namespace {

using namespace attn_serve;

static_assert(attn::tree::kSms == kPlanSms, "the lines' units here, and the SMs that the plan gives them");

struct Sizes {
  int B, total, Hq, H, d, max_new, max_len, groups, max_group, max_prefix, splits;
};

int check_sizes(const Sizes& z) {
  const int st = check_tree(z.B, z.total, z.Hq, z.H, z.d, z.max_new, z.max_len, z.splits);
  if (st != ATTN_OK) return st;
  if (z.groups < 0 || z.max_group < 0 || z.max_prefix < 0 || z.max_prefix > z.max_len) return ATTN_ERR_SHAPE;
  return ATTN_OK;
}

bool empty(const Sizes& z) { return z.B == 0 || z.total == 0 || z.max_new == 0; }

// What a CTA takes for a tile of a line, in ns: d = 128, measured alone on an SM, but for the
// few-row kernel, whose constant was fitted to a bf16 cache with d = 128 (two lines that share
// HBM).  Half the bytes a tile, d = 64 or codes, would do with fewer SMs.  64 samples of 16384
// keys, up to 1024 of their own, 4 rows a key head, us with 1350, 2000, 2700 and 3600 ns: bf16
// d = 128 83, 74.5, 74.5, 81, d = 64 54, 57, 62, 68; codes d = 128 66, 70, 73.5, 83, d = 64 56,
// 60, 62, 70.  The rows kernel with two bf16 a probability (the same case among other calls):
// 71.0 us with 1900 ns a pair, 70.0 with 2400, 71.2 with 2900.
float tile_cost(const Plan& pl, int d, bool rows_kernel, bool two) {
  const float wide = d == 128 ? 1.f : 0.9f;
  if (few(pl)) return 2700.f * pl.work.heads / attn::tree::few_warps(true, pl.rows);
  const bool pair = pl.rows > attn::tree::kBigRows;
  if (rows_kernel) return wide * (two ? pair ? 2400.f : 1300.f : pair ? 1900.f : 1100.f);
  return wide * (pair ? 2300.f : 2000.f);
}

// The line of groups, the line of sequences, and the parts of the workspace: slots of
// both, and the rows of both that are not cut.
struct Plans {
  Plan group, seq;
  bool any;  // some group may share a page
  int64_t rows;
  size_t parts() const { return 2 * (size_t)rows + (any ? tree_rows(group) : 0) + tree_rows(seq); }
};
// The lines' items and their tiles, in front of the parts.
size_t plan_bytes(const Sizes& z) {
  return ((size_t)z.B + z.groups) * sizeof(attn::tree::Item) + 32;
}
size_t bytes_of(const Sizes& z, const Plans& x) {
  return plan_bytes(z) + x.parts() * (z.d + 1) * sizeof(float);
}
// A segment of as many row tiles as CTAs take over the same keys at a time (at most 8),
// where at least nine tenths of the SMs are busy so: 2048 rows of 8 key heads over 32768 keys
// read them eight times from HBM else.
void make_teams(Plan& pl, int64_t tiles) {
  int team = 1;
  for (int t = 2; t <= 8 && t <= tiles; ++t) {
    const double busy = (double)tiles / (double)((tiles + t - 1) / t * t) * (kPlanSms / t * t) / kPlanSms;
    if (busy >= 0.9) team = t;
  }
  pl.work.rows = pl.rows * team;
  pl.work.units = (int)std::max<int64_t>(1, std::min<int64_t>(pl.ctas, kPlanSms / team));
  pl.ctas = (int64_t)pl.work.units * team;
  pl.slots = 2 * pl.ctas;
}
Plans plans(const Sizes& z, int page, bool codes) {
  Plans x{};
  x.rows = (int64_t)z.total * z.Hq;
  const int most = std::min(z.max_group, z.total);
  x.any = z.groups > 0 && most > 0 && z.max_prefix >= page;
  if (x.any) {
    x.group = tree_plan(z.groups, z.total, z.Hq, z.H, z.d, most, z.max_prefix, z.splits, codes, true);
    if (!codes && !few(x.group)) make_teams(x.group, ((int64_t)most * (z.Hq / z.H) + x.group.rows - 1) / x.group.rows);
  }
  x.seq = tree_plan(z.B, z.total, z.Hq, z.H, z.d, z.max_new, z.max_len, z.splits, codes, true);
  return x;
}

// The line of groups: over a bf16 cache many rows have a kernel of their own.  `two`:
// it holds probabilities as the sum of two bf16, as the few-row kernel does, which has
// these rows over their own keys: a row's weights keep the same bits whether its keys
// are shared or not.
template <int D, bool kCodes>
int launch_groups(const Plan& pl, bool two, const CUtensorMap& mk, const CUtensorMap& mv, const attn::tree::Params& p,
                  cudaStream_t s) {
  using namespace attn::tree;
  if (kCodes || few(pl)) return launch_line<D, kCodes, true>(pl, mk, mv, p, s);
  auto kernel = pl.rows == kBigRows ? two ? prefix_rows_kernel<D, false, true> : prefix_rows_kernel<D, false, false>
                : two               ? prefix_rows_kernel<D, true, true> : prefix_rows_kernel<D, true, false>;
  const int smem = pl.rows == kBigRows ? RowsCfg<D, false>::kSmem : RowsCfg<D, true>::kSmem;
  const int st = allow_smem(reinterpret_cast<const void*>(kernel), smem);
  if (st != ATTN_OK) return st;
  return launch(kernel, pl.ctas, kRowsThreads, smem, s, mk, mv, p, pl.work);
}

template <int D, bool kCodes>
int launch_prefix(const Plans& x, const CUtensorMap (&maps)[4], const attn::tree::Plan& plan, const attn::tree::Params& pg,
                  const attn::tree::Params& p, cudaStream_t s) {
  // No launch may come between these.  The first line waits for the plan before it lets the next kernel
  // start, and the plan for all that came before it: so the second line may read what those wrote, and write
  // its parts, beside the first, which it waits for at its end; and the join may read the plan and the
  // offsets before it waits for both.
  int st = launch(attn::tree::prefix_plan_kernel, 1, attn::tree::kPlanThreads, 0, s, plan);
  if (st != ATTN_OK) return st;
  // The second line starts as soon as every CTA of the first runs, and ends after it.
  if ((st = launch_line<D, kCodes, true>(x.seq, maps[2], maps[3], p, s)) != ATTN_OK) return st;
  if (x.any && (st = launch_groups<D, kCodes>(x.group, few(x.seq), maps[0], maps[1], pg, s)) != ATTN_OK) return st;
  const int64_t rows = x.rows;
  // 16 warps an SM, as many as the join's registers allow without spills (64 samples, with one bf16 a
  // probability, 71.5 us with 32 warps, 68.2 with 24, 67.2 with 16): all rows at once, while a warp has eight at most
  const int run = (int)std::clamp<int64_t>((rows + 16 * kPlanSms - 1) / (16 * kPlanSms), 1, 8);
  return launch(attn::tree::prefix_join_kernel<D>, (rows + 8 * run - 1) / (8 * run), 256, 0, s, pg,
                x.any ? x.group.work : x.seq.work, p, x.seq.work, run);
}

}  // namespace

extern "C" size_t attn_fwd_prefix_workspace(int B, int total, int Hq, int H, int d, int max_new, int max_len,
                                            int groups, int max_group, int max_prefix, int num_splits) {
  const Sizes z{B, total, Hq, H, d, max_new, max_len, groups, max_group, max_prefix, num_splits};
  if (check_sizes(z) != ATTN_OK || empty(z)) return 0;
  size_t most = 0;  // the cache's type and its pages' size are not known here
  for (bool codes : {false, true}) most = std::max(most, bytes_of(z, plans(z, 16, codes)));
  return most;
}

extern "C" int attn_fwd_prefix(const void* q, int64_t q_stride, const attn_paged_cache* cache, const int32_t* seqlens,
                               const int32_t* cu_seqlens, const int64_t* mask, const int32_t* cu_groups,
                               const int32_t* prefix_lens, void* o, float* lse, int B, int total, int Hq, int max_new,
                               int max_len, int groups, int max_group, int max_prefix, float scale, int num_splits,
                               void* workspace, size_t workspace_bytes, attn_stream_t stream) {
  if (!cache) return ATTN_ERR_NULL;
  const int d = cache->d;
  const Sizes z{B, total, Hq, cache->H, d, max_new, max_len, groups, max_group, max_prefix, num_splits};
  int st = check_sizes(z);
  if (st != ATTN_OK) return st;
  if (!std::isfinite(scale) || scale < 0.f) return ATTN_ERR_SCALE;
  if (empty(z)) return ATTN_OK;
  if ((st = check_cache(cache)) != ATTN_OK) return st;
  if ((st = check_rows(q, q_stride, Hq, d)) != ATTN_OK) return st;
  if (!o || !lse || !seqlens || !cu_seqlens || (groups && (!cu_groups || !prefix_lens))) return ATTN_ERR_NULL;
  if (!aligned(o, 16) || !aligned(lse, 4) || !aligned(seqlens, 4) || !aligned(cu_seqlens, 4) || !aligned(mask, 8) ||
      !aligned(cu_groups, 4) || !aligned(prefix_lens, 4) || !aligned(workspace, 16))
    return ATTN_ERR_ALIGN;
  const bool codes = cache->k_scale != nullptr;
  const Plans x = plans(z, cache->page_size, codes);
  if (!x.seq.fits || (x.any && !x.group.fits)) return ATTN_ERR_SHAPE;
  if (x.rows > INT32_MAX) return ATTN_ERR_SHAPE;
  if (!workspace || workspace_bytes < bytes_of(z, x)) return ATTN_ERR_SCRATCH;

  const attn::cache::Pages pg = pages_of(cache);
  attn::tree::Params p{};
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_ts = q_stride;
  p.lens = seqlens;
  p.cu = cu_seqlens;
  p.table = cache->page_table;
  p.mask = mask;
  p.v = cache->v;
  p.kscale = cache->k_scale;
  p.vscale = cache->v_scale;
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.B = B;
  p.total = total;
  p.Hq = Hq;
  p.H = cache->H;
  p.G = Hq / cache->H;
  p.stride = cache->page_table_stride;
  p.pages = cache->num_pages;
  p.log_page = pg.log_page;
  p.max_new = max_new;
  p.max_len = max_len;
  // scale 0 weighs every key alike; the smallest normal factor does, without 0 * inf
  p.c = (float)std::max((double)scale * 1.4426950408889634, (double)FLT_MIN);
  // the lines, then rows of d floats, then their LSE
  attn::tree::Plan plan{};
  plan.lens = seqlens;
  plan.cu = cu_seqlens;
  plan.groups = cu_groups;
  plan.prefix = prefix_lens;
  plan.group_items = static_cast<attn::tree::Item*>(workspace);
  plan.seq_items = plan.group_items + groups;
  plan.lines = reinterpret_cast<int*>(plan.seq_items + B);
  plan.B = B;
  plan.total = total;
  plan.n_groups = groups;
  plan.H = cache->H;
  plan.G = p.G;
  plan.stride = p.stride;
  plan.log_page = p.log_page;
  plan.max_new = max_new;
  plan.max_len = max_len;
  plan.max_group = max_group;
  plan.max_prefix = max_prefix;
  plan.group_work = x.any ? x.group.work : x.seq.work;
  plan.seq_work = x.seq.work;
  const bool rows_kernel = x.any && !codes && !few(x.group);
  const int team = rows_kernel ? x.group.work.rows / x.group.rows : 1;
  auto per_cta = [](const Plan& pl) { return few(pl) ? attn::tree::few_warps(true, pl.rows) / pl.work.heads : 1; };
  plan.seq_cta = per_cta(x.seq);
  plan.group_cta = !x.any ? 1 : team > 1 ? -team : per_cta(x.group);
  plan.seq_cost = tile_cost(x.seq, d, false, false);
  plan.group_cost = x.any ? team * tile_cost(x.group, d, rows_kernel, few(x.seq)) : 0.f;
  p.items = plan.seq_items;
  p.line = plan.lines + 4;
  p.n_items = B;
  attn::tree::Params of_groups = p;
  of_groups.items = plan.group_items;
  of_groups.line = plan.lines;
  of_groups.n_items = groups;
  of_groups.second = true;
  float* at = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + plan_bytes(z));
  float* lse_at = at + x.parts() * d;
  auto take = [&](size_t rows, float*& o_part, float*& lse_part) {
    o_part = at, lse_part = lse_at;
    at += rows * d, lse_at += rows;
  };
  take(x.rows, of_groups.o_row, of_groups.lse_row);
  take(x.rows, p.o_row, p.lse_row);
  if (x.any) take(tree_rows(x.group), of_groups.o_part, of_groups.lse_part);
  take(tree_rows(x.seq), p.o_part, p.lse_part);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  std::lock_guard<std::mutex> lock(attn_host::lib_mutex());
  int dev = 0, sms = 0;
  if ((st = attn_host::lib_device(&dev, &sms, &p.err)) != ATTN_OK) return st;
  plan.err = of_groups.err = p.err;
  const int64_t rows = (int64_t)cache->num_pages * cache->page_size;
  CUtensorMap maps[4];
  for (int i = 0; i < 4; ++i) {
    if (i < 2 && !x.any) continue;
    const int box = std::min(cache->page_size,
                             few(i < 2 ? x.group : x.seq) ? attn::tree::kFewTile : attn::tree::kBigTile);
    if ((st = attn_host::lib_make_cache_map(&maps[i], i % 2 ? cache->v : cache->k, rows, cache->H, d, codes, box)) != ATTN_OK)
      return st;
  }
  return d == 64 ? codes ? launch_prefix<64, true>(x, maps, plan, of_groups, p, s)
                         : launch_prefix<64, false>(x, maps, plan, of_groups, p, s)
         : codes ? launch_prefix<128, true>(x, maps, plan, of_groups, p, s)
                 : launch_prefix<128, false>(x, maps, plan, of_groups, p, s);
}
