// Host side of include/attn_norm.h and include/attn_cache.h: argument checks,
// TMA descriptors and launches.  These entry points keep no workspace in the
// library (where they need one it is the caller's), so calls on any streams and
// captured graphs share nothing but the error word.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
#include <climits>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "../../include/attn_cache.h"
#include "../../include/attn_norm.h"
#include "attn_norm_kernel.cuh"
#include "attn_serve_host.h"
#include "attn_tree_plan.h"

namespace {

using namespace attn_serve;

// ------------------------------------------------------------ norm, rotation --
int check_rotary(const attn_rotary* r, int T, int d, attn::norm::Rotary* out) {
  if (!r) return ATTN_ERR_NULL;
  if (r->rot < 0 || r->rot > d || r->rot % 16) return ATTN_ERR_SHAPE;
  *out = attn::norm::Rotary{};
  out->half = r->rot / 2;
  out->edge0 = out->edge1 = INT_MAX;
  if (r->rot == 0) return ATTN_OK;
  if (r->axes < 1 || r->axes > 3 || r->table_len < 1) return ATTN_ERR_SHAPE;
  if (r->axes > 1) {
    int sum = 0;
    for (int a = 0; a < r->axes; ++a) {
      if (r->section[a] < 0 || r->section[a] > out->half) return ATTN_ERR_SHAPE;
      sum += r->section[a];
    }
    if (sum != out->half) return ATTN_ERR_SHAPE;
    out->edge0 = r->section[0];
    if (r->axes == 3) out->edge1 = r->section[0] + r->section[1];
  }
  if (T == 0) return ATTN_OK;
  if (!r->cos || !r->sin || !r->positions) return ATTN_ERR_NULL;
  if (!aligned(r->cos, 16) || !aligned(r->sin, 16) || !aligned(r->positions, 4)) return ATTN_ERR_ALIGN;
  out->cos = r->cos;
  out->sin = r->sin;
  out->pos = r->positions;
  out->P = r->table_len;
  out->axes = r->axes;
  return ATTN_OK;
}

int check_norm(int T, int Hq, int Hk, int d, float eps) {
  if (T < 0 || Hq < 0 || Hk < 0) return ATTN_ERR_SHAPE;
  if (d != 64 && d != 128) return ATTN_ERR_HEADDIM;
  if (!std::isfinite(eps) || eps < 0.f) return ATTN_ERR_SCALE;
  if (((int64_t)Hq + Hk) * d > (1 << 20)) return ATTN_ERR_SHAPE;
  return ATTN_OK;
}

// CTAs of the gradient for queries and for keys: two an SM in all, what the
// kernel's registers allow, in proportion to the heads; fewer when there is
// less to do.  A run is four chunks at most, so that the warps' streams lie closer
// together in memory (32 heads of d = 128 are eight: 96.0 us with whole tokens, 92.7
// with four, 95.6 with two or three).  The order of the weight sums depends on these
// alone.
struct BwdPlan {
  int64_t ctas[2];
  int run[2];
};
BwdPlan bwd_plan(int T, int Hq, int Hk, int d) {
  BwdPlan pl{};
  const int H[2] = {Hq, Hk};
  int64_t share = 2 * kPlanSms;
  for (int i = 0; i < 2; ++i) {
    if (H[i] == 0 || T == 0) continue;
    const int64_t chunks = chunks_of(H[i], d, attn::norm::kBwdSteps);
    const int64_t mine = std::max<int64_t>(1, share * H[i] / (Hq + Hk));
    pl.run[i] = (int)std::clamp<int64_t>((int64_t)T * chunks / (4 * mine * attn::norm::kWarps), 1, std::min<int64_t>(chunks, 4));
    const int64_t items = (int64_t)T * ((chunks + pl.run[i] - 1) / pl.run[i]);
    pl.ctas[i] = std::min((items + attn::norm::kWarps - 1) / attn::norm::kWarps, mine);
  }
  return pl;
}

// ---------------------------------------------------------------------- tree --
template <int D, bool kCodes>
int launch_tree(const Plan& pl, const CUtensorMap& mk, const CUtensorMap& mv, const attn::tree::Params& p,
                cudaStream_t s) {
  using namespace attn::tree;
  const int st = launch_line<D, kCodes, false>(pl, mk, mv, p, s);
  if (st != ATTN_OK) return st;
  const int64_t rows = (int64_t)p.total * p.Hq;
  if (pl.many) return launch(tree_join_kernel<D, 8>, rows, 256, 0, s, p, pl.work, 1);
  const int run = (int)std::clamp<int64_t>(rows / (32 * kPlanSms), 1, 8);  // 32 warps an SM at least
  return launch(tree_join_kernel<D, 1>, (rows + 8 * run - 1) / (8 * run), 256, 0, s, p, pl.work, run);
}

}  // namespace

extern "C" int attn_qk_norm_rope(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                                 const void* wq, const void* wk, void* q_out, int64_t q_out_stride,
                                 void* k_out, int64_t k_out_stride, int T, int Hq, int Hk, int d,
                                 float eps, const attn_rotary* rotary, attn_stream_t stream) {
  int st = check_norm(T, Hq, Hk, d, eps);
  if (st != ATTN_OK) return st;
  attn::norm::Fwd p{};
  if ((st = check_rotary(rotary, T, d, &p.rot)) != ATTN_OK) return st;
  if (T == 0 || Hq + Hk == 0) return ATTN_OK;
  if ((st = check_rows(q, q_stride, Hq, d)) != ATTN_OK) return st;
  if ((st = check_rows(k, k_stride, Hk, d)) != ATTN_OK) return st;
  if ((st = check_rows(q_out, q_out_stride, Hq, d)) != ATTN_OK) return st;
  if ((st = check_rows(k_out, k_out_stride, Hk, d)) != ATTN_OK) return st;
  if ((Hq && !wq) || (Hk && !wk)) return ATTN_ERR_NULL;
  if (!aligned(wq, 16) || !aligned(wk, 16)) return ATTN_ERR_ALIGN;
  const int64_t chunks = chunks_of(Hq + Hk, d, attn::norm::kSteps);
  p.run = run_of(T * chunks, chunks, 3 * attn::norm::kWarps);
  const int64_t items = T * ((chunks + p.run - 1) / p.run);
  const int64_t grid = std::min<int64_t>((items + attn::norm::kWarps - 1) / attn::norm::kWarps, 3 * kPlanSms);
  if ((st = error_word(&p.err)) != ATTN_OK) return st;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.wq = static_cast<const __nv_bfloat16*>(wq);
  p.wk = static_cast<const __nv_bfloat16*>(wk);
  p.qo = static_cast<__nv_bfloat16*>(q_out);
  p.ko = static_cast<__nv_bfloat16*>(k_out);
  p.q_ts = q_stride;
  p.k_ts = k_stride;
  p.qo_ts = q_out_stride;
  p.ko_ts = k_out_stride;
  p.T = T;
  p.Hq = Hq;
  p.Hk = Hk;
  p.eps = eps;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool part = rotary->rot < d;
  auto kernel = d == 64 ? rotary->interleaved ? part ? attn::norm::norm_rope_kernel<64, true, true>
                                                     : attn::norm::norm_rope_kernel<64, true, false>
                          : part ? attn::norm::norm_rope_kernel<64, false, true>
                                 : attn::norm::norm_rope_kernel<64, false, false>
                : rotary->interleaved ? part ? attn::norm::norm_rope_kernel<128, true, true>
                                             : attn::norm::norm_rope_kernel<128, true, false>
                : part ? attn::norm::norm_rope_kernel<128, false, true>
                       : attn::norm::norm_rope_kernel<128, false, false>;
  return launch(kernel, grid, attn::norm::kThreads, attn::norm::kSmem, s, p);
}

extern "C" size_t attn_qk_norm_rope_bwd_workspace(int T, int Hq, int Hk, int d) {
  if (check_norm(T, Hq, Hk, d, 0.f) != ATTN_OK) return 0;
  const BwdPlan pl = bwd_plan(T, Hq, Hk, d);
  return (size_t)(pl.ctas[0] + pl.ctas[1]) * d * sizeof(float);
}

extern "C" int attn_qk_norm_rope_bwd(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                                     const void* wq, const void* wk, const void* dq_out,
                                     int64_t dq_out_stride, const void* dk_out, int64_t dk_out_stride,
                                     void* dq, int64_t dq_stride, void* dk, int64_t dk_stride,
                                     float* dwq, float* dwk, int T, int Hq, int Hk, int d, float eps,
                                     const attn_rotary* rotary, void* workspace,
                                     size_t workspace_bytes, attn_stream_t stream) {
  int st = check_norm(T, Hq, Hk, d, eps);
  if (st != ATTN_OK) return st;
  attn::norm::Bwd p{};
  if ((st = check_rotary(rotary, T, d, &p.rot)) != ATTN_OK) return st;
  if (Hq + Hk == 0 && !dwq && !dwk) return ATTN_OK;
  if ((Hq && !dwq) || (Hk && !dwk)) return ATTN_ERR_NULL;
  if (!aligned(dwq, 4) || !aligned(dwk, 4)) return ATTN_ERR_ALIGN;
  const BwdPlan pl = bwd_plan(T, Hq, Hk, d);
  const int64_t grid = pl.ctas[0] + pl.ctas[1];
  if (grid > 0) {
    if ((st = check_rows(q, q_stride, Hq, d)) != ATTN_OK) return st;
    if ((st = check_rows(k, k_stride, Hk, d)) != ATTN_OK) return st;
    if ((st = check_rows(dq_out, dq_out_stride, Hq, d)) != ATTN_OK) return st;
    if ((st = check_rows(dk_out, dk_out_stride, Hk, d)) != ATTN_OK) return st;
    if ((st = check_rows(dq, dq_stride, Hq, d)) != ATTN_OK) return st;
    if ((st = check_rows(dk, dk_stride, Hk, d)) != ATTN_OK) return st;
    if ((Hq && !wq) || (Hk && !wk)) return ATTN_ERR_NULL;
    if (!aligned(wq, 16) || !aligned(wk, 16)) return ATTN_ERR_ALIGN;
    if (!workspace || workspace_bytes < (size_t)grid * d * sizeof(float)) return ATTN_ERR_SCRATCH;
    if (!aligned(workspace, 16)) return ATTN_ERR_ALIGN;
  }
  if ((st = error_word(&p.err)) != ATTN_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (grid > 0) {
    const void *x[2] = {q, k}, *w[2] = {wq, wk}, *g[2] = {dq_out, dk_out};
    void* dx[2] = {dq, dk};
    const int64_t x_ts[2] = {q_stride, k_stride}, g_ts[2] = {dq_out_stride, dk_out_stride},
                  dx_ts[2] = {dq_stride, dk_stride};
    for (int i = 0; i < 2; ++i) {
      p.x[i] = static_cast<const __nv_bfloat16*>(x[i]);
      p.w[i] = static_cast<const __nv_bfloat16*>(w[i]);
      p.g[i] = static_cast<const __nv_bfloat16*>(g[i]);
      p.dx[i] = static_cast<__nv_bfloat16*>(dx[i]);
      p.x_ts[i] = x_ts[i];
      p.g_ts[i] = g_ts[i];
      p.dx_ts[i] = dx_ts[i];
      p.H[i] = i ? Hk : Hq;
      p.run[i] = pl.run[i];
    }
    p.T = T;
    p.ctas_q = (int)pl.ctas[0];
    p.eps = eps;
    p.part = static_cast<float*>(workspace);
    const bool part = rotary->rot < d;
    auto kernel = d == 64 ? rotary->interleaved ? part ? attn::norm::norm_rope_bwd_kernel<64, true, true>
                                                       : attn::norm::norm_rope_bwd_kernel<64, true, false>
                            : part ? attn::norm::norm_rope_bwd_kernel<64, false, true>
                                   : attn::norm::norm_rope_bwd_kernel<64, false, false>
                  : rotary->interleaved ? part ? attn::norm::norm_rope_bwd_kernel<128, true, true>
                                               : attn::norm::norm_rope_bwd_kernel<128, true, false>
                  : part ? attn::norm::norm_rope_bwd_kernel<128, false, true>
                         : attn::norm::norm_rope_bwd_kernel<128, false, false>;
    if ((st = launch(kernel, grid, attn::norm::kThreads, attn::norm::kSmem, s, p)) != ATTN_OK) return st;
  }
  // a kind without heads, as well as a batch without tokens, has no partial rows: 0
  const attn::norm::WeightSum w{static_cast<const float*>(workspace), dwq, dwk, (int)pl.ctas[0], (int)pl.ctas[1], d};
  return launch(attn::norm::norm_weight_kernel, 2 * d / 32, 1024, 0, s, w);
}

extern "C" int attn_cache_write(const attn_paged_cache* cache, const void* k, int64_t k_stride,
                                const void* v, int64_t v_stride, const int32_t* seqlens,
                                const int32_t* cu_seqlens, int B, int total, attn_stream_t stream) {
  if (B < 0 || total < 0) return ATTN_ERR_SHAPE;
  if (B == 0 || total == 0) return ATTN_OK;
  int st = check_cache(cache);
  if (st != ATTN_OK) return st;
  if ((st = check_rows(k, k_stride, cache->H, cache->d)) != ATTN_OK) return st;
  if ((st = check_rows(v, v_stride, cache->H, cache->d)) != ATTN_OK) return st;
  if (!seqlens || !cu_seqlens) return ATTN_ERR_NULL;
  if (!aligned(seqlens, 4) || !aligned(cu_seqlens, 4)) return ATTN_ERR_ALIGN;
  attn::cache::Write p{};
  const int64_t chunks = 2 * chunks_of(cache->H, cache->d, attn::cache::kSteps);
  const int run = run_of(total * chunks, kMaxRun, 4 * attn::cache::kWarps);
  p.step = (total - 1) / run + 1;
  const int64_t items = p.step * chunks;
  const int64_t grid = (items + attn::cache::kWarps - 1) / attn::cache::kWarps;
  if (grid > INT32_MAX) return ATTN_ERR_SHAPE;
  if ((st = error_word(&p.err)) != ATTN_OK) return st;
  p.c = pages_of(cache);
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.k_ts = k_stride;
  p.v_ts = v_stride;
  p.lens = seqlens;
  p.cu = cu_seqlens;
  p.B = B;
  p.total = total;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool codes = cache->k_scale != nullptr;
  auto kernel = cache->d == 64 ? codes ? attn::cache::cache_write_kernel<64, true>
                                       : attn::cache::cache_write_kernel<64, false>
                : codes ? attn::cache::cache_write_kernel<128, true>
                        : attn::cache::cache_write_kernel<128, false>;
  return launch(kernel, grid, attn::cache::kThreads, 0, s, p);
}

extern "C" int attn_cache_read(const attn_paged_cache* cache, void* k, void* v,
                               const int32_t* cu_seqlens, int B, int total, attn_stream_t stream) {
  if (B < 0 || total < 0) return ATTN_ERR_SHAPE;
  if (B == 0 || total == 0) return ATTN_OK;
  int st = check_cache(cache);
  if (st != ATTN_OK) return st;
  const int64_t hd = (int64_t)cache->H * cache->d;
  if ((st = check_rows(k, hd, cache->H, cache->d)) != ATTN_OK) return st;
  if ((st = check_rows(v, hd, cache->H, cache->d)) != ATTN_OK) return st;
  if (!cu_seqlens) return ATTN_ERR_NULL;
  if (!aligned(cu_seqlens, 4)) return ATTN_ERR_ALIGN;
  const bool codes = cache->k_scale != nullptr;
  attn::cache::Read p{};
  const int64_t chunks = 2 * chunks_of(cache->H, cache->d, attn::cache::kSteps);
  const int run = run_of(total * chunks, kMaxRun, 4 * attn::cache::kWarps);
  p.step = (total - 1) / run + 1;
  const int64_t items = p.step * chunks;
  const int64_t grid = (items + attn::cache::kWarps - 1) / attn::cache::kWarps;
  if (grid > INT32_MAX) return ATTN_ERR_SHAPE;
  if ((st = error_word(&p.err)) != ATTN_OK) return st;
  p.c = pages_of(cache);
  p.k = static_cast<__nv_bfloat16*>(k);
  p.v = static_cast<__nv_bfloat16*>(v);
  p.cu = cu_seqlens;
  p.B = B;
  p.total = total;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  auto kernel = cache->d == 64 ? codes ? attn::cache::cache_read_kernel<64, true>
                                       : attn::cache::cache_read_kernel<64, false>
                : codes ? attn::cache::cache_read_kernel<128, true>
                        : attn::cache::cache_read_kernel<128, false>;
  return launch(kernel, grid, attn::cache::kThreads, 0, s, p);
}

extern "C" size_t attn_fwd_tree_workspace(int B, int total, int Hq, int H, int d, int max_new,
                                          int max_len, int num_splits) {
  if (check_tree(B, total, Hq, H, d, max_new, max_len, num_splits) != ATTN_OK) return 0;
  if (B == 0 || total == 0 || max_new == 0) return 0;
  // the cache's type is not known here
  size_t most = 0;
  for (bool codes : {false, true})
    most = std::max(most, tree_bytes(tree_plan(B, total, Hq, H, d, max_new, max_len, num_splits, codes), d));
  return most;
}

extern "C" int attn_fwd_tree(const void* q, int64_t q_stride, const attn_paged_cache* cache,
                             const int32_t* seqlens, const int32_t* cu_seqlens, const int64_t* mask,
                             void* o, float* lse, int B, int total, int Hq, int max_new, int max_len,
                             float scale, int num_splits, void* workspace, size_t workspace_bytes,
                             attn_stream_t stream) {
  if (!cache) return ATTN_ERR_NULL;
  const int d = cache->d;
  int st = check_tree(B, total, Hq, cache->H, d, max_new, max_len, num_splits);
  if (st != ATTN_OK) return st;
  if (!std::isfinite(scale) || scale < 0.f) return ATTN_ERR_SCALE;
  if (B == 0 || total == 0 || max_new == 0) return ATTN_OK;
  if ((st = check_cache(cache)) != ATTN_OK) return st;
  if ((st = check_rows(q, q_stride, Hq, d)) != ATTN_OK) return st;
  if (!o || !lse || !seqlens || !cu_seqlens) return ATTN_ERR_NULL;
  if (!aligned(o, 16) || !aligned(lse, 4) || !aligned(seqlens, 4) || !aligned(cu_seqlens, 4) ||
      !aligned(mask, 8) || !aligned(workspace, 16))
    return ATTN_ERR_ALIGN;
  const bool codes = cache->k_scale != nullptr;
  const Plan pl = tree_plan(B, total, Hq, cache->H, d, max_new, max_len, num_splits, codes);
  if (!pl.fits) return ATTN_ERR_SHAPE;
  const size_t need = tree_bytes(pl, d);
  if (!workspace || workspace_bytes < need) return ATTN_ERR_SCRATCH;
  if ((int64_t)total * Hq > INT32_MAX) return ATTN_ERR_SHAPE;
  const int64_t rows = (int64_t)cache->num_pages * cache->page_size;
  const int box = std::min(cache->page_size, few(pl) ? attn::tree::kFewTile : attn::tree::kBigTile);

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
  p.o_part = static_cast<float*>(workspace);
  p.lse_part = p.o_part + tree_rows(pl) * d;
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
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  std::lock_guard<std::mutex> lock(attn_host::lib_mutex());
  int dev = 0, sms = 0;
  if ((st = attn_host::lib_device(&dev, &sms, &p.err)) != ATTN_OK) return st;
  CUtensorMap mk, mv;
  if ((st = attn_host::lib_make_cache_map(&mk, cache->k, rows, cache->H, d, codes, box)) != ATTN_OK) return st;
  if ((st = attn_host::lib_make_cache_map(&mv, cache->v, rows, cache->H, d, codes, box)) != ATTN_OK) return st;
  return d == 64 ? codes ? launch_tree<64, true>(pl, mk, mv, p, s) : launch_tree<64, false>(pl, mk, mv, p, s)
         : codes ? launch_tree<128, true>(pl, mk, mv, p, s)
                 : launch_tree<128, false>(pl, mk, mv, p, s);
}
