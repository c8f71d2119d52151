// Host side of what happens to the paged cache between steps (include/attn_cache.h:
// copies, accepted drafts, forks) and of include/attn_verify.h.  No workspace is kept
// in the library, so calls on any streams and captured graphs share nothing but the
// error word.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cstdint>

#include "../../include/attn_cache.h"
#include "../../include/attn_verify.h"
#include "attn_pages_kernel.cuh"
#include "attn_serve_host.h"
#include "attn_verify_kernel.cuh"

namespace {

using namespace attn_serve;

// As launch(), with clusters of `ctas`.
template <typename... KArgs, typename... Args>
int launch_clusters(void (*kernel)(KArgs...), int64_t grid, int ctas, int threads, int smem, cudaStream_t s,
                    const Args&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ctas > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  return e == cudaSuccess ? ATTN_OK : attn_host::lib_cuda_fail(e);
}

// Lets a kernel have clusters of more than eight CTAs, once per device.  Call with the
// library lock held.
int allow_wide_clusters(const void* kernel) {
  static std::set<std::pair<int, const void*>> done;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return attn_host::lib_cuda_fail(e);
  if (done.count({dev, kernel})) return ATTN_OK;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return attn_host::lib_cuda_fail(e);
  done.insert({dev, kernel});
  return ATTN_OK;
}

int64_t element_bytes(const attn_paged_cache* c) { return c->k_scale ? 1 : 2; }

bool page_size_ok(int n) { return n == 16 || n == 32 || n == 64 || n == 128 || n == 256; }

int check_fork(int B, int N, int W, int pages, int page_size) {
  if (B < 0 || N < 0 || W < 1 || pages < 1 || !page_size_ok(page_size)) return ATTN_ERR_SHAPE;
  if ((int64_t)W * page_size > INT32_MAX || (int64_t)pages * page_size > INT32_MAX) return ATTN_ERR_SHAPE;
  if ((int64_t)std::max(B, N) * W > INT32_MAX / 2) return ATTN_ERR_SHAPE;
  return ATTN_OK;
}

// 32-bit words: four for each row, old and new, and the pages that are handed out.
size_t fork_words(int B, int N, int W, int pages) {
  return 4 * ((size_t)B + N) + (size_t)std::min<int64_t>(pages, (int64_t)N * W);
}

}  // namespace

extern "C" int attn_cache_copy(const attn_paged_cache* cache, const int32_t* src, const int32_t* dst, int n,
                               attn_stream_t stream) {
  using namespace attn::pages;
  if (n < 0) return ATTN_ERR_SHAPE;
  if (n == 0) return ATTN_OK;
  int st = check_pages(cache);
  if (st != ATTN_OK) return st;
  if (!src || !dst) return ATTN_ERR_NULL;
  if (!aligned(src, 4) || !aligned(dst, 4)) return ATTN_ERR_ALIGN;
  Copy p{};
  void* mats[4] = {cache->k, cache->v, cache->k_scale, cache->v_scale};
  for (int i = 0; i < 4; ++i) {
    p.mat[i] = static_cast<uint8_t*>(mats[i]);
    p.bytes[i] = (int64_t)cache->page_size * cache->H * (i < 2 ? cache->d * element_bytes(cache) : 4);
    p.chunks[i] = p.mat[i] ? (int)((p.bytes[i] + kChunk - 1) / kChunk) : 0;
    p.all += p.chunks[i];
  }
  p.src = src;
  p.dst = dst;
  p.items = (int64_t)n * p.all;
  p.pages = cache->num_pages;
  if ((st = error_word(&p.err)) != ATTN_OK) return st;
  // (2000 pages, 541 MB: 89.8 us with 8 CTAs an SM in all, 84.6 with 16, 81.7 with 32)
  const int64_t grid = std::min<int64_t>(p.items, 32 * kPlanSms);
  return launch(cache_copy_kernel, grid, kCopyThreads, 0, reinterpret_cast<cudaStream_t>(stream), p);
}

extern "C" int attn_cache_compact(const attn_paged_cache* cache, const int32_t* seqlens, const int32_t* cu_seqlens,
                                  const int32_t* path, const int32_t* accepted, int B, int total,
                                  attn_stream_t stream) {
  using namespace attn::pages;
  if (B < 0 || total < 0) return ATTN_ERR_SHAPE;
  if (B == 0 || total == 0) return ATTN_OK;
  int st = check_cache(cache);
  if (st != ATTN_OK) return st;
  if (!seqlens || !cu_seqlens || !path || !accepted) return ATTN_ERR_NULL;
  if (!aligned(seqlens, 4) || !aligned(cu_seqlens, 4) || !aligned(path, 4) || !aligned(accepted, 4)) return ATTN_ERR_ALIGN;
  const attn::cache::Pages pg = pages_of(cache);
  Compact p{};
  p.mat[0] = static_cast<uint8_t*>(cache->k);
  p.mat[1] = static_cast<uint8_t*>(cache->v);
  p.scale[0] = cache->k_scale;
  p.scale[1] = cache->v_scale;
  p.table = cache->page_table;
  p.lens = seqlens;
  p.cu = cu_seqlens;
  p.path = path;
  p.kept = accepted;
  p.row_bytes = (int64_t)cache->H * cache->d * element_bytes(cache);
  p.stride = cache->page_table_stride;
  p.pages = cache->num_pages;
  p.log_page = pg.log_page;
  p.H = cache->H;
  p.B = B;
  p.total = total;
  p.parts = (int)((p.row_bytes / 16 + 31) / 32);
  p.scale_parts = cache->k_scale ? (cache->H + 31) / 32 : 0;
  const int64_t warps = (int64_t)B * 2 * (p.parts + p.scale_parts);
  const int64_t grid = (warps + kCompactThreads / 32 - 1) / (kCompactThreads / 32);
  if (grid > INT32_MAX) return ATTN_ERR_SHAPE;
  if ((st = error_word(&p.err)) != ATTN_OK) return st;
  return launch(cache_compact_kernel, grid, kCompactThreads, 0, reinterpret_cast<cudaStream_t>(stream), p);
}

extern "C" size_t attn_cache_fork_workspace(int B, int N, int page_table_stride, int num_pages, int page_size) {
  if (check_fork(B, N, page_table_stride, num_pages, page_size) != ATTN_OK) return 0;
  return sizeof(int) * fork_words(B, N, page_table_stride, num_pages);
}

extern "C" int attn_cache_fork(const int32_t* page_table, int page_table_stride, const int32_t* seqlens, int B,
                               const int32_t* parents, const int32_t* new_seqlens, int N, const int32_t* refs,
                               int32_t* refs_out, int num_pages, int page_size, int32_t* page_table_out,
                               int32_t* copy_src, int32_t* copy_dst, void* workspace, size_t workspace_bytes,
                               attn_stream_t stream) {
  using namespace attn::pages;
  const int W = page_table_stride;
  int st = check_fork(B, N, W, num_pages, page_size);
  if (st != ATTN_OK) return st;
  if (!refs || !refs_out || (B && (!page_table || !seqlens)) ||
      (N && (!parents || !new_seqlens || !page_table_out || !copy_src || !copy_dst)))
    return ATTN_ERR_NULL;
  for (const void* x : {(const void*)refs, (const void*)refs_out, (const void*)page_table, (const void*)seqlens,
                        (const void*)parents, (const void*)new_seqlens, (const void*)page_table_out,
                        (const void*)copy_src, (const void*)copy_dst})
    if (!aligned(x, 4)) return ATTN_ERR_ALIGN;
  auto overlap = [](const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return na && nb && x < y + nb * 4 && y < x + na * 4;
  };
  if (overlap(page_table, (size_t)B * W, page_table_out, (size_t)N * W)) return ATTN_ERR_SHAPE;
  if (refs != refs_out && overlap(refs, num_pages, refs_out, num_pages)) return ATTN_ERR_SHAPE;
  const size_t words = fork_words(B, N, W, num_pages);
  if (!aligned(workspace, 16)) return ATTN_ERR_ALIGN;
  if (words && (!workspace || workspace_bytes < words * sizeof(int))) return ATTN_ERR_SCRATCH;
  Fork p{};
  p.table = page_table;
  p.lens = seqlens;
  p.parents = parents;
  p.new_lens = new_seqlens;
  p.refs = refs;
  p.refs_out = refs_out;
  p.out = page_table_out;
  p.src = copy_src;
  p.dst = copy_dst;
  p.info = static_cast<int4*>(workspace);
  p.heir = reinterpret_cast<int*>(p.info + N);
  p.writer = p.heir + B;
  p.reader = p.writer + B;
  p.taken = p.reader + B;
  p.order = p.taken + B;
  p.B = B;
  p.N = N;
  p.W = W;
  p.pages = num_pages;
  p.vec = aligned(refs, 16) && aligned(refs_out, 16);
  p.log_page = 4;
  while ((1 << p.log_page) < page_size) ++p.log_page;
  if ((st = error_word(&p.err)) != ATTN_OK) return st;
  {
    std::lock_guard<std::mutex> lock(attn_host::lib_mutex());
    if ((st = allow_wide_clusters(reinterpret_cast<const void*>(cache_fork_kernel))) != ATTN_OK) return st;
  }
  // what is read and written in 32-bit words; a small plan gains nothing from more CTAs (64 rows: 10.3 us
  // with 8, 14.1 with 16; 256 rows forked to 512, 6000 positions: 29.2 and 25.9)
  p.ctas = ((int64_t)B + N) * W + num_pages > (1 << 18) ? kMaxForkCtas : kMaxForkCtas / 2;
  return launch_clusters(cache_fork_kernel, p.ctas, p.ctas, kForkThreads, 0, reinterpret_cast<cudaStream_t>(stream), p);
}

extern "C" int attn_verify_drafts(const int32_t* tokens, const void* probs, int64_t probs_stride, const void* draft_probs,
                                  int64_t draft_stride, int bf16, const int32_t* cu_seqlens, const int64_t* mask,
                                  const float* u_accept, const float* u_next, const int32_t* seqlens, int32_t* path,
                                  int32_t* accepted, int32_t* next_token, int32_t* seqlens_out, int B, int total, int V,
                                  attn_stream_t stream) {
  using namespace attn::verify;
  if (B < 0 || total < 0 || V < 1 || V > kMaxV) return ATTN_ERR_SHAPE;
  if (B == 0) return ATTN_OK;
  if (!cu_seqlens || !u_next || !accepted || !next_token || !seqlens != !seqlens_out) return ATTN_ERR_NULL;
  if (total && (!tokens || !probs || !u_accept || !path)) return ATTN_ERR_NULL;
  if (probs_stride < V || (draft_probs && draft_stride < V)) return ATTN_ERR_SHAPE;
  const int size = bf16 ? 2 : 4;
  for (const void* x : {(const void*)tokens, (const void*)cu_seqlens, (const void*)u_accept, (const void*)u_next,
                        (const void*)seqlens, (const void*)path, (const void*)accepted, (const void*)next_token,
                        (const void*)seqlens_out})
    if (!aligned(x, 4)) return ATTN_ERR_ALIGN;
  if (!aligned(mask, 8) || !aligned(probs, size) || !aligned(draft_probs, size)) return ATTN_ERR_ALIGN;
  Params p{};
  p.tokens = tokens;
  p.p = probs;
  p.q = draft_probs;
  p.p_stride = probs_stride;
  p.q_stride = draft_stride;
  p.cu = cu_seqlens;
  p.lens = seqlens;
  p.mask = mask;
  p.u = u_accept;
  p.u_next = u_next;
  p.path = path;
  p.kept = accepted;
  p.next = next_token;
  p.lens_out = seqlens_out;
  p.B = B;
  p.total = total;
  p.V = V;
  // CTAs of a sequence: while their warps have more than a segment each, and all fit the
  // GPU at once
  p.ctas = 1;
  while (p.ctas < kMaxCluster && p.ctas * kWarps * kSeg < V && (int64_t)2 * p.ctas * B <= 4 * kPlanSms) p.ctas *= 2;
  if ((int64_t)B * p.ctas > INT32_MAX) return ATTN_ERR_SHAPE;
  int st = error_word(&p.err);
  if (st != ATTN_OK) return st;
  auto kernel = bf16 ? draft_probs ? verify_kernel<__nv_bfloat16, true> : verify_kernel<__nv_bfloat16, false>
                : draft_probs ? verify_kernel<float, true> : verify_kernel<float, false>;
  return launch_clusters(kernel, (int64_t)B * p.ctas, p.ctas, kThreads, 0, reinterpret_cast<cudaStream_t>(stream), p);
}
