// Host services that the translation units of the norm, the paged cache and what
// is around them share: launches, checks of arguments.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cstdint>
#include <mutex>
#include <set>
#include <utility>

#include "../../include/attn_cache.h"
#include "attn_cache_kernel.cuh"
#include "attn_host.h"

namespace attn_serve {

constexpr int kPlanSms = 152;  // GB300: the split rules need no device

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline int error_word(int** err) {
  std::lock_guard<std::mutex> lock(attn_host::lib_mutex());
  int dev = 0, sms = 0;
  return attn_host::lib_device(&dev, &sms, err);
}

// Launch that may overlap the end of the stream's previous kernel.  Every kernel here
// waits for it before its first global access, but for those of attention over shared
// prefixes behind the plan, which rely on the order of their launches (attn_prefix.cu).
template <typename... KArgs, typename... Args>
int launch(void (*kernel)(KArgs...), int64_t grid, int threads, int smem, cudaStream_t s, const Args&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  return e == cudaSuccess ? ATTN_OK : attn_host::lib_cuda_fail(e);
}

// Raises the dynamic shared-memory limit of a kernel, once per device.  Call
// with the library lock held.
inline int allow_smem(const void* kernel, int bytes) {
  static std::set<std::pair<int, const void*>> done;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return attn_host::lib_cuda_fail(e);
  if (done.count({dev, kernel})) return ATTN_OK;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return attn_host::lib_cuda_fail(e);
  done.insert({dev, kernel});
  return ATTN_OK;
}

inline int check_rows(const void* x, int64_t stride, int H, int d) {
  if (H == 0) return ATTN_OK;
  if (!x) return ATTN_ERR_NULL;
  if (stride < (int64_t)H * d) return ATTN_ERR_SHAPE;
  if (!aligned(x, 16) || stride % 8) return ATTN_ERR_ALIGN;
  return ATTN_OK;
}

// Chunks of H heads of d channels when a warp holds `steps` row groups.
inline int64_t chunks_of(int H, int d, int steps) {
  const int64_t c = (int64_t)(32 / (d / 8)) * steps;
  return (H + c - 1) / c;
}

// How many of `most` pieces (chunks of a token, tokens) a warp takes one after
// the other: as many as leave the GPU's resident warps about four rounds, so
// that loads run ahead without an uneven end.
inline int run_of(int64_t pieces, int64_t most, int warps_per_sm) {
  return (int)std::clamp<int64_t>(pieces / (4 * (int64_t)kPlanSms * warps_per_sm), 1, most);
}

// --------------------------------------------------------------------- cache --
inline int check_cache(const attn_paged_cache* c) {
  if (!c) return ATTN_ERR_NULL;
  if (c->d != 64 && c->d != 128) return ATTN_ERR_HEADDIM;
  if (c->H < 1 || (int64_t)c->H * c->d > (1 << 20) || c->num_pages < 1 || c->page_table_stride < 1)
    return ATTN_ERR_SHAPE;
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128 &&
      c->page_size != 256)
    return ATTN_ERR_SHAPE;
  // rows, and positions of a sequence, are 32-bit numbers
  if ((int64_t)c->num_pages * c->page_size > INT32_MAX ||
      (int64_t)c->page_table_stride * c->page_size > INT32_MAX)
    return ATTN_ERR_SHAPE;
  if (!c->k || !c->v || !c->page_table || !c->k_scale != !c->v_scale) return ATTN_ERR_NULL;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->page_table, 4) ||
      !aligned(c->k_scale, 16) || !aligned(c->v_scale, 16))
    return ATTN_ERR_ALIGN;
  return ATTN_OK;
}

// For calls that name pages themselves: as check_cache, without the page table.
inline int check_pages(const attn_paged_cache* c) {
  if (!c) return ATTN_ERR_NULL;
  attn_paged_cache pool = *c;
  pool.page_table = static_cast<const int32_t*>(c->k);  // aligned where it matters
  pool.page_table_stride = 1;
  return check_cache(&pool);
}

// Tokens a warp writes or reads one after the other, at most: with more the warps'
// streams lie further apart (reading 98586 e4m3 tokens of 8 heads, d = 128: 100.3, 98.8
// and 99.9 us with 3, 4 and 8).
constexpr int kMaxRun = 4;

inline attn::cache::Pages pages_of(const attn_paged_cache* c) {
  attn::cache::Pages p{};
  p.k = c->k;
  p.v = c->v;
  p.ks = c->k_scale;
  p.vs = c->v_scale;
  p.table = c->page_table;
  p.stride = c->page_table_stride;
  p.pages = c->num_pages;
  p.log_page = 4;
  while ((1 << p.log_page) < c->page_size) ++p.log_page;
  p.H = c->H;
  return p;
}

}  // namespace attn_serve
