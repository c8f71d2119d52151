// Pages of the cache between steps: copies of whole pages, the rows of accepted drafts
// moved together, and the next batch's page table.
#pragma once

#include <climits>

#include "attn_rows.cuh"

namespace attn {
namespace pages {

// A matrix of the cache in 16-byte units, or a table of scales in 4-byte ones.
struct Copy {
  uint8_t* mat[4];     // keys, values, their scales
  int64_t bytes[4];    // of a page
  int chunks[4], all;  // pieces of kChunk bytes that a page has of each, and of all
  const int *src, *dst;
  int64_t items;
  int pages;
  int* err;
};

// ---------------------------------------------------------------------- copy --
// An item is kChunk bytes of one matrix of one pair's page: every thread four 16-byte
// loads, then its stores.  Items follow each other through a page, so that CTAs that
// run together read and write one stretch of memory.  HBM bounds it: 541 MB in 81.7 us,
// 0.99 of the rate of a plain copy.
constexpr int kCopyThreads = 256;
constexpr int kCopyUnits = 4;
constexpr int kChunk = kCopyThreads * kCopyUnits * 16;

__global__ void __launch_bounds__(kCopyThreads) cache_copy_kernel(const __grid_constant__ Copy p) {
  grid_dep_wait();
  grid_dep_launch();
  for (int64_t item = blockIdx.x; item < p.items; item += gridDim.x) {
    const int64_t pair = item / p.all;
    int chunk = (int)(item - pair * p.all), m = 0;
    const int from = p.src[pair], to = p.dst[pair];
    if (from == -1) continue;
    if ((unsigned)from >= (unsigned)p.pages || (unsigned)to >= (unsigned)p.pages) {
      if (threadIdx.x == 0) atomicOr(p.err, rows::kBadIndex);
      continue;
    }
    while (chunk >= p.chunks[m]) chunk -= p.chunks[m++];
    const int64_t bytes = p.bytes[m], at = (int64_t)chunk * kChunk + threadIdx.x * 16;
    const uint8_t* s = p.mat[m] + from * bytes + at;
    uint8_t* d = p.mat[m] + to * bytes + at;
    uint4 x[kCopyUnits];
#pragma unroll
    for (int u = 0; u < kCopyUnits; ++u)
      if (at + u * (kCopyThreads * 16) < bytes) x[u] = *reinterpret_cast<const uint4*>(s + u * (kCopyThreads * 16));
#pragma unroll
    for (int u = 0; u < kCopyUnits; ++u)
      if (at + u * (kCopyThreads * 16) < bytes) *reinterpret_cast<uint4*>(d + u * (kCopyThreads * 16)) = x[u];
  }
}

// ------------------------------------------------------------------- compact --
struct Compact {
  uint8_t* mat[2];  // keys, values
  float* scale[2];  // or null
  const int *table, *lens, *cu, *path, *kept;
  int64_t row_bytes;  // of a token's heads, a multiple of 16
  int stride, pages, log_page, H;
  int B, total;
  int parts, scale_parts;  // groups of 32 units, and of 32 heads' scales, of a row
  int* err;
};

// A warp moves 32 units (16 bytes, or a head's scale) of all rows that a sequence keeps,
// a lane one unit: it loads eight rows' and stores them, then the next eight.  Paths
// increase, so a row is read before, or with, the rows that are written over it.  The launch
// and a chain of four dependent loads bound it (256 trees of up to 64 drafts: 5.5 us).
constexpr int kCompactThreads = 128;
constexpr int kMoves = 8;

template <class T>
__device__ __forceinline__ void move_rows(const T* from, T* to, const int64_t (&src)[kMoves], const int64_t (&dst)[kMoves]) {
  T x[kMoves];
#pragma unroll
  for (int u = 0; u < kMoves; ++u)
    if (dst[u] >= 0) x[u] = from[src[u]];
#pragma unroll
  for (int u = 0; u < kMoves; ++u)
    if (dst[u] >= 0) to[dst[u]] = x[u];
}

__global__ void __launch_bounds__(kCompactThreads) cache_compact_kernel(const __grid_constant__ Compact p) {
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const bool falls = rows::offsets_fall(p.cu, p.B, threadIdx.x, kCompactThreads);
  if (blockIdx.x == 0 && warp == 0) rows::check_offsets(p.cu, p.B, p.total, p.err);
  const int64_t item = (int64_t)blockIdx.x * (kCompactThreads / 32) + warp;
  const int each = 2 * (p.parts + p.scale_parts);
  const int64_t b = item / each;
  if (__syncthreads_or(falls) || b >= p.B) return;
  int part = (int)(item - b * each);
  const int m = part >= each / 2;
  part -= m * (each / 2);
  const bool first = part == 0 && m == 0;  // the warp that reports
  const int q0 = p.cu[b], len = p.lens[b], kept = p.kept[b];
  const int64_t n = (int64_t)p.cu[b + 1] - q0;
  if ((b == 0 ? q0 != 0 : q0 < 0) || q0 + n > p.total || len < n || len > (int64_t)p.stride << p.log_page) {
    if (first && lane == 0) atomicOr(p.err, rows::kBadSeqlens);
    return;
  }
  bool bad = kept < 0 || kept > n;
  for (int j = lane; !bad && j < kept; j += 32) {
    const int at = p.path[q0 + j];
    bad = at < 0 || at >= n || (j > 0 && p.path[q0 + j - 1] >= at);
  }
  if (__any_sync(0xffffffffu, bad)) {
    if (first && lane == 0) atomicOr(p.err, rows::kBadIndex);
    return;
  }
  const int base = len - (int)n, page = 1 << p.log_page;
  const int64_t table = b * p.stride;
  for (int j0 = 0; j0 < kept; j0 += 32) {
    // this lane's move: rows of the cache, or -1
    int from = -1, to = -1;
    if (j0 + lane < kept) {
      const int at = p.path[q0 + j0 + lane], ps = base + at, pd = base + j0 + lane;
      if (at != j0 + lane) {
        const int is = p.table[table + (ps >> p.log_page)], id = p.table[table + (pd >> p.log_page)];
        if ((unsigned)is < (unsigned)p.pages && (unsigned)id < (unsigned)p.pages) {
          from = (is << p.log_page) + (ps & (page - 1));
          to = (id << p.log_page) + (pd & (page - 1));
        } else if (first) {
          atomicOr(p.err, rows::kBadIndex);
        }
      }
    }
    const uint32_t moves = __ballot_sync(0xffffffffu, to >= 0);
    for (int i = 0; i < 32 && moves >> i; i += kMoves) {
      if (!((moves >> i) & ((1u << kMoves) - 1))) continue;
      int64_t src[kMoves], dst[kMoves];
      const bool scales = part >= p.parts;
      const int unit = 32 * (scales ? part - p.parts : part) + lane;
      const bool live = scales ? unit < p.H : unit < p.row_bytes / 16;
#pragma unroll
      for (int u = 0; u < kMoves; ++u) {
        const int s = __shfl_sync(0xffffffffu, from, i + u), d = __shfl_sync(0xffffffffu, to, i + u);
        if (scales) {  // [pages, H, page]
          src[u] = (((int64_t)(s >> p.log_page) * p.H + unit) << p.log_page) + (s & (page - 1));
          dst[u] = (((int64_t)(d >> p.log_page) * p.H + unit) << p.log_page) + (d & (page - 1));
        } else {
          src[u] = s * (p.row_bytes / 16) + unit;
          dst[u] = d * (p.row_bytes / 16) + unit;
        }
        if (d < 0 || !live) dst[u] = -1;
      }
      if (scales)
        move_rows(p.scale[m], p.scale[m], src, dst);
      else
        move_rows(reinterpret_cast<const uint4*>(p.mat[m]), reinterpret_cast<uint4*>(p.mat[m]), src, dst);
    }
  }
}

// ---------------------------------------------------------------------- fork --
struct Fork {
  const int *table, *lens, *parents, *new_lens, *refs;
  int *refs_out, *out, *src, *dst;
  int *heir, *writer, *reader;  // [B] a row's first child, its first that writes to the last page, whether one only reads it
  int* taken;                   // [B] pages that the first child takes over
  int4* info;                   // [N] parent; 4 pages kept + 2 (first child) + 1 (copies the last); pages; first request
  int* order;                   // free pages, lowest first, as many as are asked for
  int B, N, W, pages, log_page;
  bool vec;  // counts lie on multiples of 16 bytes
  int ctas;  // of the cluster
  int* err;
};

// One cluster does all of it, in steps that its barrier parts: what it works on is
// some hundred kilobytes of integers, and a launch for each step would cost more than
// the step.  Pages are handed out lowest first, in the order of the rows that ask, and
// counts only ever add up, so no atomic's order shows in what comes out.  Latency bounds it,
// of four barriers and the dependent loads between them (64 rows going on: 10.5 us), and the
// cluster's 16 SMs where many counts change (256 rows forked to 512, 6000 positions: 26 us).
constexpr int kMaxForkCtas = 16;  // of a cluster (not a portable size)
constexpr int kForkThreads = 1024;
constexpr int kForkWarps = kForkThreads / 32;
constexpr int kAtOnce = 4;  // loads of a lane in flight

struct ForkShared {
  int free, asks;  // of this CTA's part
  int bad;             // error bits
  int free_of[kForkWarps];
  int warp[kForkWarps];
};

// Exclusive place of this thread among the CTA's, from its count; `sum` the CTA's count.
__device__ __forceinline__ int place_of(int count, int* warps, int& sum) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  int upto = count;
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
  sum = __reduce_add_sync(0xffffffffu, mine);
  return before + upto - count;
}

__device__ __forceinline__ int load_cluster32(const void* p, uint32_t rank) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(map_cluster(smem_u32(p), rank)) : "memory");
  return v;
}

// What becomes of new row i.
struct NewRow {
  int parent, had, needs, keep, last;
  bool grows;  // into a page that holds something
};
__device__ __forceinline__ NewRow new_row(const Fork& p, int i) {
  NewRow r;
  r.parent = p.parents[i];
  const int mask = (1 << p.log_page) - 1, len = r.parent >= 0 ? p.lens[r.parent] : 0, to = p.new_lens[i];
  r.had = (len + mask) >> p.log_page;
  r.needs = (to + mask) >> p.log_page;
  r.keep = min(r.had, r.needs);
  r.grows = to > len && (len & mask);
  r.last = r.had > 0 ? p.table[(int64_t)r.parent * p.W + r.had - 1] : -1;
  return r;
}

// Counts of pages i .. i + 3 (below hi; 1 behind it).
__device__ __forceinline__ int4 counts_at(const Fork& p, int i, int hi) {
  if (p.vec && i + 3 < hi) return *reinterpret_cast<const int4*>(p.refs + i);
  int4 x = make_int4(1, 1, 1, 1);
  if (i < hi) x.x = p.refs[i];
  if (i + 1 < hi) x.y = p.refs[i + 1];
  if (i + 2 < hi) x.z = p.refs[i + 2];
  if (i + 3 < hi) x.w = p.refs[i + 3];
  return x;
}

__global__ void __launch_bounds__(kForkThreads, 1) cache_fork_kernel(const __grid_constant__ Fork p) {
  __shared__ ForkShared sm;
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const uint32_t rank = cluster_ctarank();
  const int thread = (int)rank * kForkThreads + threadIdx.x, all = p.ctas * kForkThreads;
  const int wide = thread / 32, warps = all / 32;
  const int most = p.W << p.log_page;
  if (threadIdx.x == 0) sm.free = sm.asks = sm.bad = 0;
  __syncthreads();
  // each CTA has a run of the new rows
  const int run = (p.N + p.ctas - 1) / p.ctas;
  const int i0 = (int)min((int64_t)rank * run, (int64_t)p.N), i1 = (int)min((int64_t)i0 + run, (int64_t)p.N);

  // ------------------------------------------------ is the plan possible? --
  int bad = 0;
  for (int b = thread; b < p.B; b += all) p.heir[b] = p.writer[b] = INT_MAX, p.reader[b] = p.taken[b] = 0;
  for (int i = i0 + (int)threadIdx.x; i < i1; i += kForkThreads) {
    if (p.parents[i] < -1 || p.parents[i] >= p.B) bad |= rows::kBadIndex;
    if (p.new_lens[i] < 0 || p.new_lens[i] > most) bad |= rows::kBadSeqlens;
  }
  // each warp has a stretch of pages: counts copied, free ones counted
  const int stretch = ((p.pages + warps - 1) / warps + 127) & ~127;
  const int lo = (int)min((int64_t)wide * stretch, (int64_t)p.pages), hi = (int)min((int64_t)lo + stretch, (int64_t)p.pages);
  int mine = 0;
#pragma unroll 4
  for (int i = lo + 4 * lane; i < hi; i += 128) {
    const int4 x = counts_at(p, i, hi);
    mine += (x.x == 0) + (x.y == 0) + (x.z == 0) + (x.w == 0);
    if (p.refs_out == p.refs) continue;
    if (p.vec && i + 3 < hi) {
      *reinterpret_cast<int4*>(p.refs_out + i) = x;
    } else {
      p.refs_out[i] = x.x;
      if (i + 1 < hi) p.refs_out[i + 1] = x.y;
      if (i + 2 < hi) p.refs_out[i + 2] = x.z;
      if (i + 3 < hi) p.refs_out[i + 3] = x.w;
    }
  }
  for (int b = wide; b < p.B; b += warps) {
    const int len = p.lens[b];
    if (len < 0 || len > most) {
      bad |= rows::kBadSeqlens;
      continue;
    }
    const int n = (len + (1 << p.log_page) - 1) >> p.log_page;
    const int* row = p.table + (int64_t)b * p.W;
    for (int j = lane; j < n; j += 32 * kAtOnce) {
      int page[kAtOnce], count[kAtOnce];
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) page[u] = j + 32 * u < n ? row[j + 32 * u] : -1;
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) count[u] = (unsigned)page[u] < (unsigned)p.pages ? p.refs[page[u]] : 0;
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u)
        if (j + 32 * u < n && count[u] < 1) bad |= rows::kBadIndex;
    }
  }
  mine = __reduce_add_sync(0xffffffffu, mine);
  bad = __reduce_or_sync(0xffffffffu, bad);
  if (lane == 0) {
    sm.free_of[warp] = mine;
    atomicAdd(&sm.free, mine);
    if (bad) atomicOr(&sm.bad, bad);
  }
  cluster_sync();
  // (counts of pages and of requests are 32-bit numbers, and so are their sums)
  const bool other = lane < p.ctas;
  int there = other ? load_cluster32(&sm.free, lane) : 0;
  const int free_all = __reduce_add_sync(0xffffffffu, there);
  const int free_before = __reduce_add_sync(0xffffffffu, lane < (int)rank ? there : 0) +
                          __reduce_add_sync(0xffffffffu, lane < warp ? sm.free_of[lane] : 0);  // of the warp's stretch
  bad = __reduce_or_sync(0xffffffffu, other ? load_cluster32(&sm.bad, lane) : 0);

  // --------------------------------------------------- who writes where? --
  // (a thread's first row stays in registers)
  NewRow first{};
  if (!bad)
    for (int i = i0 + (int)threadIdx.x; i < i1; i += kForkThreads) {
      const NewRow r = new_row(p, i);
      if (i == i0 + (int)threadIdx.x) first = r;
      if (r.parent < 0) continue;
      atomicMin(p.heir + r.parent, i);
      if (r.grows)
        atomicMin(p.writer + r.parent, i);
      else if (r.keep == r.had)
        atomicOr(p.reader + r.parent, 1);
    }
  cluster_sync();
  // A row that grows into a page leaves it where nobody else has it, once the first
  // of those that grow has kept it; the others copy it.
  int asks = 0;
  for (int from = i0; from < i1 && !bad; from += kForkThreads) {
    const int i = from + threadIdx.x;
    int4 x = make_int4(-1, 0, 0, 0);
    if (i < i1) {
      const NewRow r = from == i0 ? first : new_row(p, i);
      bool c = false, heir = false;
      if (r.parent >= 0) {
        const int count = r.grows ? p.refs[r.last] : 1, reader = __ldcg(p.reader + r.parent),
                  writer = __ldcg(p.writer + r.parent);
        heir = __ldcg(p.heir + r.parent) == i;
        c = r.grows && !(count == 1 && !reader && writer == i);
        if (heir) p.taken[r.parent] = r.keep - c;
      }
      p.src[i] = c ? r.last : -1;
      x = make_int4(r.parent, 4 * (r.keep - c) + 2 * heir + c, r.needs, r.needs - r.keep + c);
    }
    int sum;
    x.w = asks + place_of(x.w, sm.warp, sum);  // among its CTA's
    if (i < i1) p.info[i] = x;
    asks += sum;
  }
  if (threadIdx.x == 0) sm.asks = asks;
  cluster_sync();
  there = other ? load_cluster32(&sm.asks, lane) : 0;
  const int asks_all = __reduce_add_sync(0xffffffffu, there);
  if (asks_all > free_all) bad |= rows::kNoPages;
  if (bad) {  // nothing changes hands
    if (thread == 0) atomicOr(p.err, bad);
    for (int64_t i = thread; i < (int64_t)p.N * p.W; i += all) p.out[i] = -1;
    for (int i = thread; i < p.N; i += all) p.src[i] = p.dst[i] = -1;
    cluster_sync();  // no CTA leaves while others read its shared memory
    return;
  }
  // the lowest free pages, as many as are asked for
  int at = free_before;
#pragma unroll 4
  for (int from = lo; from < hi; from += 128) {
    if (at >= asks_all) break;  // the same in the whole warp
    const int i = from + 4 * lane;
    const int4 x = counts_at(p, i, hi);
    const int is[4] = {x.x == 0, x.y == 0, x.z == 0, x.w == 0};
    int place = 0, sum = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t vote = __ballot_sync(0xffffffffu, is[e]);
      place += __popc(vote & ((1u << lane) - 1));
      sum += __popc(vote);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (is[e] && at + place < asks_all) p.order[at + place] = i + e;
      place += is[e];
    }
    at += sum;
  }
  cluster_sync();

  // --------------------------------------------------------- the new rows --
  for (int i = wide; i < p.N; i += warps) {
    const int4 x = __ldcg(p.info + i);
    const bool c = x.y & 1, heir = x.y & 2;
    const int held = x.y >> 2, needs = x.z;  // pages that stay the parent's, and of the row
    const int first = x.w + __reduce_add_sync(0xffffffffu, lane < i / run ? there : 0);  // of row i's CTA
    const int* row = p.table + (int64_t)x.x * p.W;
    for (int j0 = lane; j0 < p.W; j0 += 32 * kAtOnce) {
      int page[kAtOnce];
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        const int j = j0 + 32 * u;
        page[u] = j < held ? row[j] : j < needs ? __ldcg(p.order + first + (j - held)) : -1;
      }
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        const int j = j0 + 32 * u;
        if (j < p.W) p.out[(int64_t)i * p.W + j] = page[u];
        if (j < held) {
          if (!heir) atomicAdd(p.refs_out + page[u], 1);
        } else if (j < needs) {
          p.refs_out[page[u]] = 1;
          if (c && j == held) p.dst[i] = page[u];
        }
      }
    }
    if (!c && lane == 0) p.dst[i] = -1;
  }
  // old rows give up what their first child did not take over
  for (int b = wide; b < p.B; b += warps) {
    const int from = __ldcg(p.taken + b), n = (p.lens[b] + (1 << p.log_page) - 1) >> p.log_page;
    const int* row = p.table + (int64_t)b * p.W;
    for (int j = from + lane; j < n; j += 32 * kAtOnce) {
      int page[kAtOnce], count[kAtOnce];
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) page[u] = j + 32 * u < n ? row[j + 32 * u] : -1;
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) count[u] = page[u] >= 0 ? atomicSub(p.refs_out + page[u], 1) : 1;
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u)
        if (count[u] < 1) atomicOr(p.err, rows::kBadIndex);
    }
  }
}

}  // namespace pages
}  // namespace attn
