// Writing packed keys and values into a paged cache, and reading it back.
//
// The heads of a token's keys, and of its values, are cut into chunks of kSteps
// row groups; a warp takes one chunk of tokens that are `step` apart, the next
// token's rows on their way while it works on the current ones; all warps
// together so sweep the packed rows in order, which DRAM serves faster than as
// many streams as there are warps.  d / 8 lanes
// hold a row, eight channels each: 16 bytes of bf16, 8 bytes of codes.  Writing,
// the row maximum is a shuffle reduction in bf16.  (With 16 codes a lane each 16-byte
// store fills half a sector: 113 us against 99.7 for the 612 MB of reading back a
// batch of eight.)  Every byte moves once, so HBM bounds both (launch latency for a few
// tokens: runs of one).
//
// A CTA first looks for a decrease in the offsets, all of them, with all its threads
// (one token for 64 sequences 2.65 -> 3.1 us, the batch of eight 97.4 -> 98.8; with each
// warp looking for itself 3.0, but 30 against 9.3 for 4096 sequences, and 105.9).
#pragma once

#include <climits>

#include "attn_rows.cuh"

namespace attn {
namespace cache {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kSteps = 4;

struct Pages {
  void *k, *v;
  float *ks, *vs;  // [pages, H, page]
  const int* table;
  int stride, pages, log_page, H;
};

struct Write {
  Pages c;
  const __nv_bfloat16 *k, *v;
  int64_t k_ts, v_ts;
  const int *lens, *cu;
  int B, total;
  int step;  // a warp takes tokens t, t + step, ..
  int* err;
};

struct Read {
  Pages c;
  __nv_bfloat16 *k, *v;
  const int* cu;
  int B, total;
  int step;  // a warp takes tokens t, t + step, ..
  int* err;
};

// Where a warp's tokens lie in the cache.  The search and the loads that depend
// on it happen once per sequence and page that its tokens fall in.
struct Cursor {
  int b = -1, start = 0, end = 0, shift = 0;  // packed tokens start .. end-1 sit at positions t + shift
  int page_at = -1;                           // index of the page in the sequence
  int64_t row0 = -1;                          // first row of that page, or -1
  bool ok = false;                            // the sequence's lengths are possible
};

// Row of packed token t of `total`, or -1 (behind the last sequence, or reported).
// lens null: the packed tokens are the whole sequences.  For the whole warp.
__device__ __forceinline__ int64_t find_row(Cursor& c, const Pages& pg, const int* __restrict__ cu,
                                            const int* __restrict__ lens, int B, int total, int t, int* err) {
  const int lane = threadIdx.x % 32;
  if (c.b < 0 || t < c.start || t >= c.end) {
    c.b = rows::find_sequence(cu, B, t);
    c.page_at = -1;
    c.ok = false;
    if (c.b >= B) {
      c.start = t, c.end = INT_MAX;  // nor do the tokens behind it
      return -1;
    }
    c.start = cu[c.b], c.end = cu[c.b + 1];
    // 64-bit differences: the offsets may hold anything
    const int64_t n = (int64_t)c.end - c.start, len = lens ? lens[c.b] : n;
    c.ok = (c.b > 0 ? c.start >= 0 : c.start == 0) && c.end <= total && t >= c.start && t < c.end &&
           len >= n && len <= (int64_t)pg.stride << pg.log_page;
    if (!c.ok) {
      if (lane == 0) atomicOr(err, rows::kBadSeqlens);
      c.start = t, c.end = t < INT_MAX ? t + 1 : t;  // the next token is looked up again
      return -1;
    }
    c.shift = (int)(len - n) - c.start;
  }
  if (!c.ok) return -1;
  const int pos = t + c.shift, at = pos >> pg.log_page;
  if (at != c.page_at) {
    c.page_at = at;
    const int page = pg.table[(int64_t)c.b * pg.stride + at];
    const bool in = (unsigned)page < (unsigned)pg.pages;
    if (!in && lane == 0) atomicOr(err, rows::kBadIndex);
    c.row0 = in ? (int64_t)page << pg.log_page : -1;
  }
  return c.row0 < 0 ? -1 : c.row0 + (pos & ((1 << pg.log_page) - 1));
}

// Two fp32 values as e4m3, nearest even, at most 448; lo in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// The two e4m3 codes of a 16-bit word as fp32 (exact: every code is an fp16 value).
__device__ __forceinline__ void from_e4m3x2(uint16_t w, float& lo, float& hi) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(w));
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.f32.f16 %0, a;\n cvt.f32.f16 %1, b;\n}\n"
      : "=f"(lo), "=f"(hi)
      : "r"(h));
}

// Largest magnitude of a pair of bf16, the pairs' maximum; a NaN wins.
__device__ __forceinline__ uint32_t abs_pair(uint32_t x) { return x & 0x7fff7fffu; }
__device__ __forceinline__ uint32_t max_pair(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

template <int D, bool kCodes>
__global__ void __launch_bounds__(kThreads, 4) cache_write_kernel(const __grid_constant__ Write p) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes, kChunk = kRows * kSteps;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int slice = lane % kLanes, row = lane / kLanes;
  grid_dep_wait();
  grid_dep_launch();
  const bool falls = rows::offsets_fall(p.cu, p.B, threadIdx.x, kThreads);
  if (blockIdx.x == 0 && warp == 0) rows::check_offsets(p.cu, p.B, p.total, p.err);
  const int H = p.c.H, chunks = (H + kChunk - 1) / kChunk;
  const int64_t item = (int64_t)blockIdx.x * kWarps + warp;
  const int64_t t0 = item / (2 * chunks);
  const int ch = (int)(item - t0 * 2 * chunks);
  const bool isv = ch >= chunks;
  const int h0 = (isv ? ch - chunks : ch) * kChunk + row;  // this lane's first head
  const int64_t ts = isv ? p.v_ts : p.k_ts;
  const __nv_bfloat16* src = (isv ? p.v : p.k) + h0 * D + 8 * slice;
  uint8_t* dst = static_cast<uint8_t*>(isv ? p.c.v : p.c.k) + (h0 * D + 8 * slice) * (kCodes ? 1 : 2);
  float* sdst = (isv ? p.c.vs : p.c.ks) + ((int64_t)h0 << p.c.log_page);
  auto load = [&](int64_t t, uint4 (&x)[kSteps]) {
    const __nv_bfloat16* at = src + t * ts;
#pragma unroll
    for (int u = 0; u < kSteps; ++u) {
      x[u] = make_uint4(0, 0, 0, 0);
      if (h0 + u * kRows < H) x[u] = *reinterpret_cast<const uint4*>(at + u * kRows * D);
    }
  };
  uint4 x[kSteps];
  if (t0 < p.step) load(t0, x);  // on its way while the token's place is looked up
  if (__syncthreads_or(falls) || t0 >= p.step) return;
  Cursor cur;
  for (int64_t t = t0; t < p.total; t += p.step) {
    uint4 next[kSteps];
    if (t + p.step < p.total) load(t + p.step, next);
    const int64_t r = find_row(cur, p.c, p.cu, p.lens, p.B, p.total, (int)t, p.err);
    if (r >= 0) {
      uint8_t* at = dst + r * H * D * (kCodes ? 1 : 2);
      if (!kCodes) {
#pragma unroll
        for (int u = 0; u < kSteps; ++u)
          if (h0 + u * kRows < H) *reinterpret_cast<uint4*>(at + u * kRows * D * 2) = x[u];
      } else {
        // the rows' largest magnitudes, in bf16 (a maximum rounds nothing)
        uint32_t top[kSteps];
#pragma unroll
        for (int u = 0; u < kSteps; ++u)
          top[u] = max_pair(max_pair(abs_pair(x[u].x), abs_pair(x[u].y)), max_pair(abs_pair(x[u].z), abs_pair(x[u].w)));
#pragma unroll
        for (int off = 1; off < kLanes; off <<= 1)
#pragma unroll
          for (int u = 0; u < kSteps; ++u) top[u] = max_pair(top[u], __shfl_xor_sync(0xffffffffu, top[u], off));
        // lane u of a row does the division of row group u for all its lanes
        uint32_t mine = top[0];
#pragma unroll
        for (int u = 1; u < kSteps; ++u) mine = slice % kSteps == u ? top[u] : mine;
        mine = max_pair(mine, mine >> 16);
        // the floor keeps 1 / scale finite; a NaN passes it
        float scale = __fdiv_rn(__uint_as_float(mine << 16), 448.f);
        if (scale < 0x1p-64f) scale = 0x1p-64f;
        const float inv = __frcp_rn(scale);
        const int64_t page = r >> p.c.log_page;
        if (slice < kSteps && h0 + slice * kRows < H)
          sdst[(page * H << p.c.log_page) + (r - (page << p.c.log_page)) + ((int64_t)slice * kRows << p.c.log_page)] = scale;
#pragma unroll
        for (int u = 0; u < kSteps; ++u) {
          const float f = __shfl_sync(0xffffffffu, inv, row * kLanes + u);
          float y[8];
          rows::unpack(x[u], y);
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] *= f;
          uint2 codes;
          codes.x = e4m3x2(y[0], y[1]) | e4m3x2(y[2], y[3]) << 16;
          codes.y = e4m3x2(y[4], y[5]) | e4m3x2(y[6], y[7]) << 16;
          if (h0 + u * kRows < H) *reinterpret_cast<uint2*>(at + u * kRows * D) = codes;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kSteps; ++u) x[u] = next[u];
  }
}

// A lane's eight channels: 16 bytes of bf16, or 8 of codes (in the low half).
template <bool kCodes>
__device__ __forceinline__ void load8(const uint8_t* at, uint32_t (&x)[kCodes ? 2 : 4]) {
  if (kCodes) {
    const uint2 v = *reinterpret_cast<const uint2*>(at);
    x[0] = v.x, x[1] = v.y;
  } else {
    const uint4 v = *reinterpret_cast<const uint4*>(at);
    x[0] = v.x, x[1] = v.y, x[kCodes ? 0 : 2] = v.z, x[kCodes ? 1 : 3] = v.w;
  }
}

template <int D, bool kCodes>
__global__ void __launch_bounds__(kThreads, 4) cache_read_kernel(const __grid_constant__ Read p) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes, kChunk = kRows * kSteps;
  constexpr int kSize = kCodes ? 1 : 2;  // bytes of a channel
  constexpr int kWords = kCodes ? 2 : 4;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int slice = lane % kLanes, row = lane / kLanes;
  grid_dep_wait();
  grid_dep_launch();
  const bool falls = rows::offsets_fall(p.cu, p.B, threadIdx.x, kThreads);
  if (blockIdx.x == 0 && warp == 0) rows::check_offsets(p.cu, p.B, p.total, p.err);
  const int H = p.c.H, chunks = (H + kChunk - 1) / kChunk;
  const int64_t item = (int64_t)blockIdx.x * kWarps + warp;
  const int64_t t0 = item / (2 * chunks);
  const int ch = (int)(item - t0 * 2 * chunks);
  const bool isv = ch >= chunks;
  const int h0 = (isv ? ch - chunks : ch) * kChunk + row;  // this lane's first head
  const uint8_t* src = static_cast<const uint8_t*>(isv ? p.c.v : p.c.k) + (h0 * D + 8 * slice) * kSize;
  const float* ssrc = (isv ? p.c.vs : p.c.ks) + ((int64_t)h0 << p.c.log_page);
  __nv_bfloat16* dst = (isv ? p.v : p.k) + h0 * D + 8 * slice;
  auto load = [&](int64_t r, uint32_t (&x)[kSteps][kWords], float (&sc)[kSteps]) {
    const uint8_t* at = src + r * H * D * kSize;
    const int64_t page = r >> p.c.log_page;
    const float* sat = ssrc + (page * H << p.c.log_page) + (r - (page << p.c.log_page));
#pragma unroll
    for (int u = 0; u < kSteps; ++u)
      if (r >= 0 && h0 + u * kRows < H) {
        load8<kCodes>(at + u * kRows * D * kSize, x[u]);
        if (kCodes) sc[u] = sat[(int64_t)u * kRows << p.c.log_page];
      }
  };
  if (__syncthreads_or(falls) || t0 >= p.step) return;
  Cursor cur;
  uint32_t x[kSteps][kWords];
  float sc[kSteps];
  int64_t r = find_row(cur, p.c, p.cu, nullptr, p.B, p.total, (int)t0, p.err);
  load(r, x, sc);
  for (int64_t t = t0; t < p.total; t += p.step) {
    uint32_t next[kSteps][kWords];
    float nsc[kSteps];
    int64_t rn = -1;
    if (t + p.step < p.total) {
      rn = find_row(cur, p.c, p.cu, nullptr, p.B, p.total, (int)(t + p.step), p.err);
      load(rn, next, nsc);
    }
    if (r >= 0) {
      __nv_bfloat16* at = dst + t * H * D;
#pragma unroll
      for (int u = 0; u < kSteps; ++u) {
        if (h0 + u * kRows >= H) continue;
        uint4 out;
        if (kCodes) {
          float f[8];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            from_e4m3x2((uint16_t)(x[u][j / 2] >> (16 * (j & 1))), f[2 * j], f[2 * j + 1]);
#pragma unroll
          for (int j = 0; j < 8; ++j) f[j] *= sc[u];
          out = rows::pack(f);
        } else {
          out = make_uint4(x[u][0], x[u][1], x[u][kCodes ? 0 : 2], x[u][kCodes ? 1 : 3]);
        }
        *reinterpret_cast<uint4*>(at + u * kRows * D) = out;
      }
    }
    r = rn;
#pragma unroll
    for (int u = 0; u < kSteps; ++u) {
      sc[u] = nsc[u];
#pragma unroll
      for (int j = 0; j < kWords; ++j) x[u][j] = next[u][j];
    }
  }
}

}  // namespace cache
}  // namespace attn
