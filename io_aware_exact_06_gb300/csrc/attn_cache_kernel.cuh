// Writing packed keys and values into a paged cache, and reading it back.
//
// The rows of a token (its H key heads, then its H value heads) are cut into
// chunks; a warp takes one chunk of `run` tokens, `step` tokens apart, the next
// token's rows on their way while it works on the current ones; all warps
// together so sweep the packed rows in order, which DRAM serves faster than as
// many streams as there are warps.  Writing: d / 8
// lanes hold a row's bf16 channels, 16 bytes each; the row maximum is a shuffle
// reduction and the codes leave 8 bytes a lane.  Reading: d / 16 lanes hold a
// row's codes, 16 bytes each (bf16 caches: d / 8 lanes), and write 32 bytes a
// lane.  Every byte moves once, so HBM bounds both (launch latency for a few
// tokens: runs of one).
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

// Row of packed token t, or -1 (behind the last sequence, or reported).  lens
// null: the packed tokens are the whole sequences.  For the whole warp.
__device__ __forceinline__ int64_t find_row(Cursor& c, const Pages& pg, const int* __restrict__ cu,
                                            const int* __restrict__ lens, int B, int t, int* err) {
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
    c.ok = c.start >= 0 && t >= c.start && t < c.end && len >= n && len <= (int64_t)pg.stride << pg.log_page;
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

__device__ __forceinline__ int64_t scale_at(const Pages& c, int64_t r, int h) {
  const int64_t page = r >> c.log_page, in = r & ((1 << c.log_page) - 1);
  return ((page * c.H + h) << c.log_page) + in;
}

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
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

template <int D, bool kCodes>
__global__ void __launch_bounds__(kThreads, 4) cache_write_kernel(const __grid_constant__ Write p) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes, kChunk = kRows * kSteps;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int slice = lane % kLanes, row = lane / kLanes;
  grid_dep_wait();
  grid_dep_launch();
  if (blockIdx.x == 0 && warp == 0) rows::check_offsets(p.cu, p.B, p.total, p.err);
  const int H = p.c.H, chunks = (2 * H + kChunk - 1) / kChunk;
  const int64_t item = (int64_t)blockIdx.x * kWarps + warp;
  if (item / chunks >= p.step) return;
  const int t0 = (int)(item / chunks);
  const int h0 = (int)(item % chunks) * kChunk;
  auto load = [&](int t, uint4 (&x)[kSteps]) {
#pragma unroll
    for (int u = 0; u < kSteps; ++u) {
      const int h = h0 + u * kRows + row;
      x[u] = make_uint4(0, 0, 0, 0);
      if (h < 2 * H)
        x[u] = *reinterpret_cast<const uint4*>((h < H ? p.k + t * p.k_ts + (int64_t)h * D
                                                      : p.v + t * p.v_ts + (int64_t)(h - H) * D) + 8 * slice);
    }
  };
  uint4 x[kSteps];
  load(t0, x);  // on its way while the token's place is looked up
  Cursor cur;
  for (int64_t tt = t0; tt < p.total; tt += p.step) {
    const int t = (int)tt;
    uint4 next[kSteps];
    if (tt + p.step < p.total) load(t + p.step, next);
    const int64_t r = find_row(cur, p.c, p.cu, p.lens, p.B, t, p.err);
    if (r >= 0) {
#pragma unroll
      for (int u = 0; u < kSteps; ++u) {
        const int h = h0 + u * kRows + row;
        const int hh = h < H ? h : h - H;
        void* base = h < H ? p.c.k : p.c.v;
        const int64_t at = (r * H + hh) * D + 8 * slice;
        if (!kCodes) {
          if (h < 2 * H) *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(base) + at) = x[u];
          continue;
        }
        float f[8], top = 0.f;
        rows::unpack(x[u], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max_nan(top, fabsf(f[i]));
#pragma unroll
        for (int off = 1; off < kLanes; off <<= 1)
          top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, off));
        // the floor keeps 1 / scale finite; a NaN passes it
        float scale = __fdiv_rn(top, 448.f);
        if (scale < 0x1p-64f) scale = 0x1p-64f;
        const float inv = __frcp_rn(scale);
        if (h < 2 * H) {
          uint2 codes;
          codes.x = e4m3x2(f[0] * inv, f[1] * inv) | e4m3x2(f[2] * inv, f[3] * inv) << 16;
          codes.y = e4m3x2(f[4] * inv, f[5] * inv) | e4m3x2(f[6] * inv, f[7] * inv) << 16;
          *reinterpret_cast<uint2*>(reinterpret_cast<uint8_t*>(base) + at) = codes;
          if (slice == 0) (h < H ? p.c.ks : p.c.vs)[scale_at(p.c, r, hh)] = scale;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kSteps; ++u) x[u] = next[u];
  }
}

template <int D, bool kCodes>
__global__ void __launch_bounds__(kThreads, 4) cache_read_kernel(const __grid_constant__ Read p) {
  constexpr int kPer = kCodes ? 16 : 8;  // channels a lane holds
  constexpr int kLanes = D / kPer, kRows = 32 / kLanes, kChunk = kRows * kSteps;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int slice = lane % kLanes, row = lane / kLanes;
  grid_dep_wait();
  grid_dep_launch();
  if (blockIdx.x == 0 && warp == 0) rows::check_offsets(p.cu, p.B, p.total, p.err);
  const int H = p.c.H, chunks = (2 * H + kChunk - 1) / kChunk;
  const int64_t item = (int64_t)blockIdx.x * kWarps + warp;
  if (item / chunks >= p.step) return;
  const int t0 = (int)(item / chunks);
  const int h0 = (int)(item % chunks) * kChunk;
  Cursor cur;
  auto load = [&](int64_t r, uint4 (&x)[kSteps], float (&sc)[kSteps]) {
#pragma unroll
    for (int u = 0; u < kSteps; ++u) {
      const int h = h0 + u * kRows + row;
      const int hh = h < H ? h : h - H;
      x[u] = make_uint4(0, 0, 0, 0);
      sc[u] = 0.f;
      if (r >= 0 && h < 2 * H) {
        const char* base = reinterpret_cast<const char*>(h < H ? p.c.k : p.c.v);
        x[u] = *reinterpret_cast<const uint4*>(base + ((r * H + hh) * D + kPer * slice) * (kCodes ? 1 : 2));
        if (kCodes) sc[u] = (h < H ? p.c.ks : p.c.vs)[scale_at(p.c, r, hh)];
      }
    }
  };
  uint4 x[kSteps];
  float sc[kSteps];
  int64_t r = find_row(cur, p.c, p.cu, nullptr, p.B, t0, p.err);
  load(r, x, sc);
  for (int64_t tt = t0; tt < p.total; tt += p.step) {
    const int t = (int)tt;
    uint4 next[kSteps];
    float nsc[kSteps];
    int64_t rn = -1;
    if (tt + p.step < p.total) {
      rn = find_row(cur, p.c, p.cu, nullptr, p.B, t + p.step, p.err);
      load(rn, next, nsc);
    }
    if (r >= 0) {
#pragma unroll
      for (int u = 0; u < kSteps; ++u) {
        const int h = h0 + u * kRows + row;
        if (h >= 2 * H) continue;
        __nv_bfloat16* dst =
            (h < H ? p.k + ((int64_t)t * H + h) * D : p.v + ((int64_t)t * H + h - H) * D) + kPer * slice;
        if (!kCodes) {
          *reinterpret_cast<uint4*>(dst) = x[u];
          continue;
        }
        const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float f[8];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            from_e4m3x2((uint16_t)(w[2 * i + j / 2] >> (16 * (j & 1))), f[2 * j], f[2 * j + 1]);
#pragma unroll
          for (int j = 0; j < 8; ++j) f[j] *= sc[u];
          *reinterpret_cast<uint4*>(dst + 8 * i) = rows::pack(f);
        }
      }
    }
    r = rn;
#pragma unroll
    for (int u = 0; u < kSteps; ++u) x[u] = next[u], sc[u] = nsc[u];
  }
}

}  // namespace cache
}  // namespace attn
