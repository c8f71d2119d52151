// Writing packed keys and values into a paged cache, and reading it back.
//
// The rows of a token (its H key heads, then its H value heads) are cut into
// chunks; a warp takes one chunk of one token.  Writing: d / 8 lanes hold a
// row's bf16 channels, 16 bytes each; the row maximum is a shuffle reduction
// and the codes leave 8 bytes a lane.  Reading: d / 16 lanes hold a row's
// codes, 16 bytes each (bf16 caches: d / 8 lanes), and write 32 bytes a lane.
// Every byte moves once, so HBM bounds both (launch latency for a few tokens).
#pragma once

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
  int* err;
};

struct Read {
  Pages c;
  __nv_bfloat16 *k, *v;
  const int* cu;
  int B, total;
  int* err;
};

// Row of position pos of sequence b in the cache, or -1 with the error bit set
// if the table or its page is out of range.
__device__ __forceinline__ int64_t cache_row(const Pages& c, int b, int pos, int* err) {
  const int lane = threadIdx.x % 32;
  const int at = pos >> c.log_page;
  if (pos < 0 || at >= c.stride) {
    if (lane == 0) atomicOr(err, rows::kBadSeqlens);
    return -1;
  }
  const int page = c.table[(int64_t)b * c.stride + at];
  if ((unsigned)page >= (unsigned)c.pages) {
    if (lane == 0) atomicOr(err, rows::kBadIndex);
    return -1;
  }
  return ((int64_t)page << c.log_page) + (pos & ((1 << c.log_page) - 1));
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
__global__ void __launch_bounds__(kThreads) cache_write_kernel(const __grid_constant__ Write p) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes, kChunk = kRows * kSteps;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int slice = lane % kLanes, row = lane / kLanes;
  grid_dep_wait();
  grid_dep_launch();
  if (blockIdx.x == 0 && warp == 0) rows::check_offsets(p.cu, p.B, p.total, p.err);
  const int H = p.c.H, chunks = (2 * H + kChunk - 1) / kChunk;
  const int64_t item = (int64_t)blockIdx.x * kWarps + warp;
  if (item >= (int64_t)p.total * chunks) return;
  const int t = (int)(item / chunks);
  const int h0 = (int)(item - (int64_t)t * chunks) * kChunk;
  uint4 x[kSteps];  // on their way while the token's place is looked up
#pragma unroll
  for (int u = 0; u < kSteps; ++u) {
    const int h = h0 + u * kRows + row;
    x[u] = make_uint4(0, 0, 0, 0);
    if (h < 2 * H) {
      const __nv_bfloat16* src = h < H ? p.k + t * p.k_ts + (int64_t)h * D
                                       : p.v + t * p.v_ts + (int64_t)(h - H) * D;
      x[u] = *reinterpret_cast<const uint4*>(src + 8 * slice);
    }
  }
  const int b = rows::find_sequence(p.cu, p.B, t);
  if (b >= p.B) return;  // behind the last sequence
  const int start = p.cu[b], end = p.cu[b + 1], len = p.lens[b];
  // the whole sequence is refused when it is longer than its table
  if (start < 0 || t < start || t >= end || len < end - start || len > (int64_t)p.c.stride << p.c.log_page) {
    if (lane == 0) atomicOr(p.err, rows::kBadSeqlens);
    return;
  }
  const int64_t r = cache_row(p.c, b, len - (end - t), p.err);
  if (r < 0) return;
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

template <int D, bool kCodes>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const __grid_constant__ Read p) {
  constexpr int kPer = kCodes ? 16 : 8;  // channels a lane holds
  constexpr int kLanes = D / kPer, kRows = 32 / kLanes, kChunk = kRows * kSteps;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int slice = lane % kLanes, row = lane / kLanes;
  grid_dep_wait();
  grid_dep_launch();
  if (blockIdx.x == 0 && warp == 0) rows::check_offsets(p.cu, p.B, p.total, p.err);
  const int H = p.c.H, chunks = (2 * H + kChunk - 1) / kChunk;
  const int64_t item = (int64_t)blockIdx.x * kWarps + warp;
  if (item >= (int64_t)p.total * chunks) return;
  const int t = (int)(item / chunks);
  const int h0 = (int)(item - (int64_t)t * chunks) * kChunk;
  const int b = rows::find_sequence(p.cu, p.B, t);
  if (b >= p.B) return;
  const int start = p.cu[b], end = p.cu[b + 1];
  if (start < 0 || t < start || t >= end || end - start > (int64_t)p.c.stride << p.c.log_page) {
    if (lane == 0) atomicOr(p.err, rows::kBadSeqlens);
    return;
  }
  const int64_t r = cache_row(p.c, b, t - start, p.err);
  if (r < 0) return;
  uint4 x[kSteps];
  float sc[kSteps];
#pragma unroll
  for (int u = 0; u < kSteps; ++u) {
    const int h = h0 + u * kRows + row;
    const int hh = h < H ? h : h - H;
    x[u] = make_uint4(0, 0, 0, 0);
    sc[u] = 0.f;
    if (h < 2 * H) {
      const char* base = reinterpret_cast<const char*>(h < H ? p.c.k : p.c.v);
      x[u] = *reinterpret_cast<const uint4*>(base + ((r * H + hh) * D + kPer * slice) * (kCodes ? 1 : 2));
      if (kCodes) sc[u] = (h < H ? p.c.ks : p.c.vs)[scale_at(p.c, r, hh)];
    }
  }
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

}  // namespace cache
}  // namespace attn
