// Row-wise building blocks of the norm, cache and tree kernels: 16-byte vectors
// of bf16, the search of a packed token's sequence, sums over the lanes of a row.
#pragma once

#include <cuda_bf16.h>
#include <cstdint>

#include "sm100_ptx.cuh"

namespace attn {
namespace rows {

constexpr int kBadSeqlens = 2;  // bits of the library's error word
constexpr int kBadIndex = 8;

__device__ __forceinline__ void unpack(const uint4& w, float (&f)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(u[i] << 16);
    f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint4 pack(const float (&f)[8]) {
  return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
}

// Sum over the kLanes consecutive lanes that share a row.
template <int kLanes>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int off = 1; off < kLanes; off <<= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
  return x;
}

// The sequence of packed token t: the number of ends cu[1..B] that are <= t,
// found by the whole warp, 32 probes a step (two dependent loads for up to
// 1024 sequences).  B when t lies behind the last sequence.  Whatever cu
// holds, it reads cu[1..B] only.
__device__ __forceinline__ int find_sequence(const int* __restrict__ cu, int B, int t) {
  const int lane = threadIdx.x % 32;
  int lo = 0, n = B;  // the answer lies in [lo, lo + n]
  while (n > 32) {
    const int step = (n + 31) / 32;
    const int at = lo + (int)min((int64_t)(lane + 1) * step, (int64_t)n);  // the end of sequence at - 1
    const int cnt = __popc(__ballot_sync(0xffffffffu, cu[at] <= t));
    const int skip = (int)min((int64_t)cnt * step, (int64_t)n);
    lo += skip;
    n = min(step, n - skip);
  }
  const bool le = lane < n && cu[lo + 1 + lane] <= t;
  return lo + __popc(__ballot_sync(0xffffffffu, le));
}

// A warp's check of the packed offsets: from 0, never decreasing, at most total.
__device__ __forceinline__ void check_offsets(const int* __restrict__ cu, int B, int total, int* err) {
  const int lane = threadIdx.x % 32;
  bool bad = false;
  for (int i = lane; i <= B; i += 32) {
    const int c = cu[i];
    bad |= i == 0 ? c != 0 : c < cu[i - 1];
    bad |= c > total;
  }
  if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(err, kBadSeqlens);
}

// Whether the packed offsets decrease anywhere, as far as this one of `n` threads
// looks: then they place no token (a search in them finds any sequence).
__device__ __forceinline__ bool offsets_fall(const int* __restrict__ cu, int B, int thread, int n) {
  bool falls = false;
  for (int i = thread; i < B; i += n) falls |= cu[i + 1] < cu[i];
  return falls;
}

}  // namespace rows
}  // namespace attn
