// Norm of every query and key head with the rotary rotation, and its gradient.
//
// A row (token, head) of d channels is held by d / 8 lanes, 16 bytes each, so
// a warp holds 32 / (d / 8) rows (2 at d = 128, 4 at d = 64) and takes kSteps
// such groups of one token's heads.  The row's sum of squares is a shuffle
// reduction; the partner channel of a half-split pair sits rot / 16 lanes away
// in the same register, that of an interleaved pair in the same lane.  Nothing
// goes through shared memory in the forward; each element is read and written
// once, so HBM bounds it (and launch latency for a few tokens).
#pragma once

#include "attn_rows.cuh"

namespace attn {
namespace norm {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kSteps = 4;  // row groups a warp loads before it uses the first

struct Rotary {
  const float *cos, *sin;  // [P, half]
  const int* pos;          // [axes, T]
  int P, half, axes;
  int edge0, edge1;  // first pair of axis 1 and of axis 2
};

struct Fwd {
  const __nv_bfloat16 *q, *k, *wq, *wk;
  __nv_bfloat16 *qo, *ko;
  int64_t q_ts, k_ts, qo_ts, ko_ts;
  int T, Hq, Hk;
  float eps;
  Rotary rot;
  int* err;
};

struct Bwd {
  const __nv_bfloat16 *q, *k, *wq, *wk, *gq, *gk;
  __nv_bfloat16 *dq, *dk;
  int64_t q_ts, k_ts, gq_ts, gk_ts, dq_ts, dk_ts;
  int T, Hq, Hk;
  float eps;
  Rotary rot;
  float* part;  // [gridDim.x][2][D]
  int* err;
};

// cos and sin of this lane's pairs (8 half-split, 4 interleaved) for token t,
// and whether the lane's channels rotate at all.  False if a position lies
// outside the table.
template <bool kInter>
__device__ __forceinline__ bool load_angles(const Rotary& r, int T, int t, int slice, float (&c)[8],
                                            float (&s)[8], bool* rotates) {
  constexpr int kPairs = kInter ? 4 : 8;
  *rotates = 8 * slice < 2 * r.half;
  if (r.half == 0) return true;
  int p[3];
  bool ok = true;
#pragma unroll
  for (int a = 0; a < 3; ++a) {
    p[a] = a < r.axes ? r.pos[(int64_t)a * T + t] : 0;
    ok &= (unsigned)p[a] < (unsigned)r.P;
  }
  if (!ok) return false;
  if (*rotates) {
    const int j0 = kInter ? 4 * slice : (8 * slice) % r.half;
    const int ax0 = (j0 >= r.edge0) + (j0 >= r.edge1);
    const int ax1 = (j0 + kPairs - 1 >= r.edge0) + (j0 + kPairs - 1 >= r.edge1);
    if (ax0 == ax1) {
      const int64_t at = (int64_t)(ax0 == 0 ? p[0] : ax0 == 1 ? p[1] : p[2]) * r.half + j0;
#pragma unroll
      for (int i = 0; i < kPairs; i += 4) {
        const float4 cv = *reinterpret_cast<const float4*>(r.cos + at + i);
        const float4 sv = *reinterpret_cast<const float4*>(r.sin + at + i);
        c[i] = cv.x, c[i + 1] = cv.y, c[i + 2] = cv.z, c[i + 3] = cv.w;
        s[i] = sv.x, s[i + 1] = sv.y, s[i + 2] = sv.z, s[i + 3] = sv.w;
      }
    } else {  // an axis ends inside the lane's pairs
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        const int j = j0 + i;
        const int64_t at = (int64_t)(j >= r.edge1 ? p[2] : j >= r.edge0 ? p[1] : p[0]) * r.half + j;
        c[i] = r.cos[at];
        s[i] = r.sin[at];
      }
    }
  }
  return true;
}

// y rotated by (c, s), or by its inverse with kBack.  Every lane of the warp calls it.
template <bool kInter, bool kBack>
__device__ __forceinline__ void rotate(float (&y)[8], const float (&c)[8], const float (&s)[8],
                                       bool rotates, int half, int slice) {
  if (kInter) {
    if (!rotates) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = y[2 * i], b = y[2 * i + 1], si = kBack ? -s[i] : s[i];
      y[2 * i] = a * c[i] - b * si;
      y[2 * i + 1] = b * c[i] + a * si;
    }
  } else {
    const bool low = 8 * slice < half;
    const int lane = threadIdx.x % 32;
    const int src = rotates ? lane + (low ? half / 8 : -(half / 8)) : lane;
    const float sign = low != kBack ? -1.f : 1.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float other = __shfl_sync(0xffffffffu, y[i], src);
      if (rotates) y[i] = y[i] * c[i] + sign * (other * s[i]);
    }
  }
}

template <int D, bool kInter>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const __grid_constant__ Fwd p) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes, kChunk = kRows * kSteps;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int slice = lane % kLanes, row = lane / kLanes;
  grid_dep_wait();
  grid_dep_launch();
  const int H = p.Hq + p.Hk;
  const int chunks = (H + kChunk - 1) / kChunk;
  const int64_t item = (int64_t)blockIdx.x * kWarps + warp;
  if (item >= (int64_t)p.T * chunks) return;
  const int t = (int)(item / chunks);
  const int h0 = (int)(item - (int64_t)t * chunks) * kChunk;
  uint4 x[kSteps];
#pragma unroll
  for (int u = 0; u < kSteps; ++u) {
    const int h = h0 + u * kRows + row;
    x[u] = make_uint4(0, 0, 0, 0);
    if (h < H) {
      const __nv_bfloat16* src = h < p.Hq ? p.q + t * p.q_ts + (int64_t)h * D
                                          : p.k + t * p.k_ts + (int64_t)(h - p.Hq) * D;
      x[u] = *reinterpret_cast<const uint4*>(src + 8 * slice);
    }
  }
  float c[8], s[8], w[2][8];
  bool rotates;
  const bool ok = load_angles<kInter>(p.rot, p.T, t, slice, c, s, &rotates);
  if (!ok) {  // the same for the whole warp: one token
    if (lane == 0) atomicOr(p.err, rows::kBadIndex);
    return;
  }
  if (p.Hq) rows::unpack(*reinterpret_cast<const uint4*>(p.wq + 8 * slice), w[0]);
  if (p.Hk) rows::unpack(*reinterpret_cast<const uint4*>(p.wk + 8 * slice), w[1]);
#pragma unroll
  for (int u = 0; u < kSteps; ++u) {
    const int h = h0 + u * kRows + row;
    float y[8];
    rows::unpack(x[u], y);
    float sq = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) sq = fmaf(y[i], y[i], sq);
    const float r = rsqrtf(rows::row_sum<kLanes>(sq) * (1.0f / D) + p.eps);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = y[i] * r * (h < p.Hq ? w[0][i] : w[1][i]);
    rotate<kInter, false>(y, c, s, rotates, p.rot.half, slice);
    if (h < H) {
      __nv_bfloat16* dst = h < p.Hq ? p.qo + t * p.qo_ts + (int64_t)h * D
                                    : p.ko + t * p.ko_ts + (int64_t)(h - p.Hq) * D;
      *reinterpret_cast<uint4*>(dst + 8 * slice) = rows::pack(y);
    }
  }
}

// Gradient.  With n = x r and g the output's gradient rotated back:
//   dw = sum over rows of g n,   dn = g w,   dx = r (dn - n mean(dn n)),
// both row sums (x^2 and g w x) in one reduction.  Persistent CTAs; a lane
// keeps its 8 channels of dwq and dwk in registers over all its rows, the CTA
// adds its warps' through shared memory and writes one partial row, and
// norm_weight_kernel adds the CTAs' in a fixed order: no atomics, so results
// repeat bit for bit.
template <int D, bool kInter>
__global__ void __launch_bounds__(kThreads) norm_rope_bwd_kernel(const __grid_constant__ Bwd p) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes, kChunk = kRows * kSteps;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int slice = lane % kLanes, row = lane / kLanes;
  __shared__ float sm[kWarps][2][D];
  grid_dep_wait();
  grid_dep_launch();
  // a chunk holds heads of one kind, so that its weight gradient has one home
  const int cq = (p.Hq + kChunk - 1) / kChunk, ck = (p.Hk + kChunk - 1) / kChunk;
  const int chunks = cq + ck;
  float acc[2][8], w[2][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[0][i] = acc[1][i] = w[0][i] = w[1][i] = 0.f;
  if (p.Hq) rows::unpack(*reinterpret_cast<const uint4*>(p.wq + 8 * slice), w[0]);
  if (p.Hk) rows::unpack(*reinterpret_cast<const uint4*>(p.wk + 8 * slice), w[1]);
  for (int64_t item = (int64_t)blockIdx.x * kWarps + warp; item < (int64_t)p.T * chunks;
       item += (int64_t)gridDim.x * kWarps) {
    const int t = (int)(item / chunks);
    const int ch = (int)(item - (int64_t)t * chunks);
    const bool isk = ch >= cq;
    const int h0 = (isk ? ch - cq : ch) * kChunk, H = isk ? p.Hk : p.Hq;
    const __nv_bfloat16* xs = isk ? p.k + t * p.k_ts : p.q + t * p.q_ts;
    const __nv_bfloat16* gs = isk ? p.gk + t * p.gk_ts : p.gq + t * p.gq_ts;
    __nv_bfloat16* ds = isk ? p.dk + t * p.dk_ts : p.dq + t * p.dq_ts;
    uint4 xv[kSteps], gv[kSteps];
#pragma unroll
    for (int u = 0; u < kSteps; ++u) {
      const int h = h0 + u * kRows + row;
      xv[u] = gv[u] = make_uint4(0, 0, 0, 0);
      if (h < H) {
        xv[u] = *reinterpret_cast<const uint4*>(xs + (int64_t)h * D + 8 * slice);
        gv[u] = *reinterpret_cast<const uint4*>(gs + (int64_t)h * D + 8 * slice);
      }
    }
    float c[8], s[8];
    bool rotates;
    if (!load_angles<kInter>(p.rot, p.T, t, slice, c, s, &rotates)) {
      if (lane == 0) atomicOr(p.err, rows::kBadIndex);
      continue;
    }
#pragma unroll
    for (int u = 0; u < kSteps; ++u) {
      const int h = h0 + u * kRows + row;
      float x[8], g[8];
      rows::unpack(xv[u], x);
      rows::unpack(gv[u], g);
      rotate<kInter, true>(g, c, s, rotates, p.rot.half, slice);
      float sq = 0.f, dot = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        sq = fmaf(x[i], x[i], sq);
        dot = fmaf(g[i] * (isk ? w[1][i] : w[0][i]), x[i], dot);
      }
      sq = rows::row_sum<kLanes>(sq);
      dot = rows::row_sum<kLanes>(dot);
      const float r = rsqrtf(sq * (1.0f / D) + p.eps);
      const float coef = dot * (1.0f / D) * r * r;
      float dx[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        dx[i] = r * (g[i] * (isk ? w[1][i] : w[0][i]) - x[i] * coef);
        const float dw = h < H ? g[i] * (x[i] * r) : 0.f;
        acc[0][i] += isk ? 0.f : dw;
        acc[1][i] += isk ? dw : 0.f;
      }
      if (h < H) *reinterpret_cast<uint4*>(ds + (int64_t)h * D + 8 * slice) = rows::pack(dx);
    }
  }
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
      for (int off = kLanes; off < 32; off <<= 1)
        acc[m][i] += __shfl_xor_sync(0xffffffffu, acc[m][i], off);
      if (row == 0) sm[warp][m][8 * slice + i] = acc[m][i];
    }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
    float v = 0.f;
#pragma unroll
    for (int wp = 0; wp < kWarps; ++wp) v += sm[wp][i / D][i % D];
    p.part[(int64_t)blockIdx.x * 2 * D + i] = v;
  }
}

struct WeightSum {
  const float* part;  // [G][2][D]
  float *dwq, *dwk;
  int G, D;
};

// dwq and dwk: the G partial rows of 2 D floats added up.  32 columns a CTA,
// 32 slices of rows each, then the slices in shared memory.
__global__ void __launch_bounds__(1024) norm_weight_kernel(const __grid_constant__ WeightSum p) {
  __shared__ float sm[32][33];
  const int col = blockIdx.x * 32 + threadIdx.x % 32, sl = threadIdx.x / 32;
  grid_dep_wait();
  grid_dep_launch();
  float v = 0.f;
  for (int g = sl; g < p.G; g += 32) v += p.part[(int64_t)g * 2 * p.D + col];
  sm[sl][threadIdx.x % 32] = v;
  __syncthreads();
  if (sl == 0) {
    v = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) v += sm[i][threadIdx.x];
    float* dst = col < p.D ? p.dwq : p.dwk;
    if (dst) dst[col % p.D] = v;
  }
}

}  // namespace norm
}  // namespace attn
