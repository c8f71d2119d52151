// Norm of every query and key head with the rotary rotation, and its gradient.
//
// A row (token, head) of d channels is held by d / 8 lanes, so a warp holds
// 32 / (d / 8) rows (2 at d = 128, 4 at d = 64) at a time.  A lane holds two
// groups of four neighbouring channels, chosen so that both channels of a pair
// are its own: groups s and s + rot / 8 of a half-split rotation, neighbouring
// groups of an interleaved one and of the channels that do not rotate.  So the
// rotation needs no exchange and a lane only its own four cosines and sines (a
// 16-byte slice of the row instead took 8 shuffles a row and 16 registers of
// angles); the row's sum of squares is a shuffle reduction.  Each element
// is read and written once: HBM and instruction issue bound it (launch latency for
// a few tokens).
//
// The heads of a token are cut into chunks of kSteps (forward) or kBwdSteps row
// groups, and a warp takes runs of a token's chunks, one run after the other:
// the whole token when there are tokens enough to fill the GPU four times over,
// one chunk when there are few.  Loads run a chunk ahead: each lane copies its own
// channels to its own place in shared memory (cp.async) and reads them back there,
// so no thread waits for another and no register is held.  More in flight is
// slower: 16381 tokens of 32 + 8 heads, d = 128, take 61.7 us (5.5 TB/s) forward
// with two stages, 62.5 with three, 63.6 with four, 67.3 with two and a fourth CTA
// an SM; the gradient of 16384 tokens 92.7 us (5.5 TB/s), 94.7 with three stages.
#pragma once

#include "attn_rows.cuh"

namespace attn {
namespace norm {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kSteps = 4;     // row groups of a chunk, forward
constexpr int kBwdSteps = 2;  // gradient: two tensors are loaded
constexpr int kStages = 2;    // chunks in shared memory, forward and gradient: 64 bytes a lane each
constexpr int kSmem = kStages * kThreads * 64;

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
  int run;  // chunks of a warp
  float eps;
  Rotary rot;
  int* err;
};

struct Bwd {
  const __nv_bfloat16 *x[2], *w[2], *g[2];  // queries, keys
  __nv_bfloat16* dx[2];
  int64_t x_ts[2], g_ts[2], dx_ts[2];
  int H[2], run[2];
  int T;
  int ctas_q;  // CTAs 0 .. ctas_q - 1 take the queries, the others the keys
  float eps;
  Rotary rot;
  float* part;  // [gridDim.x][D]
  int* err;
};

// Two fp32 values in a 64-bit register and the packed instructions on them: half
// the issue slots of a row's arithmetic, which bounds the gradient.
typedef unsigned long long Two;
__device__ __forceinline__ Two two(float lo, float hi) {
  Two r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void parts(Two x, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x));
}
__device__ __forceinline__ Two mul2(Two a, Two b) {
  Two r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ Two add2(Two a, Two b) {
  Two r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ Two fma2(Two a, Two b, Two c) {
  Two r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ Two swapped(Two x) {
  float lo, hi;
  parts(x, lo, hi);
  return two(hi, lo);
}
// Two bf16 (a word) as fp32, and back with one rounding.
__device__ __forceinline__ Two wide(uint32_t w) { return two(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)); }
__device__ __forceinline__ uint32_t narrow(Two x) {
  float lo, hi;
  parts(x, lo, hi);
  return rows::pack2(lo, hi);
}
// A lane's eight channels as four pairs.
__device__ __forceinline__ void wide(const uint4& v, Two (&y)[4]) {
  y[0] = wide(v.x), y[1] = wide(v.y), y[2] = wide(v.z), y[3] = wide(v.w);
}
__device__ __forceinline__ uint4 narrow(const Two (&y)[4]) {
  return make_uint4(narrow(y[0]), narrow(y[1]), narrow(y[2]), narrow(y[3]));
}

// The first channels of lane `slice`'s two groups.
template <bool kInter>
__device__ __forceinline__ void lane_channels(int half, int slice, int& a, int& b) {
  if (kInter || 8 * slice >= 2 * half) {
    a = 8 * slice;
    b = a + 4;
  } else {
    a = 4 * slice;
    b = a + half;
  }
}

// A lane's eight channels of a row: group a in the low half, b in the high.
__device__ __forceinline__ uint4 load_row(const __nv_bfloat16* row, int a, int b) {
  const uint2 lo = *reinterpret_cast<const uint2*>(row + a), hi = *reinterpret_cast<const uint2*>(row + b);
  return make_uint4(lo.x, lo.y, hi.x, hi.y);
}
__device__ __forceinline__ void store_row(__nv_bfloat16* row, int a, int b, const uint4& v) {
  *reinterpret_cast<uint2*>(row + a) = make_uint2(v.x, v.y);
  *reinterpret_cast<uint2*>(row + b) = make_uint2(v.z, v.w);
}

// cos and sin of this lane's four pairs for token t (1 and 0 where its channels
// do not rotate).  False if a position lies outside the table.
template <bool kInter>
__device__ __forceinline__ bool load_angles(const Rotary& r, int T, int t, int slice, float (&c)[4], float (&s)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = 1.f, s[i] = 0.f;
  if (r.half == 0) return true;
  int p[3];
  bool ok = true;
#pragma unroll
  for (int a = 0; a < 3; ++a) {
    p[a] = a < r.axes ? r.pos[(int64_t)a * T + t] : 0;
    ok &= (unsigned)p[a] < (unsigned)r.P;
  }
  if (!ok) return false;
  const int j0 = 4 * slice;  // the lane's first pair, half-split or interleaved
  if (j0 < r.half) {
    const int ax0 = (j0 >= r.edge0) + (j0 >= r.edge1);
    const int ax1 = (j0 + 3 >= r.edge0) + (j0 + 3 >= r.edge1);
    if (ax0 == ax1) {
      const int64_t at = (int64_t)(ax0 == 0 ? p[0] : ax0 == 1 ? p[1] : p[2]) * r.half + j0;
      const float4 cv = *reinterpret_cast<const float4*>(r.cos + at);
      const float4 sv = *reinterpret_cast<const float4*>(r.sin + at);
      c[0] = cv.x, c[1] = cv.y, c[2] = cv.z, c[3] = cv.w;
      s[0] = sv.x, s[1] = sv.y, s[2] = sv.z, s[3] = sv.w;
    } else {  // an axis ends inside the lane's pairs
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int j = j0 + i;
        const int64_t at = (int64_t)(j >= r.edge1 ? p[2] : j >= r.edge0 ? p[1] : p[0]) * r.half + j;
        c[i] = r.cos[at];
        s[i] = r.sin[at];
      }
    }
  }
  return true;
}

// A lane's rotation: the factors of y and of the other channel of its pair.
// Half-split, pair i of channels (i, i + 4): own[i / 2], other[i / 2] hold two
// pairs; interleaved, (2 i, 2 i + 1): own[i], other[i] hold (c, c) and (-s, s).
// kBack turns the other way.  kPart: some channels do not rotate (`on` 0 in their
// lanes, else all ones).  Turned by cos = 1 and sin = 0 alone an infinity or a NaN
// would reach the other channel of the pair through 0 inf.  (Half of the channels
// rotated, 16381 tokens: 63.0 us with the mask, 66.6 with a branch, 63.9 with
// predicated products; full rotation, which has none of it, 61.8.)
template <bool kInter, bool kBack, bool kPart>
struct Turn {
  Two own[kInter ? 4 : 2], other[kInter ? 4 : 2];
  __device__ __forceinline__ void set(const float (&c)[4], const float (&s0)[4]) {
    float s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] = kBack ? -s0[i] : s0[i];
    if (kInter) {
#pragma unroll
      for (int i = 0; i < 4; ++i) own[i] = two(c[i], c[i]), other[i] = two(-s[i], s[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) own[i] = two(c[2 * i], c[2 * i + 1]), other[i] = two(s[2 * i], s[2 * i + 1]);
    }
  }
  __device__ __forceinline__ void turn(Two (&y)[4], Two on) const {
    auto partner = [&](Two x) { return kPart ? x & on : x; };
    if (kInter) {
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = fma2(partner(swapped(y[i])), other[i], mul2(y[i], own[i]));
    } else {
      const Two minus = two(-1.f, -1.f);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const Two a = y[i], b = y[i + 2], bs = mul2(partner(b), other[i]);
        y[i] = fma2(a, own[i], mul2(bs, minus));
        y[i + 2] = fma2(b, own[i], mul2(partner(a), other[i]));
      }
    }
  }
};

// 8 bytes from global to shared memory; zeros where `there` is false.
__device__ __forceinline__ void copy8(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(there ? 8 : 0) : "memory");
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Until this thread's copies of all but its last kStages - 2 chunks have landed.
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
}
__device__ __forceinline__ uint4 lane_load(uint32_t a) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "r"(a)
               : "memory");
  return r;
}

// A warp's chunks in order: run after run (item, item + stride, ..), chunk after
// chunk of a run.
struct Runs {
  int64_t item, items, stride;
  int runs, run, chunks;  // runs of a token, chunks of a run and of a token
  int t, ch, end;
  __device__ __forceinline__ void place() {
    t = (int)(item / runs);
    ch = (int)(item - (int64_t)t * runs) * run;
    end = min(chunks, ch + run);
  }
  __device__ __forceinline__ bool more() const { return item < items; }
  // true when the next chunk begins a run
  __device__ __forceinline__ bool next() {
    if (++ch < end) return false;
    item += stride;
    if (more()) place();
    return true;
  }
};

template <int D, bool kInter, bool kPart>
__global__ void __launch_bounds__(kThreads, 3) norm_rope_kernel(const __grid_constant__ Fwd p) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes, kChunk = kRows * kSteps;
  extern __shared__ __align__(16) uint8_t smem[];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int slice = lane % kLanes, row = lane / kLanes;
  const uint32_t mine = smem_u32(smem) + (warp * kStages * kSteps * 32 + lane) * 16;
  grid_dep_wait();
  grid_dep_launch();
  const int H = p.Hq + p.Hk;
  int ca, cb;
  lane_channels<kInter>(p.rot.half, slice, ca, cb);
  const Two on = 4 * slice < p.rot.half ? ~0ull : 0ull;  // the lane's channels rotate
  Runs use;
  use.chunks = (H + kChunk - 1) / kChunk;
  use.run = p.run;
  use.runs = (use.chunks + p.run - 1) / p.run;
  use.items = (int64_t)p.T * use.runs;
  use.stride = (int64_t)gridDim.x * kWarps;
  use.item = (int64_t)blockIdx.x * kWarps + warp;
  if (!use.more()) return;
  use.place();
  Runs ahead = use;
  int slot = 0;
  auto feed = [&]() {
    if (ahead.more()) {
      const __nv_bfloat16* qs = p.q + ahead.t * p.q_ts;
      const __nv_bfloat16* ks = p.k + ahead.t * p.k_ts;
#pragma unroll
      for (int u = 0; u < kSteps; ++u) {
        const int h = ahead.ch * kChunk + u * kRows + row;
        const __nv_bfloat16* src = h < p.Hq ? qs + h * D : ks + (h - p.Hq) * D;
        if (h >= H) src = p.Hq ? p.q : p.k;  // not read
        const uint32_t dst = mine + (slot * kSteps + u) * 512;
        copy8(dst, src + ca, h < H);
        copy8(dst + 8, src + cb, h < H);
      }
      ahead.next();
    }
    copies_done();
    slot = slot == kStages - 1 ? 0 : slot + 1;
  };
#pragma unroll 1
  for (int i = 0; i < kStages - 1; ++i) feed();
  uint4 wq = make_uint4(0, 0, 0, 0), wk = wq;
  if (p.Hq) wq = load_row(p.wq, ca, cb);
  if (p.Hk) wk = load_row(p.wk, ca, cb);
  Turn<kInter, false, kPart> turn;
  bool ok = false, fresh = true;
  int from = 0;
  while (use.more()) {
    const int t = use.t, ch = use.ch;
    if (fresh) {  // the same for the whole warp: one token
      float c[4], s[4];
      ok = load_angles<kInter>(p.rot, p.T, t, slice, c, s);
      turn.set(c, s);
      if (!ok && lane == 0) atomicOr(p.err, rows::kBadIndex);
    }
    copies_wait();
    feed();
    if (ok) {
      __nv_bfloat16* qd = p.qo + t * p.qo_ts;
      __nv_bfloat16* kd = p.ko + t * p.ko_ts;
#pragma unroll
      for (int u = 0; u < kSteps; ++u) {
        const int h = ch * kChunk + u * kRows + row;
        const bool isq = h < p.Hq;
        Two y[4], w[4];
        wide(lane_load(mine + (from * kSteps + u) * 512), y);
        wide(isq ? wq : wk, w);
        Two sq2 = mul2(y[0], y[0]);
#pragma unroll
        for (int i = 1; i < 4; ++i) sq2 = fma2(y[i], y[i], sq2);
        float sq, hi;
        parts(sq2, sq, hi);
        const float r = rsqrtf(rows::row_sum<kLanes>(sq + hi) * (1.0f / D) + p.eps);
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = mul2(mul2(y[i], two(r, r)), w[i]);
        turn.turn(y, on);
        if (h < H) store_row(isq ? qd + h * D : kd + (h - p.Hq) * D, ca, cb, narrow(y));
      }
    }
    from = from == kStages - 1 ? 0 : from + 1;
    fresh = use.next();
  }
}

// Gradient.  With n = x r and g the output's gradient rotated back:
//   dw = sum over rows of g n,   dn = g w,   dx = r (dn - n mean(dn n)),
// both row sums (x^2 and g w x) in one reduction.  Persistent CTAs, each for
// queries or for keys alone (in proportion to their heads), so that a lane
// carries one weight and the 8 channels of one weight gradient in registers over
// all its rows; the CTA adds its warps' through shared memory and writes one
// partial row, and norm_weight_kernel adds the CTAs' in a fixed order: no
// atomics, so results repeat bit for bit.
template <int D, bool kInter, bool kPart>
__global__ void __launch_bounds__(kThreads, 2) norm_rope_bwd_kernel(const __grid_constant__ Bwd p) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes, kChunk = kRows * kBwdSteps;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float sm[kWarps][D];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int slice = lane % kLanes, row = lane / kLanes;
  const uint32_t mine = smem_u32(smem) + (warp * kStages * 2 * kBwdSteps * 32 + lane) * 16;
  grid_dep_wait();
  grid_dep_launch();
  const int kind = (int)blockIdx.x >= p.ctas_q;
  const int cta = blockIdx.x - (kind ? p.ctas_q : 0), ctas = kind ? gridDim.x - p.ctas_q : p.ctas_q;
  const int H = p.H[kind];
  Runs use;
  use.chunks = (H + kChunk - 1) / kChunk;
  use.run = p.run[kind];
  use.runs = (use.chunks + use.run - 1) / use.run;
  use.items = (int64_t)p.T * use.runs;
  use.stride = (int64_t)ctas * kWarps;
  use.item = (int64_t)cta * kWarps + warp;
  if (use.more()) use.place();
  Runs ahead = use;
  int ca, cb;
  lane_channels<kInter>(p.rot.half, slice, ca, cb);
  const Two on = 4 * slice < p.rot.half ? ~0ull : 0ull;  // the lane's channels rotate
  const __nv_bfloat16 *xb = p.x[kind], *gb = p.g[kind];
  __nv_bfloat16* db = p.dx[kind];
  const int64_t x_ts = p.x_ts[kind], g_ts = p.g_ts[kind], dx_ts = p.dx_ts[kind];
  int slot = 0;
  auto feed = [&]() {
    if (ahead.more()) {
      const __nv_bfloat16 *xs = xb + ahead.t * x_ts, *gs = gb + ahead.t * g_ts;
#pragma unroll
      for (int u = 0; u < kBwdSteps; ++u) {
        const int h = ahead.ch * kChunk + u * kRows + row;
        const bool there = h < H;
        const int at = there ? h * D : 0;
        const uint32_t dst = mine + (slot * kBwdSteps + u) * 1024;
        copy8(dst, xs + at + ca, there);
        copy8(dst + 8, xs + at + cb, there);
        copy8(dst + 512, gs + at + ca, there);
        copy8(dst + 520, gs + at + cb, there);
      }
      ahead.next();
    }
    copies_done();
    slot = slot == kStages - 1 ? 0 : slot + 1;
  };
#pragma unroll 1
  for (int i = 0; i < kStages - 1; ++i) feed();
  Two acc[4], w[4];
  wide(load_row(p.w[kind], ca, cb), w);
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i] = two(0.f, 0.f);
  Turn<kInter, true, kPart> turn;
  bool ok = false, fresh = true;
  int from = 0;
  while (use.more()) {
    const int t = use.t, ch = use.ch;
    if (fresh) {
      float c[4], s[4];
      ok = load_angles<kInter>(p.rot, p.T, t, slice, c, s);
      turn.set(c, s);
      if (!ok && lane == 0) atomicOr(p.err, rows::kBadIndex);
    }
    copies_wait();
    feed();
    if (ok) {
#pragma unroll
      for (int u = 0; u < kBwdSteps; ++u) {
        const int h = ch * kChunk + u * kRows + row;
        const uint32_t at = mine + (from * kBwdSteps + u) * 1024;
        Two x[4], g[4];
        wide(lane_load(at), x);
        wide(lane_load(at + 512), g);
        turn.turn(g, on);
        Two sq2 = mul2(x[0], x[0]), xg[4], dot2;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          xg[i] = mul2(x[i], g[i]);
          if (i) sq2 = fma2(x[i], x[i], sq2);
          dot2 = i ? fma2(xg[i], w[i], dot2) : mul2(xg[i], w[i]);
        }
        float sa, sb, da, db2;
        parts(sq2, sa, sb);
        parts(dot2, da, db2);
        Two sums = two(sa + sb, da + db2);
#pragma unroll
        for (int off = 1; off < kLanes; off <<= 1) {
          float a, b;
          parts(sums, a, b);
          sums = add2(sums, two(__shfl_xor_sync(0xffffffffu, a, off), __shfl_xor_sync(0xffffffffu, b, off)));
        }
        float sq, dot;
        parts(sums, sq, dot);
        // rows that do not exist hold zeros, and with eps = 0 would give 0 * inf
        const float r = h < H ? rsqrtf(sq * (1.0f / D) + p.eps) : 0.f;
        const float coef = -dot * (1.0f / D) * r * r;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc[i] = fma2(xg[i], two(r, r), acc[i]);
          x[i] = mul2(fma2(x[i], two(coef, coef), mul2(g[i], w[i])), two(r, r));
        }
        if (h < H) store_row(db + t * dx_ts + h * D, ca, cb, narrow(x));
      }
    }
    from = from == kStages - 1 ? 0 : from + 1;
    fresh = use.next();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a, b;
    parts(acc[i], a, b);
#pragma unroll
    for (int off = kLanes; off < 32; off <<= 1) {
      a += __shfl_xor_sync(0xffffffffu, a, off);
      b += __shfl_xor_sync(0xffffffffu, b, off);
    }
    const int ch = (i < 2 ? ca : cb) + 2 * (i & 1);
    if (row == 0) sm[warp][ch] = a, sm[warp][ch + 1] = b;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < D; i += kThreads) {
    float v = 0.f;
#pragma unroll
    for (int wp = 0; wp < kWarps; ++wp) v += sm[wp][i];
    p.part[(int64_t)blockIdx.x * D + i] = v;
  }
}

struct WeightSum {
  const float* part;  // [Gq + Gk][D]
  float *dwq, *dwk;
  int Gq, Gk, D;
};

// dwq and dwk: the partial rows of their CTAs added up.  32 columns a CTA, 32
// slices of rows each, then the slices in shared memory.
__global__ void __launch_bounds__(1024) norm_weight_kernel(const __grid_constant__ WeightSum p) {
  __shared__ float sm[32][33];
  const int per = p.D / 32, lane = threadIdx.x % 32, sl = threadIdx.x / 32;
  const bool isk = (int)blockIdx.x >= per;
  const int col = (blockIdx.x - (isk ? per : 0)) * 32 + lane;
  const float* part = p.part + (isk ? (int64_t)p.Gq * p.D : 0) + col;
  const int G = isk ? p.Gk : p.Gq;
  grid_dep_wait();
  grid_dep_launch();
  float v = 0.f;
#pragma unroll 4
  for (int g = sl; g < G; g += 32) v += part[(int64_t)g * p.D];
  sm[sl][lane] = v;
  __syncthreads();
  if (sl == 0) {
    v = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) v += sm[i][lane];
    float* dst = isk ? p.dwk : p.dwq;
    if (dst) dst[col] = v;
  }
}

}  // namespace norm
}  // namespace attn
