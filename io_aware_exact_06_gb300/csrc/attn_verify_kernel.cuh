// Verification of drafted tokens against the target's probabilities.
//
// A walk from the first new token down its tree.  At a node with target row p and draft
// row q, after j rejected children, what is left of the target is
//   w_j = max(p - s_j q, 0),   s_0 = 0,  s_(j+1) = s_j + z_j,  z_0 = 1,  z_j = sum w_j
// (the residual of a rejection, taken without norming it: max(max(p - a q, 0) - b q, 0) is
// max(p - (a + b) q, 0)).  The next child, token x, is accepted where u q(x) z_j < w_j(x).
// Without q drafts count as certain: w is p with rejected tokens at 0, z is 1 less their
// p.  Where no child is left the next token is the first x with C(x) > u C(V - 1), C the
// running sum of w (of p where nothing is left of it).
//
// What the tests need of the rows is gathered at the start, two values for each token, so
// the walk itself waits for no memory; only a rejection with a sibling after it, and the
// end, need a pass over rows of V.  One cluster has a sequence; a pass is cut evenly over
// its CTAs, which read the last node's rows once: HBM bounds a large batch, a few
// dependent loads and barriers a small one.
//
// The tests are in fp64.  Sums are exact: a weight is an integer, p - s q in units of
// 2^-45 (up to 2^18 of them fit 64 bits), s q taken in two fp32 parts, so C does not depend
// on how a row is cut, and a draw next to a border falls where it does in fp64.
#pragma once

#include "attn_rows.cuh"

namespace attn {
namespace verify {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxNew = 64;
constexpr int kMaxV = 1 << 18;
constexpr int kSeg = 1024;  // elements that a warp sums at a time
constexpr int kMaxSegs = kMaxV / kSeg;
constexpr int kMaxCluster = 8;

struct Params {
  const int* tokens;
  const void *p, *q;  // target and draft rows
  int64_t p_stride, q_stride;
  const int *cu, *lens;
  const int64_t* mask;
  const float *u, *u_next;
  int *path, *kept, *next, *lens_out;
  int B, total, V, ctas;  // of a cluster
  int* err;
};

__device__ __forceinline__ float clean(float x) { return fminf(fmaxf(x, 0.f), 1.f); }  // NaN: 0
__device__ __forceinline__ float load(const float* x) { return *x; }
__device__ __forceinline__ float load(const __nv_bfloat16* x) { return __bfloat162float(*x); }

// a x + 3 * 2^22, which leaves the nearest integer to a x in the low bits of the word.
constexpr float kMagic = 12582912.f;
__device__ __forceinline__ int low(float x) { return __float_as_int(x) - 0x4b400000; }
// x in [0, 1] in units of 2^-45: the nearest multiple of 2^-22, and what that leaves.
__device__ __forceinline__ int64_t units(float x) {
  const float a = fmaf(x, 0x1p22f, kMagic);
  const float rest = fmaf(x, 0x1p22f, kMagic - a);
  return (int64_t)low(a) * (1 << 23) + low(fmaf(rest, 0x1p23f, kMagic));
}

// s as two fp32.
struct Times {
  float hi, lo;
};
// Weight of an element.
template <bool kDraft>
__device__ __forceinline__ uint64_t weight(float p, float q, const Times& s) {
  const int64_t a = units(clean(p));
  if (!kDraft) return (uint64_t)a;
  q = clean(q);
  const float t = s.hi * q;
  if (t >= 1.f) return 0;
  // what rounding the product and s took from it: below 2^-24
  const int64_t b = units(t) + low(fmaf(fmaf(s.lo, q, fmaf(s.hi, q, -t)), 0x1p45f, kMagic));
  return (uint64_t)max(a - b, (int64_t)0);
}

struct Shared {
  int q0, n, len;  // the sequence's rows; n is -1 where it is refused
  float p[kMaxNew], q[kMaxNew], u[kMaxNew];  // p and q of a node's token at its parent
  int token[kMaxNew], parent[kMaxNew], path[kMaxNew];
  int out[kMaxNew], outs;  // tokens rejected at the node (without q)
  uint64_t seg[kMaxSegs];  // sums of this CTA's segments
  uint64_t sum;
};
template <class V>
__device__ __forceinline__ void fetch(V& x, uint32_t rank) {  // what CTA `rank` has in x
  static_assert(sizeof(V) == 4, "a word");
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(map_cluster(smem_u32(&x), rank)) : "memory");
  *reinterpret_cast<uint32_t*>(&x) = v;
}

__device__ __forceinline__ uint64_t warp_sum(uint64_t x) {
#pragma unroll
  for (int off = 16; off; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
  return x;
}
__device__ __forceinline__ uint64_t load_cluster(const void* p, uint32_t rank) {
  uint64_t v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(map_cluster(smem_u32(p), rank)) : "memory");
  return v;
}

// kVec: rows in 16-byte vectors (their starts and strides are multiples of 16 bytes).
template <class T, bool kDraft, bool kVec>
__global__ void __launch_bounds__(kThreads, 2) verify_kernel(const __grid_constant__ Params p) {
  __shared__ Shared sm;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int b = blockIdx.x / p.ctas;
  const uint32_t rank = p.ctas > 1 ? cluster_ctarank() : 0;
  grid_dep_wait();
  grid_dep_launch();
  const T* rows_p = static_cast<const T*>(p.p);
  const T* rows_q = static_cast<const T*>(p.q);
  // The first CTA reads what the walk goes by, and the others take it from there: all of
  // them then come to the same barriers, whatever happens to the tensors meanwhile.
  if (rank == 0) {
    const bool falls = rows::offsets_fall(p.cu, p.B, threadIdx.x, kThreads);
    if (blockIdx.x == 0 && warp == 0) rows::check_offsets(p.cu, p.B, p.total, p.err);
    const bool none = __syncthreads_or(falls);
    if (threadIdx.x == 0) {
      const int q0 = p.cu[b], len = p.lens ? p.lens[b] : 0;
      const int64_t n = (int64_t)p.cu[b + 1] - q0;
      const bool fits = !none && (b == 0 ? q0 == 0 : q0 >= 0) && n >= 0 && n <= kMaxNew && q0 + n <= p.total &&
                        (!p.lens || len >= n);
      sm.q0 = q0, sm.n = fits ? (int)n : -1, sm.len = len;
    }
    __syncthreads();
  }
  if (rank == 0 && (int)threadIdx.x < sm.n) {
    const int q0 = sm.q0;
    const int i = threadIdx.x, tok = p.tokens[q0 + i];
    int parent = i - 1;
    if (p.mask) {
      const uint64_t below = (uint64_t)p.mask[q0 + i] & ((1ull << i) - 1);
      parent = 63 - __clzll((long long)below);  // none: -1
    }
    const bool in = tok >= 0 && tok < p.V;
    if (i > 0 && !in && rank == 0) atomicOr(p.err, rows::kBadIndex);
    sm.token[i] = in ? tok : -1;  // never accepted
    sm.parent[i] = parent;
    sm.u[i] = p.u[q0 + i];
    const bool real = in && parent >= 0;
    sm.p[i] = real ? clean(load(rows_p + (q0 + parent) * p.p_stride + tok)) : 0.f;
    if (kDraft) sm.q[i] = real ? clean(load(rows_q + (q0 + parent) * p.q_stride + tok)) : 0.f;
  }
  if (p.ctas > 1) {
    cluster_sync();
    if (rank > 0) {
      if (threadIdx.x < kMaxNew) {
        const int i = threadIdx.x;
        fetch(sm.p[i], 0), fetch(sm.u[i], 0), fetch(sm.token[i], 0), fetch(sm.parent[i], 0);
        if (kDraft) fetch(sm.q[i], 0);
      } else if (threadIdx.x == kMaxNew) {
        fetch(sm.q0, 0), fetch(sm.n, 0);
      }
    }
  }
  if (threadIdx.x == 0) sm.outs = 0, sm.path[0] = 0;
  __syncthreads();
  const int q0 = sm.q0, n = sm.n;
  if (n <= 0) {
    if (rank == 0 && threadIdx.x == 0) {
      if (n < 0) atomicOr(p.err, rows::kBadSeqlens);
      p.kept[b] = 0;
      p.next[b] = -1;
      if (p.lens_out) p.lens_out[b] = sm.len;
    }
    if (p.ctas > 1) cluster_sync();  // the first CTA's memory has been read
    return;
  }

  // The sum of the weights left at node `at`, in units of 2^-45; this CTA's share of the
  // row is segments seg0 .. seg1 - 1.
  const int segs = (p.V + kSeg - 1) / kSeg, each = (segs + p.ctas - 1) / p.ctas;
  const int seg0 = min((int)rank * each, segs), seg1 = min(seg0 + each, segs);
  uint64_t before = 0, mine = 0;
  auto gone = [&](int token) {  // whether it was rejected at the node (without q)
    bool is = false;
    for (int k = 0; k < sm.outs; ++k) is |= sm.out[k] == token;
    return is;
  };
  auto pass = [&](int at, double times, bool removed) {
    const T* row_p = rows_p + (q0 + at) * p.p_stride;
    const T* row_q = kDraft ? rows_q + (q0 + at) * p.q_stride : nullptr;
    Times s;
    s.hi = (float)times;
    s.lo = (float)(times - s.hi);
    const bool both = kDraft && times != 0.0;
    constexpr int kPer = 16 / sizeof(T), kSteps = kSeg / (32 * kPer);
    if (threadIdx.x == 0) sm.sum = 0;
    __syncthreads();
    for (int seg = seg0 + warp; seg < seg1; seg += kWarps) {
      uint64_t sum = 0;
      const int from = seg * kSeg;
      if (kVec && from + kSeg <= p.V) {
        uint4 xp[kSteps], xq[kSteps];
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          xp[k] = *reinterpret_cast<const uint4*>(row_p + from + (32 * k + lane) * kPer);
          if (both) xq[k] = *reinterpret_cast<const uint4*>(row_q + from + (32 * k + lane) * kPer);
        }
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          const T* ep = reinterpret_cast<const T*>(&xp[k]);
          const T* eq = reinterpret_cast<const T*>(&xq[k]);
#pragma unroll
          for (int e = 0; e < kPer; ++e)
            sum += both ? weight<true>(load(ep + e), load(eq + e), s) : weight<false>(load(ep + e), 0.f, s);
        }
      } else {
#pragma unroll 8
        for (int x = from + lane; x < min(from + kSeg, p.V); x += 32)
          sum += both ? weight<true>(load(row_p + x), load(row_q + x), s) : weight<false>(load(row_p + x), 0.f, s);
      }
      sum = warp_sum(sum);
      if (removed)
        for (int k = 0; k < sm.outs; ++k)
          if (sm.out[k] / kSeg == seg) sum -= weight<false>(load(row_p + sm.out[k]), 0.f, s);
      if (lane == 0) {
        sm.seg[seg - seg0] = sum;
        atomicAdd(reinterpret_cast<unsigned long long*>(&sm.sum), (unsigned long long)sum);
      }
    }
    uint64_t total = 0;
    if (p.ctas > 1) {
      cluster_sync();
      before = 0;
      for (int c = 0; c < p.ctas; ++c) {
        const uint64_t v = load_cluster(&sm.sum, c);
        total += v;
        if (c < (int)rank) before += v;
        if (c == (int)rank) mine = v;
      }
      cluster_sync();  // the sums may change again
    } else {
      __syncthreads();
      before = 0, total = mine = sm.sum;
      __syncthreads();
    }
    return total;
  };

  // The walk; every thread of the cluster takes it, over the same data.
  int cur = 0, kept = 1;
  double s = 0.0, z = 1.0;
  bool stale = false;  // z is that of the rejection before
  for (int i = 1; i < n; ++i) {
    if (sm.parent[i] != cur) continue;
    if (stale) z = (double)pass(cur, s, false) * 0x1p-45, stale = false;
    const double left = kDraft ? fmax((double)sm.p[i] - s * (double)sm.q[i], 0.0)
                               : gone(sm.token[i]) ? 0.0 : (double)sm.p[i];
    const double test = (double)sm.u[i] * z * (kDraft ? (double)sm.q[i] : 1.0);
    if (sm.token[i] >= 0 && test < left) {
      if (threadIdx.x == 0) sm.path[kept] = i;
      cur = i, ++kept;
      s = 0.0, z = 1.0;
      if (!kDraft) {
        __syncthreads();
        if (threadIdx.x == 0) sm.outs = 0;
        __syncthreads();
      }
    } else if (kDraft) {
      s += z;
      stale = true;
    } else {
      z -= left;
      if (left > 0.0) {  // a token once
        __syncthreads();
        if (threadIdx.x == 0) sm.out[sm.outs++] = sm.token[i];
        __syncthreads();
      }
    }
  }

  // The next token.
  uint64_t total = pass(cur, s, !kDraft);
  bool removed = !kDraft;
  if (total == 0 && (kDraft ? s != 0.0 : sm.outs > 0)) {  // nothing is left: the target's own row
    s = 0.0, removed = false;
    total = pass(cur, s, false);
  }
  const double draw = fmax((double)p.u_next[b], 0.0) * (double)total;  // NaN: 0
  uint64_t want = draw < (double)total ? (uint64_t)draw : total - 1;
  if (want >= total) want = total - 1;
  if (total == 0) {
    if (rank == 0 && threadIdx.x == 0) p.next[b] = -1;
  } else if (warp == 0 && want >= before && want - before < mine) {  // it lies in this CTA's part
    want -= before;
    int seg = seg0;
    for (int base = 0; base < seg1 - seg0; base += 32) {  // the segment
      uint64_t upto = base + lane < seg1 - seg0 ? sm.seg[base + lane] : 0;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const uint64_t v = __shfl_up_sync(0xffffffffu, upto, off);
        if (lane >= off) upto += v;
      }
      const uint32_t over = __ballot_sync(0xffffffffu, upto > want);
      if (over) {
        const int k = __ffs(over) - 1;
        const uint64_t front = __shfl_sync(0xffffffffu, upto, k > 0 ? k - 1 : 0);
        if (k > 0) want -= front;
        seg = seg0 + base + k;
        break;
      }
      want -= __shfl_sync(0xffffffffu, upto, 31);
    }
    const T* row_p = rows_p + (q0 + cur) * p.p_stride;
    const T* row_q = kDraft ? rows_q + (q0 + cur) * p.q_stride : nullptr;
    Times sf;
    sf.hi = (float)s;
    sf.lo = (float)(s - sf.hi);
    for (int base = seg * kSeg;; base += 32) {  // its element
      const int x = base + lane;
      uint64_t upto = 0;
      if (x < p.V) {
        upto = kDraft && s != 0.0 ? weight<true>(load(row_p + x), load(row_q + x), sf) : weight<false>(load(row_p + x), 0.f, sf);
        if (removed && gone(x)) upto = 0;
      }
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const uint64_t v = __shfl_up_sync(0xffffffffu, upto, off);
        if (lane >= off) upto += v;
      }
      const uint32_t over = __ballot_sync(0xffffffffu, upto > want);
      if (over || base + 32 >= p.V) {
        if (lane == 0) p.next[b] = over ? base + __ffs(over) - 1 : p.V - 1;
        break;
      }
      want -= __shfl_sync(0xffffffffu, upto, 31);
    }
  }
  if (rank == 0) {
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kThreads) p.path[q0 + i] = i < kept ? sm.path[i] : -1;
    if (threadIdx.x == 0) {
      p.kept[b] = kept;
      if (p.lens_out) p.lens_out[b] = sm.len - n + kept;
    }
  }
}

}  // namespace verify
}  // namespace attn
