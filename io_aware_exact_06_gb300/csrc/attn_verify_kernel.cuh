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
// its CTAs, which read the last node's rows once.  A few dependent loads and barriers bound
// a small batch (8 chains of 5, 50021 tokens: 8.6 us); a large one is bounded by those of its
// sequences that need several passes, one behind the other, 6 us each (64 trees of up to 16,
// 131072 tokens in fp32: 41 us, of which HBM needs 10; most end after 16 to 22).
//
// The tests are in fp64.  Sums are exact: a weight is an integer, p - s q in units of
// 2^-43 (up to 2^18 of them fit 64 bits), s q taken in two fp32 parts, so C does not depend
// on how a row is cut, and a draw next to a border falls where it does in fp64.  (A weight is
// off by 2^-44, and by 2^-46 from fp32 below the multiples of 2^-22.)
#pragma once

#include <cstring>

#include "attn_rows.cuh"

namespace attn {
namespace verify {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxNew = 64;
constexpr int kMaxV = 1 << 18;
constexpr int kSeg = 1024;  // elements that a warp sums at a time
constexpr int kMaxSegs = kMaxV / kSeg + 1;
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

__device__ __forceinline__ float load(const float* x) { return *x; }
__device__ __forceinline__ float load(const __nv_bfloat16* x) { return __bfloat162float(*x); }
__device__ __forceinline__ float clean(float x) { return __saturatef(x); }  // to [0, 1]; NaN: 0

// a x + 3 * 2^22, which leaves the nearest integer to a x in the low bits of the word.
constexpr float kMagic = 12582912.f;
constexpr int kMagicBits = 0x4b400000;
// x in [0, 1] as hi + rest in units of 2^-22, hi whole (in `a`, as above), rest at most a half.
__device__ __forceinline__ float split(float x, float& a, float& hi) {
  a = fmaf(x, 0x1p22f, kMagic);
  hi = a - kMagic;
  return fmaf(x, 0x1p22f, -hi);
}

// Weights of a lane's elements so far: hi in units of 2^-22, lo of 2^-43.  For up to 32
// elements both are 32-bit numbers.
struct Sum {
  int hi = 0, lo = 0;
  __device__ __forceinline__ uint64_t units() const { return (uint64_t)((int64_t)hi * (1 << 21) + lo); }
};

// s as two fp32.
struct Times {
  float hi, lo;
};
// How a row is weighed: p itself, p - q, p - s q.
enum : int { kAlone = 0, kOnce = 1, kScaled = 2 };
template <int kHow>
__device__ __forceinline__ void weigh(float p, float q, const Times& s, Sum& sum) {
  float pa, ph;
  const float pr = split(clean(p), pa, ph);
  if (kHow == kAlone) {
    sum.hi += __float_as_int(pa) - kMagicBits;
    sum.lo += __float_as_int(fmaf(pr, 0x1p21f, kMagic)) - kMagicBits;
    return;
  }
  q = clean(q);
  // s q as t and what rounding the product and s took from it (where s q is above 1 that
  // is more than p: the weight is 0)
  const float t = kHow == kOnce ? q : fminf(s.hi * q, 1.f);
  float ta, th;
  float rest = pr - split(t, ta, th);
  if (kHow == kScaled) rest = fmaf(fmaf(s.lo, q, fmaf(s.hi, q, -t)), -0x1p22f, rest);
  if (ph - th + rest > 0.f) {
    sum.hi += __float_as_int(pa) - __float_as_int(ta);
    sum.lo += __float_as_int(fmaf(rest, 0x1p21f, kMagic)) - kMagicBits;  // rest is below 2
  }
}

// Two elements at once, as pairs of fp32 in 64 bits, between 0 and 1.
using Pair = unsigned long long;
__device__ __forceinline__ Pair pair(float a, float b) {
  Pair r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
  Pair r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ Pair sub2(Pair a, Pair b) { return fma2(b, pair(-1.f, -1.f), a); }
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
  Pair r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ int first_of(Pair x) { return (int)(uint32_t)x; }
__device__ __forceinline__ int second_of(Pair x) { return (int)(uint32_t)(x >> 32); }

template <int kHow>
__device__ __forceinline__ void weigh2(Pair p, Pair q, const Times& s, Sum& sum) {
  const Pair up = pair(0x1p22f, 0x1p22f), down = pair(0x1p21f, 0x1p21f), magic = pair(kMagic, kMagic);
  const Pair pa = fma2(p, up, magic), minus_ph = sub2(magic, pa);
  Pair rest = fma2(p, up, minus_ph);
  if (kHow == kAlone) {
    const Pair lo = fma2(rest, down, magic);
    sum.hi += (int)((uint32_t)first_of(pa) + (uint32_t)second_of(pa) - 2u * kMagicBits);
    sum.lo += (int)((uint32_t)first_of(lo) + (uint32_t)second_of(lo) - 2u * kMagicBits);
    return;
  }
  Pair t = q;
  if (kHow == kScaled) {
    const Pair x = mul2(pair(s.hi, s.hi), q);
    t = pair(fminf(__int_as_float(first_of(x)), 1.f), fminf(__int_as_float(second_of(x)), 1.f));
  }
  const Pair ta = fma2(t, up, magic), minus_th = sub2(magic, ta);
  rest = sub2(rest, fma2(t, up, minus_th));
  if (kHow == kScaled) {
    const Pair e = fma2(pair(s.lo, s.lo), q, fma2(pair(s.hi, s.hi), q, mul2(t, pair(-1.f, -1.f))));
    rest = fma2(e, pair(-0x1p22f, -0x1p22f), rest);
  }
  const Pair all = fma2(sub2(minus_th, minus_ph), pair(1.f, 1.f), rest), lo = fma2(rest, down, magic);
  if (__int_as_float(first_of(all)) > 0.f) {
    sum.hi += first_of(pa) - first_of(ta);
    sum.lo += first_of(lo) - kMagicBits;
  }
  if (__int_as_float(second_of(all)) > 0.f) {
    sum.hi += second_of(pa) - second_of(ta);
    sum.lo += second_of(lo) - kMagicBits;
  }
}

struct Shared {
  int q0, n, len;  // the sequence's rows; n is -1 where it is refused
  float p[kMaxNew], q[kMaxNew], u[kMaxNew];  // p and q of a node's token at its parent
  int token[kMaxNew], parent[kMaxNew], path[kMaxNew];
  int out[kMaxNew], outs;  // tokens rejected at the node (without q)
  int cur, kept, at;       // the walk: its node, how many tokens it has, the token it has come to
  double s, z;
  Times times;             // s
  uint64_t seg[kMaxSegs];  // sums of this CTA's segments
  uint64_t sum[2];         // theirs, of passes by turns
};
template <int kValue>
struct Int {
  static constexpr int value = kValue;
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

template <class T, bool kDraft>
__global__ void __launch_bounds__(kThreads, 4) verify_kernel(const __grid_constant__ Params p) {
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
  if (threadIdx.x == 0) sm.outs = sm.cur = sm.path[0] = 0, sm.kept = 1, sm.s = 0.0, sm.z = 1.0, sm.times = {0.f, 0.f};
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

  constexpr int kPer = 16 / sizeof(T);  // elements of a 16-byte vector
  uint64_t before = 0, mine = 0;        // of the cluster's sum: in front of this CTA's part, and that
  auto gone = [&](int token) {          // whether it was rejected at the node (without q)
    bool is = false;
    for (int k = 0; k < sm.outs; ++k) is |= sm.out[k] == token;
    return is;
  };
  // A node's rows and s.  Vectors lie on multiples of 16 bytes, `shift` elements of the
  // first in front of the row; where p and q lie differently elements are loaded singly.
  struct Row {
    const T *p, *q;
    int shift;
    bool together;
    Times s;
    int how;
  };
  auto row_of = [&](bool alone) {  // of the walk's node; alone: p itself
    Row r;
    r.p = rows_p + (q0 + sm.cur) * p.p_stride;
    r.q = kDraft ? rows_q + (q0 + sm.cur) * p.q_stride : r.p;
    const uint64_t a = reinterpret_cast<uint64_t>(r.p), b = reinterpret_cast<uint64_t>(r.q);
    r.shift = (int)(a % 16 / sizeof(T));
    r.s = sm.times;
    r.how = !kDraft || alone || r.s.hi == 0.f ? kAlone : r.s.hi == 1.f && r.s.lo == 0.f ? kOnce : kScaled;
    r.together = r.how == kAlone || (a - b) % 16 == 0;
    return r;
  };
  // Vector v of a row, element by element: those outside the row are 0.
  auto singly = [&](const T* row, int v, int shift) {
    T e[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int x = v * kPer - shift + k;
      e[k] = T(0.f);
      if (x >= 0 && x < p.V) e[k] = row[x];
    }
    uint4 x;
    memcpy(&x, e, 16);
    return x;
  };
  auto inside = [&](const Row& r, int v) {  // both rows' vectors lie on 16 bytes, and inside
    return r.together && v * kPer >= r.shift && (v + 1) * kPer - r.shift <= p.V;
  };
  // The weights of a vector's elements, two by two.
  auto weigh_vector = [&](const Row& r, const uint4& xp, const uint4& xq, auto how, Sum& sum) {
    constexpr int kHow = decltype(how)::value;
    const uint32_t up[4] = {xp.x, xp.y, xp.z, xp.w}, uq[4] = {xq.x, xq.y, xq.z, xq.w};
    auto two = [&](const uint32_t (&u)[4], int k) {
      const uint32_t lo = kPer == 4 ? u[2 * k % 4] : u[k] << 16, hi = kPer == 4 ? u[(2 * k + 1) % 4] : u[k] & 0xffff0000u;
      return pair(clean(__uint_as_float(lo)), clean(__uint_as_float(hi)));
    };
#pragma unroll
    for (int k = 0; k < kPer / 2; ++k) weigh2<kHow>(two(up, k), kHow ? two(uq, k) : 0, r.s, sum);
  };
  auto with_how = [&](const Row& r, auto f) {
    if (r.how == kAlone) f(Int<kAlone>());
    else if (r.how == kOnce) f(Int<kOnce>());
    else f(Int<kScaled>());
  };
  // The sum of the weights left at a node, in units of 2^-43; this CTA's share of the row
  // is segments seg0 .. seg1 - 1.
  int seg0 = 0, seg1 = 0, passes = 0;
  auto pass = [&](const Row& r, bool removed) {
    const int segs = (p.V + r.shift + kSeg - 1) / kSeg, each = (segs + p.ctas - 1) / p.ctas;
    seg0 = min((int)rank * each, segs), seg1 = min(seg0 + each, segs);
    uint64_t* const at = &sm.sum[passes++ & 1];  // read by others until they come to the next pass's barrier
    if (threadIdx.x == 0) *at = 0;
    __syncthreads();
    constexpr int kSteps = kSeg / 32 / kPer;  // vectors of a lane in a segment
    for (int seg = seg0 + warp; seg < seg1; seg += kWarps) {
      Sum part;
      const int v0 = seg * (kSeg / kPer);
      const bool whole = r.together && v0 * kPer >= r.shift && (seg + 1) * kSeg - r.shift <= p.V;
      with_how(r, [&](auto how) {
        constexpr int kHow = decltype(how)::value;
        if (whole) {
          const uint4* ap = reinterpret_cast<const uint4*>(r.p - r.shift) + v0 + lane;
          const uint4* aq = reinterpret_cast<const uint4*>(r.q - r.shift) + v0 + lane;
#pragma unroll
          for (int k = 0; k < kSteps; k += 4) {
            uint4 xp[4], xq[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              xp[u] = ap[32 * (k + u)];
              if (kHow) xq[u] = aq[32 * (k + u)];
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) weigh_vector(r, xp[u], xq[u], how, part);
          }
        } else {
#pragma unroll 1
          for (int k = 0; k < kSteps; ++k) {
            const uint4 xp = singly(r.p, v0 + 32 * k + lane, r.shift);
            const uint4 xq = kHow ? singly(r.q, v0 + 32 * k + lane, r.shift) : xp;
            weigh_vector(r, xp, xq, how, part);
          }
        }
      });
      uint64_t sum = warp_sum(part.units());
      if (removed)
        for (int k = 0; k < sm.outs; ++k)
          if ((sm.out[k] + r.shift) / kSeg == seg) {
            Sum out;
            weigh<kAlone>(load(r.p + sm.out[k]), 0.f, r.s, out);
            sum -= out.units();
          }
      if (lane == 0) {
        sm.seg[seg - seg0] = sum;
        atomicAdd(reinterpret_cast<unsigned long long*>(at), (unsigned long long)sum);
      }
    }
    if (p.ctas == 1) {
      __syncthreads();
      return before = 0, mine = *at;
    }
    cluster_sync();
    const uint64_t there = lane < p.ctas ? load_cluster(at, lane) : 0;
    before = warp_sum(lane < (int)rank ? there : 0);
    mine = __shfl_sync(0xffffffffu, there, rank);
    return warp_sum(there);
  };

  // The walk.  One warp of each CTA takes it, over the same data in all, up to where it
  // needs a sum over a row.  A test is made in fp32, and in fp64 where that could go either
  // way: the SM has few units for it (all tests in fp64, by every warp: 4 us and more).
  for (int i = 1;;) {
    if (warp == 0) {
      int cur = sm.cur, kept = sm.kept;
      double s = sm.s, z = sm.z;
      Times sf = sm.times;
      float zf = (float)z;
      bool stale = false;  // z is that of the rejection before
      for (; i < n; ++i) {
        if (sm.parent[i] != cur) continue;
        if (stale) break;
        const float pi = sm.p[i], qi = kDraft ? sm.q[i] : 1.f, ui = sm.u[i];
        const bool never = sm.token[i] < 0 || (!kDraft && gone(sm.token[i]));
        const float left = kDraft ? fmaf(-sf.hi, qi, pi) : pi, test = ui * qi * zf;
        // three roundings of test, two of left, and s.lo: below 2^-21 of what they are made of
        const float unsure = 0x1p-20f * (fabsf(test) + pi + sf.hi * qi);
        bool yes = test < fmaxf(left, 0.f);
        if (!(fabsf(test - left) > unsure))
          yes = (double)ui * qi * z < (kDraft ? fmax((double)pi - s * qi, 0.0) : (double)pi);
        if (yes && !never) {
          cur = i;
          s = 0.0, z = 1.0, sf.hi = sf.lo = 0.f, zf = 1.f;
          __syncwarp();
          if (lane == 0) sm.path[kept] = i, sm.outs = 0;
          ++kept;
        } else if (kDraft) {
          s += z;
          sf.hi = (float)s, sf.lo = (float)(s - sf.hi);
          stale = true;
        } else if (!never) {
          z -= pi;
          zf = (float)z;
          __syncwarp();
          if (lane == 0) sm.out[sm.outs++] = sm.token[i];  // a token once
        }
        __syncwarp();
      }
      if (lane == 0) sm.cur = cur, sm.kept = kept, sm.s = s, sm.z = z, sm.times = sf, sm.at = i;
    }
    __syncthreads();
    i = sm.at;
    if (i >= n) break;
    const uint64_t sum = pass(row_of(false), false);
    if (threadIdx.x == 0) sm.z = (double)sum * 0x1p-43;
    __syncthreads();
  }
  const int kept = sm.kept;

  // The next token.
  Row r = row_of(false);
  bool removed = !kDraft;
  uint64_t total = pass(r, removed);
  if (total == 0 && (kDraft ? r.how != kAlone : sm.outs > 0)) {  // nothing is left: the target's own row
    r = row_of(true), removed = false;
    total = pass(r, false);
  }
  uint64_t want = 0;
  if (warp == 0) {
    const double draw = fmax((double)p.u_next[b], 0.0) * (double)total;  // NaN: 0
    want = draw < (double)total ? (uint64_t)draw : total - 1;
    if (want >= total) want = total - 1;
  }
  if (total == 0) {
    if (rank == 0 && threadIdx.x == 0) p.next[b] = -1;
  } else if (warp == 0 && want >= before && want - before < mine) {  // it lies in this CTA's part
    want -= before;
    // Where running sums of the lanes' counts pass `want`: that lane; want is less what
    // is in front of it.
    auto pick = [&](uint64_t count) {
      uint64_t upto = count;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const uint64_t v = __shfl_up_sync(0xffffffffu, upto, off);
        if (lane >= off) upto += v;
      }
      const uint32_t over = __ballot_sync(0xffffffffu, upto > want);
      const int k = over ? __ffs(over) - 1 : 32;
      const uint64_t front = __shfl_sync(0xffffffffu, upto, k > 0 ? k - 1 : 0);
      if (k > 0) want -= front;
      return k;
    };
    int seg = seg0;
    for (int base = 0; base < seg1 - seg0; base += 32) {
      const int k = pick(base + lane < seg1 - seg0 ? sm.seg[base + lane] : 0);
      seg = seg0 + base + k;
      if (k < 32) break;
    }
    // 32 elements to a lane, then one
    const auto removed_at = [&](int x) {
      Sum out;
      if (removed && gone(x)) weigh<kAlone>(load(r.p + x), 0.f, r.s, out);
      return out.units();
    };
    Sum part;
    with_how(r, [&](auto how) {
#pragma unroll 2
      for (int k = 0; k < 32 / kPer; ++k) {
        const int v = seg * (kSeg / kPer) + lane * (32 / kPer) + k;
        uint4 xp, xq = make_uint4(0, 0, 0, 0);
        if (inside(r, v)) {
          xp = *reinterpret_cast<const uint4*>(r.p + v * kPer - r.shift);
          if (decltype(how)::value) xq = *reinterpret_cast<const uint4*>(r.q + v * kPer - r.shift);
        } else {
          xp = singly(r.p, v, r.shift);
          if (decltype(how)::value) xq = singly(r.q, v, r.shift);
        }
        weigh_vector(r, xp, xq, how, part);
      }
    });
    uint64_t count = part.units();
    const int from = seg * kSeg - r.shift;
    if (removed)
      for (int k = 0; k < sm.outs; ++k)
        if ((sm.out[k] - from) >> 5 == lane && sm.out[k] >= from) count -= removed_at(sm.out[k]);
    const int run = min(pick(count), 31);
    const int x = from + 32 * run + lane;
    Sum one;
    if (x >= 0 && x < p.V)
      with_how(r, [&](auto how) { weigh<decltype(how)::value>(load(r.p + x), kDraft ? load(r.q + x) : 0.f, r.s, one); });
    const int k = min(pick(one.units() - (x >= 0 && x < p.V ? removed_at(x) : 0)), 31);
    if (lane == 0) p.next[b] = min(max(from + 32 * run + k, 0), p.V - 1);
  }
  if (rank == 0) {
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kThreads) p.path[q0 + i] = i < kept ? sm.path[i] : -1;
    if (threadIdx.x == 0) {
      p.kept[b] = kept;
      if (p.lens_out) p.lens_out[b] = sm.len - n + kept;
    }
  }
  if (p.ctas > 1) cluster_sync();  // its sum has been read
}

}  // namespace verify
}  // namespace attn
