// The line of groups over a bf16 cache, many query rows: S = Q K^T and O += P V on
// tcgen05 over keys that every row sees.
//
// Nothing is masked but what a last tile has behind the prefix, and no value is hidden
// from a row, so the roles of attn_tree_tile_kernel.cuh that clean and convert are not
// there, and a softmax thread keeps its row's 128 scores in registers, as in the dense
// forward: one read of a score from tensor memory, one write of its probability.
//
// Warps: 0-3 and 4-7 softmax groups A and B (a thread owns a row), which also bring
// their query tile into shared memory and write the piece's end; 8 copies keys and values;
// 9 issues the products.  kPair, for more than 128 rows: A and B take two row tiles over
// the same key tiles.  Else: A takes the even key tiles of a piece, B the odd ones, and
// they meet at its end.
//
// A segment is `team` row tiles (pairs of them), and as many CTAs beside each other take
// one of them each over the same share of the keys, which so come from HBM once: a pair of
// tiles has 64 KB of them for 1.1 us of products.
//
// kTwo: a probability is the sum of two bf16, its rounding and what that leaves, each with
// its product with V, as in attn_tree_few_kernel.cuh; a tile of scores has room for both.  One
// bf16 in its place, and O divided by the sum with the largest of them as rounded, is what
// attn_tree_tile_kernel.cuh does for the rows that it has over their own keys.  (64 samples of
// 16384 keys, one token each: 67.2 us so, 69.9 with two.)
//
// The chain of a row tile bounds it: S, softmax, P V, and back to S.  With one bf16 a pair of
// tiles takes 3140 cycles over 128 keys, d = 128, with 2048 of products; 1812 rows over 32768 keys of 8
// heads 213 us on 136 SMs, 0.64 of their tensor pipe.
#pragma once

#include "attn_tree_tile_kernel.cuh"

namespace attn {
namespace tree {

constexpr int kRowsThreads = 384;
// Registers after setmaxnreg: 256 threads of softmax, 128 of the rest; 384 x 168 in all.
constexpr int kRowsSoftmaxRegs = 184, kRowsRestRegs = 120;
constexpr int kFlags = 16;  // segments whose flags are kept: the copies run at most five ahead
constexpr float kRowsLazy = 16.f;  // growth (log2) of a row maximum that is worth a rescale

struct RowsShared {
  uint64_t bars[32];
  uint32_t tmem;
  int abort;
  int bad[kFlags];  // the segment reads a page outside the cache
  // where the groups meet
  float2 ml[2][kBigRows];  // [group]: maxima of raw scores, sums
  float fix[2][kBigRows];  // what rounding the largest probabilities adds to the sum
};

template <int D, bool kPair>
struct RowsCfg {
  static constexpr int kMat = kBigTile * D * 2;  // a tile of keys or values, and of queries
  static constexpr int kChunk = kBigTile * 128;  // 128 rows of 128 bytes
  static constexpr int kQ = (kPair ? 2 : 1) * kMat;
  static constexpr int kRows = (kPair ? 2 : 1) * kBigRows;
  static constexpr int kStages = D == 64 ? 8 : 4;  // tiles on their way, keys and values by turns
  static constexpr int kTurn = 8 * 32 * 128;                   // 32 rows of 32 columns for each softmax warp
  static constexpr int kOffRing = kQ;
  static constexpr int kOffTurn = kOffRing + kStages * kMat;
  static constexpr int kOffShared = kOffTurn + kTurn;
  static constexpr int kSmem = kOffShared + (kPair ? (int)offsetof(RowsShared, ml) : (int)sizeof(RowsShared));
  static constexpr int bFull = 0, bEmpty = bFull + kStages, bSF = bEmpty + kStages, bPF = bSF + 2, bOF = bPF + 2,
                       bQF = bOF + 2, bDrain = bQF + 2, kBars = bDrain + 1;
};

// What rounding a and b to the bf16 in `as` leaves of them, as bf16.
__device__ __forceinline__ uint32_t rest_of(float a, float b, uint32_t as) {
  return rows::pack2(a - __uint_as_float(as << 16), b - __uint_as_float(as & 0xffff0000u));
}

// Rows `step` apart as tokens and heads of a group of G.
struct Rows {
  int row, tok, g, step, dtok, dg, G;
  __device__ __forceinline__ Rows(int G_, int first, int step_) : row(first), step(step_), G(G_) {
    tok = row / G, g = row - tok * G;
    dtok = step / G, dg = step - dtok * G;
  }
  __device__ __forceinline__ void next() {
    row += step, tok += dtok, g += dg;
    if (g >= G) g -= G, ++tok;
  }
};

template <int D, bool kPair, bool kTwo>
struct RowsRole {
  using C = RowsCfg<D, kPair>;
  const Params& p;
  const Work& w;
  RowsShared& ss;
  uint8_t* smem_ptr;
  uint32_t smem, tmem;

  __device__ __forceinline__ uint32_t bar(int i) const { return smem_u32(&ss.bars[i]); }
  // Bounded, as in Big: once one wait has run out no thread waits twice more, every role
  // goes through its loops to the end, and the rows come out as NaN.
  mutable bool dead = false;
  __device__ __forceinline__ void wait(int i, uint32_t parity) const {
    if (dead || mbar_try_wait(bar(i), parity)) return;
    if (aborted()) {
      dead = true;
    } else if (!mbar_wait(bar(i), parity, kWaitNs)) {
      dead = true;
      *(volatile int*)&ss.abort = 1;
      atomicOr(p.err, kTimedOut);
    }
  }
  __device__ __forceinline__ bool aborted() const { return *(volatile int*)&ss.abort != 0; }
  __device__ __forceinline__ int head(const Walk<true>& k) const { return k.seg / (k.segs / p.H); }
  // this CTA's row of the segment, and whether there is one
  __device__ __forceinline__ int row0(const Walk<true>& k) const {
    return k.seg % (k.segs / p.H) * w.rows + (int)blockIdx.x % (w.rows / C::kRows) * C::kRows;
  }
  __device__ __forceinline__ bool busy(const Walk<true>& k) const { return row0(k) < k.s.n * p.G; }
  // to the next piece with rows
  __device__ __forceinline__ bool next(Walk<true>& k) const {
    while (k.next(p, w))
      if (busy(k)) return true;
    return false;
  }

  // -------------------------------------------------------------- producer --
  // Boxes behind the prefix, and those of a page outside the cache, are copied from behind
  // the tensor: TMA fills them with zeros.
  __device__ __forceinline__ void produce(Walk<true> k, const CUtensorMap* map_k, const CUtensorMap* map_v) {
    const int lane = threadIdx.x % 32;
    const int page = 1 << p.log_page, none = p.pages << p.log_page;
    const int box = min(page, kBigTile), per = kBigTile / box;  // rows of a copy, copies of a tile
    const int batch = 32 / per;                                 // tiles whose page numbers one load fetches
    int s = 0, round = 0, seg = 0;
    do {
      const int h = head(k), len = k.s.len, end = k.tile + k.piece();
      const int* table = p.table + k.s.table(p, k.b);
      auto fetch = [&](int tile) {
        const int64_t pos = (int64_t)tile * kBigTile + lane * box;
        return pos < len ? table[pos >> p.log_page] : -1;
      };
      int ids = fetch(k.tile);
      for (int t0 = k.tile; t0 < end; t0 += batch) {
        const int next = t0 + batch < end ? fetch(t0 + batch) : -1;
        const bool wrong = (unsigned)ids >= (unsigned)p.pages;
        const uint32_t wrongs = __ballot_sync(0xffffffffu, wrong && (int64_t)t0 * kBigTile + lane * box < len);
        if (wrong) ids = -1;
        for (int t = t0; t < min(t0 + batch, end); ++t) {
          const int key0 = t * kBigTile;
          const int id = __shfl_sync(0xffffffffu, ids, (t - t0) * per + lane % per);
          const int row = id < 0 ? none : (id << p.log_page) + ((key0 + lane % per * box) & (page - 1));
#pragma unroll 1
          for (int m = 0; m < 2; ++m) {
            if (round > 0) wait(C::bEmpty + s, (round & 1) ^ 1);
            __syncwarp();
            if (!__any_sync(0xffffffffu, dead)) {
              const uint32_t full = bar(C::bFull + s);
              if (lane == 0) {
                if (m == 0 && (wrongs >> ((t - t0) * per) & ((1u << per) - 1))) {
                  ss.bad[seg % kFlags] = 1;
                  atomicOr(p.err, rows::kBadIndex);
                }
                mbar_arrive_expect_tx(full, C::kMat);
              }
              __syncwarp();
              if (lane < per) {
                const uint32_t dst = smem + C::kOffRing + s * C::kMat + lane * box * 128;
#pragma unroll
                for (int f = 0; f < D / 64; ++f) tma_load_3d(dst + f * C::kChunk, m ? map_v : map_k, full, f * 64, h, row);
              }
            }
            if (++s == C::kStages) s = 0, ++round;
          }
        }
        ids = next;
      }
      ++seg;
    } while (next(k));
  }

  // -------------------------------------------------------------- products --
  __device__ __forceinline__ void scores(uint32_t tmem, uint32_t smem, int g, int slot) {
    const uint32_t d = tmem + 128 * g;
    const uint64_t a = make_sdesc(smem + (kPair ? g * C::kMat : 0), 16, 1024, kSwizzle128B);
    const uint64_t b = make_sdesc(smem + C::kOffRing + slot * C::kMat, 16, 1024, kSwizzle128B);
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      const uint64_t off = (uint64_t)(((kk / 4) * C::kChunk + (kk % 4) * 32) >> 4);
      mma_ss(d, a + off, b + off, make_idesc_bf16(128, 128, false), kk > 0);
    }
  }
  __device__ __forceinline__ void values(uint32_t tmem, uint32_t smem, int g, int slot, bool accumulate) {
    const uint64_t b = make_sdesc(smem + C::kOffRing + slot * C::kMat, C::kChunk, 1024, kSwizzle128B);
#pragma unroll
    for (int part = 0; part < (kTwo ? 2 : 1); ++part)
#pragma unroll
      for (int kk = 0; kk < kBigTile / 16; ++kk)
        mma_ts(tmem + 256 + D * g, tmem + 128 * g + 64 * part + 8 * kk, b + (uint64_t)((kk * 2048) >> 4),
               make_idesc_bf16(128, D, true), part > 0 || kk > 0 || accumulate);
  }
  // One thread issues every product, in the order of the steps (a step is a key tile, or
  // with kPair a key tile of one row tile): S(0), S(1), then for each step j its P V and
  // S(j + 2).  The warp's lanes look at a step's barriers side by side, and what descriptors
  // are made of is the same in every lane for the compiler to see, so that they are made in
  // uniform registers: this thread is what the others wait for (a pair of tiles of 2048
  // cycles of products took it 4100 with lane 0 alone).
  __device__ __forceinline__ void multiply(Walk<true> k) {
    const int lane = threadIdx.x % 32;
    auto uniform = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
    const uint32_t tm = uniform(tmem), base = uniform(smem);
    int kslot = 0, kround = 0, vslot = 1, vround = 0;  // keys and values take slots by turns
    uint32_t pcount = 0;                               // parity of the groups' next probabilities
    int seg = 0;
    auto advance = [](int& slot, int& round) {
      slot += 2;
      if (slot >= C::kStages) slot -= C::kStages, ++round;
    };
    do {
      const int tiles = k.piece(), n = kPair ? 2 * tiles : tiles;
#pragma unroll 1
      for (int i = 0; i < n + 2; i += 2) {
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const int step = i + g, j = step - 2;
          const bool first = !kPair || g == 0, last = !kPair || g == 1;  // of a key tile
          const bool pv = j >= 0 && j < n, s = step < n;
          if (!pv && !s) continue;
          int on = -1, parity = 0;  // what this lane waits for
          if (lane == 0 && s && first) on = C::bFull + kslot, parity = kround;
          if (lane == 1 && pv && first) on = C::bFull + vslot, parity = vround;
          if (lane == 2 && pv) on = C::bPF + g, parity = pcount >> g;
          if (lane == 3 && s && step < 2) on = C::bQF + g, parity = seg;
          if (on >= 0) wait(on, parity & 1);
          dead = __any_sync(0xffffffffu, dead);
          tc_fence_after();
          const int ku = uniform(kslot), vu = uniform(vslot);
          if (lane == 0 && !dead) {
            if (pv) {
              values(tm, base, g, vu, j > 1);
              if (!s) mma_commit(bar(C::bOF + g));
            }
            if (s) {
              scores(tm, base, g, ku);
              mma_commit(bar(C::bSF + g));
            }
          }
          __syncwarp();
          if (pv) pcount ^= 1u << g;
          if (pv && last) advance(vslot, vround);
          if (s && last) advance(kslot, kround);
        }
      }
      ++seg;
    } while (next(k));
    if (lane == 0) {
      mma_commit(bar(C::bDrain));
      mbar_wait(bar(C::bDrain), 0, 100000000ull);
    }
  }

  // --------------------------------------------------------------- softmax --
  // `threads` threads bring 128 query rows of the segment, from `first` on, to `to`.
  template <int kThreads>
  __device__ __forceinline__ void load_queries(const Walk<true>& k, int first, uint32_t to, int thread) {
    constexpr int kCh = D / 8, kPer = kBigRows * kCh / kThreads;  // 16-byte chunks of a row, of a thread
    constexpr int kStep = kThreads / kCh;                         // rows between them
    const int h = head(k), M = k.s.n * p.G, ch = thread % kCh;
    const Rows from(p.G, first + thread / kCh, kStep);
    const __nv_bfloat16* base = p.q + (int64_t)k.s.q0 * p.q_ts + (int64_t)h * p.G * D + ch * 8;
    uint4 x[kPer];
    Rows at = from;
#pragma unroll
    for (int i = 0; i < kPer; ++i, at.next()) {
      x[i] = make_uint4(0, 0, 0, 0);
      if (at.row < M) x[i] = *reinterpret_cast<const uint4*>(base + at.tok * p.q_ts + (int64_t)at.g * D);
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int r = thread / kCh + i * kStep;
      const uint4 y = no_infinity(x[i]);
      sts128(to + (ch / 8) * C::kChunk + swz<128>(r, ch % 8), y.x, y.y, y.z, y.w);
    }
    fence_async_smem();
  }

  __device__ __forceinline__ void softmax(Walk<true> k, int g, bool firstp) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int r = 32 * (warp % 4) + lane;
    const uint32_t mine = tmem + ((uint32_t)(32 * (warp % 4)) << 16);  // this warp's lanes of TMEM
    const uint32_t colS = mine + 128 * g, colO = mine + 256 + D * g;
    const float c2 = p.c;
    float* turn = reinterpret_cast<float*>(smem_ptr + C::kOffTurn) + warp * 32 * 32;
    uint32_t scount = 0, ocount[2] = {0, 0};
    uint32_t ring = 0;  // tiles of the pieces before
    int seg = 0;
    // The slot of a tile's keys (values: 1) is free for this group.  Its scores' barrier tells
    // so of the keys, and of the values of its tile before, whose product was issued in front
    // of the scores: commits of their own would cost the issuing thread 130 cycles each.
    auto release = [&](int j, int values) {
      if (threadIdx.x % 128 == 0) mbar_arrive(bar(C::bEmpty + (int)((2 * (ring + j) + values) % C::kStages)));
    };
    const int unit = (int)blockIdx.x / (w.rows / C::kRows);
    auto bring = [&](const Walk<true>& x) {
      if (kPair)
        load_queries<128>(x, row0(x) + g * kBigRows, smem + g * C::kMat, threadIdx.x % 128);
      else
        load_queries<256>(x, row0(x), smem, threadIdx.x);
      mbar_arrive(bar(C::bQF + g));
      if (!kPair) mbar_arrive(bar(C::bQF + (g ^ 1)));
    };
    bring(k);
    bool more = true;
    do {
      const int n = k.piece(), len = k.s.len;
      float m = -INFINITY, l = 0.f, fix = 0.f;  // m: of raw scores
      for (int j = kPair ? 0 : g; j < n; j += kPair ? 1 : 2) {
        wait(C::bSF + g, scount++ & 1);
        tc_fence_after();
        release(j, 0);
        if (j >= (kPair ? 1 : 2)) release(j - (kPair ? 1 : 2), 1);
        const int keys = len - (k.tile + j) * kBigTile;  // of the prefix, from this tile on
        float s[128], top[2];
        auto read = [&]() {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t x[32];
            tmem_ld_x32(colS + 32 * q, x);
            tmem_ld_wait_x32(x);
#pragma unroll
            for (int i = 0; i < 32; ++i) s[32 * q + i] = __uint_as_float(x[i]);
          }
        };
        auto maxima = [&]() {
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const float* y = s + 64 * half;
            float a = fmaxf(y[0], y[1]), b = fmaxf(y[2], y[3]), c = fmaxf(y[4], y[5]), d = fmaxf(y[6], y[7]);
#pragma unroll
            for (int i = 8; i < 64; i += 8) {
              a = max3f(a, y[i], y[i + 1]);
              b = max3f(b, y[i + 2], y[i + 3]);
              c = max3f(c, y[i + 4], y[i + 5]);
              d = max3f(d, y[i + 6], y[i + 7]);
            }
            top[half] = fmaxf(max3f(a, b, c), d);
          }
        };
        if (keys >= kBigTile) {
          read();
          maxima();
        } else {
          read();
#pragma unroll
          for (int i = 0; i < 128; ++i) s[i] = i < keys ? s[i] : -INFINITY;
          maxima();
        }
        const float to = fmaxf(m, fmaxf(top[0], top[1]));
        float alpha = 1.f;
        bool grow = false;
        if (m == -INFINITY) {
          m = to;  // nothing is in O yet but zeros
        } else if ((to - m) * c2 > kRowsLazy) {
          grow = true;
          alpha = ex2((m - to) * c2);
          m = to;
        }
        const float neg = m == -INFINITY ? 0.f : -m * c2;
        // of one part: O is divided by the sum with the largest probability of each half as rounded
        float f = 0.f;
#pragma unroll
        for (int half = 0; half < (kTwo ? 0 : 2); ++half) {
          const float pm = ex2(fmaf(top[half], c2, neg));
          f += __bfloat162float(__float2bfloat16(pm)) - pm;
        }
        float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t pw[16], pr[16];  // probabilities as rounded, and what that leaves of them
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            float e[4];
            pfma(e[0], e[1], s[32 * q + i], s[32 * q + i + 1], c2, neg, neg);
            pfma(e[2], e[3], s[32 * q + i + 2], s[32 * q + i + 3], c2, neg, neg);
#pragma unroll
            for (int z = 0; z < 4; ++z) e[z] = ex2(e[z]);
            padd(s0, s1, e[0], e[1]);
            padd(s2, s3, e[2], e[3]);
            pw[i / 2] = rows::pack2(e[0], e[1]);
            pw[i / 2 + 1] = rows::pack2(e[2], e[3]);
            if (kTwo) {
              pr[i / 2] = rest_of(e[0], e[1], pw[i / 2]);
              pr[i / 2 + 1] = rest_of(e[2], e[3], pw[i / 2 + 1]);
            }
          }
          tmem_st_x16(colS + 16 * q, pw);
          if (kTwo) tmem_st_x16(colS + 64 + 16 * q, pr);
        }
        l = l * alpha + ((s0 + s1) + (s2 + s3));
        fix = fix * alpha + f;
        if (j >= (kPair ? 1 : 2) && __any_sync(0xffffffffu, grow)) {
#pragma unroll 1
          for (int col = 0; col < D; col += 32) {
            uint32_t o[32];
            tmem_ld_x32(colO + col, o);
            tmem_ld_wait_x32(o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
            tmem_st_x32(colO + col, o);
          }
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(bar(C::bPF + g));
      }
      // ------------------------------------------------- the piece's end --
      const int first_row = row0(k) + (kPair ? g * kBigRows : 0), M = k.s.n * p.G, h = head(k), q0 = k.s.q0;
      const bool whole = k.tile == 0 && n == k.tiles;
      more = next(k);  // k is the next piece's from here on
      if (kPair && more) bring(k);  // the last S product has read this group's queries
      if (kPair || n > g) {
        wait(C::bOF + g, ocount[g]++ & 1);
        release(kPair ? n - 1 : n - 1 - ((n - 1 - g) & 1), 1);
      }
      ring += n;
      if (!kPair) {
        if (n > (g ^ 1)) wait(C::bOF + (g ^ 1), ocount[g ^ 1]++ & 1);
        ss.ml[g][r] = make_float2(m, l);
        ss.fix[g][r] = fix;
        asm volatile("bar.sync 2, 256;" ::: "memory");
      }
      tc_fence_after();
      const bool poison = aborted() || *(volatile int*)&ss.bad[seg % kFlags];
      if (threadIdx.x == 0) ss.bad[(seg + kFlags / 2) % kFlags] = 0;
      const float2 a = kPair ? make_float2(m, l) : ss.ml[0][r];
      const float2 b = kPair ? make_float2(-INFINITY, 0.f) : ss.ml[1][r];
      const float mm = fmaxf(a.x, b.x);
      // a side counts unless it saw nothing (a sum of NaN is not nothing, nor is one without a maximum)
      const bool sa = a.y != 0.f, sb = !kPair && b.y != 0.f;
      const float wa = sa ? (a.x == -INFINITY ? 1.f : ex2((a.x - mm) * c2)) : 0.f;
      const float wb = sb ? (b.x == -INFINITY ? 1.f : ex2((b.x - mm) * c2)) : 0.f;
      const float ls = (sa ? wa * a.y : 0.f) + (sb ? wb * b.y : 0.f);
      const float lo = kPair ? l + fix : ls + wa * ss.fix[0][r] + wb * ss.fix[1][r];
      const float inv = ls != 0.f ? 1.f / lo : 0.f;
      const int64_t slot = whole ? -1 : (int64_t)(2 * unit + !firstp) * w.rows + first_row % w.rows;
      float* const part = whole ? p.o_row : p.o_part;
      // where a row goes
      auto place = [&](const Rows& x) {
        return whole ? (int64_t)(q0 + x.tok) * p.Hq + h * p.G + x.g : slot + (x.row - first_row);
      };
      if (first_row + r < M && (kPair || g == 0)) {
        float lse = ls != 0.f ? ((mm == -INFINITY ? 0.f : mm * c2) + lg2(ls)) * 0.69314718055994531f : -INFINITY;
        if (poison) lse = INFINITY;  // makes the join of the pieces a NaN row
        (whole ? p.lse_row : p.lse_part)[place(Rows(p.G, first_row + r, 1))] = lse;
      }
      int64_t to[8];  // of rows 4 i + lane / 8 of this warp
      Rows x(p.G, first_row + 32 * (warp % 4) + lane / 8, 4);
#pragma unroll
      for (int i = 0; i < 8; ++i, x.next()) to[i] = x.row < M ? place(x) * D : -1;
#pragma unroll 1
      for (int col = kPair ? 0 : g * (D / 2); col < (kPair ? D : (g + 1) * (D / 2)); col += 32) {
        uint32_t xa[32], xb[32];
        tmem_ld_x32((kPair ? colO : mine + 256) + col, xa);
        if (!kPair) tmem_ld_x32(mine + 256 + D + col, xb);
        tmem_ld_wait_x32(xa);
        if (!kPair) tmem_ld_wait_x32(xb);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 32; i += 4) {  // 16-byte chunk c of row r at 128 r + 16 (c ^ r % 8)
          float y[4];
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            y[z] = sa ? wa * __uint_as_float(xa[i + z]) : 0.f;
            if (!kPair) y[z] += sb ? wb * __uint_as_float(xb[i + z]) : 0.f;
            y[z] = inv != 0.f ? y[z] * inv : 0.f;
            if (poison) y[z] = NAN;
          }
          *reinterpret_cast<float4*>(turn + 32 * lane + 4 * ((i / 4) ^ (lane & 7))) = make_float4(y[0], y[1], y[2], y[3]);
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int rr = 4 * i + lane / 8, ch = lane % 8;
          if (to[i] >= 0)
            *reinterpret_cast<float4*>(part + to[i] + col + 4 * ch) =
                *reinterpret_cast<const float4*>(turn + 32 * rr + 4 * (ch ^ (rr & 7)));
        }
      }
      tc_fence_before();
      // every thread has read the piece's flags (and both groups' O, maxima and queries)
      if (!kPair) {
        asm volatile("bar.sync 2, 256;" ::: "memory");
        if (more) bring(k);
      }
      firstp = false;
      ++seg;
    } while (more);
  }
};

template <int D, bool kPair, bool kTwo>
__global__ void __launch_bounds__(kRowsThreads, 1)
prefix_rows_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                   const __grid_constant__ Params p, const __grid_constant__ Work w) {
  using C = RowsCfg<D, kPair>;
  extern __shared__ __align__(1024) uint8_t smem_rows[];
  static_assert(C::kBars <= 32, "barriers");
  static_assert(C::kSmem <= 227 * 1024, "shared memory");
  RowsShared& ss = *reinterpret_cast<RowsShared*>(smem_rows + C::kOffShared);
  const int warp = threadIdx.x / 32;
  auto init = [&](int first, int n, int count) {
    for (int i = 0; i < n; ++i) mbar_init(smem_u32(&ss.bars[first + i]), count);
  };
  if (threadIdx.x == 0) {
    init(C::bFull, C::kStages, 1);
    init(C::bEmpty, C::kStages, kPair ? 2 : 1);  // groups that take a tile
    init(C::bSF, 2, 1);
    init(C::bPF, 2, 128);
    init(C::bOF, 2, 1);
    init(C::bQF, 2, kPair ? 128 : 256);
    init(C::bDrain, 1, 1);
    fence_mbar_init();
    ss.abort = 0;
    for (int i = 0; i < kFlags; ++i) ss.bad[i] = 0;
  }
  begin_line(p);
  grid_dep_launch();
  if (smem_u32(smem_rows) & 1023u) {  // the swizzled tiles would be read askew
    if (threadIdx.x == 0) atomicOr(p.err, kTimedOut);
    end_line(p);
    return;
  }
  Walk<true> k;
  if (!find_place(p, w, blockIdx.x / (w.rows / C::kRows), false, k)) {  // the whole CTA
    end_line(p);
    return;
  }
  if (threadIdx.x >= 128) {  // queries, one row to a thread
    const int row = k.seg % (k.segs / p.H) * w.rows + (int)blockIdx.x % (w.rows / C::kRows) * C::kRows + (int)threadIdx.x - 128;
    if (row < k.s.n * p.G) {
      const int tok = row / p.G;
      const __nv_bfloat16* q = p.q + (int64_t)(k.s.q0 + tok) * p.q_ts + (int64_t)(k.seg / (k.segs / p.H) * p.G + row - tok * p.G) * D;
      prefetch(q);
      if (D == 128) prefetch(q + 64);
    }
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(&ss.tmem), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  RowsRole<D, kPair, kTwo> role{p, w, ss, smem_rows, smem_u32(smem_rows), ss.tmem};
  const bool firstp = role.busy(k), any = firstp || role.next(k);
  if (warp < 8) {
    regs_inc<kRowsSoftmaxRegs>();
    if (any) role.softmax(k, warp / 4, firstp);
  } else {
    regs_dec<kRowsRestRegs>();
    if (!any) {
    } else if (warp == 8)
      role.produce(k, &map_k, &map_v);
    else if (warp == 9)
      role.multiply(k);
    __syncwarp();
  }
  if (role.aborted()) {  // let copies in flight land before the CTA leaves
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 1000000ull) {
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(ss.tmem, 512);
  }
  end_line(p);
}

}  // namespace tree
}  // namespace attn
