// Attention of the newest tokens over the paged cache for many query rows of a
// key head (a tree of drafts times the heads of a group), on the tensor cores'
// tcgen05 products.
//
// A segment is (sequence, key head, 128 or 256 query rows); persistent CTAs, one an
// SM, take equal shares of the line of 128-key tiles.  A key tile costs the tensor
// core 1024 cycles for 128 rows (S = Q K^T and O += P V, 128 x 128 x d each; d = 128)
// whatever part of the rows is real; its e4m3 bytes take 1410 cycles from HBM (bf16:
// 2820).  Trees of 64 drafts (8 sequences of up to 16384 keys, 64 query and 8 key
// heads, d = 128) take 284 us with e4m3 codes and 225 us with a bf16 cache, 820 and
// 1040 TFLOP/s: what bounds them is the way of one row tile around the roles (scores
// 600 cycles, softmax 2100 or 1650, P V 600, and some 200 for each look at a
// barrier), of which two are under way at a time.  Shared memory is busy for 3200 of
// the 5300 cycles that two row tiles take over codes: 1536 for the products'
// operands, 1024 for the key scales (every thread takes all 128 of a tile, 512 bytes
// into its registers), 640 for copies and conversions.  So a score is multiplied by
// its key's scale once, and goes back to tensor memory (reading the scales again in
// the second pass: 330 us; loading them a batch ahead: 292).
//
// Warps: 0-3 and 4-7 softmax groups A and B (a thread owns a row), each with its own
// S and O in TMEM, so that one group's softmax runs beside the other's products;
// 8-11 operands: they write the segment's Q tile, turn a tile's codes of V into fp16
// values, and clean values that rows may not see; 12 and 14 TMA producers of keys and
// values; 13 issues the products.  kPair, for more than 128 rows of a head: A and B
// take the two row tiles over the same key tiles, which are copied and converted once
// for both (trees of 64 drafts 311 -> 299 us, bf16 320 -> 268).  Else: A takes the
// even key tiles of a segment, B the odd ones, and they meet at the segment's end.
//
// The roles' code lies in loops kept short (32 keys of a softmax row, 16 channels
// of a conversion at a time): fourteen warps run six different loops at once, and
// unrolled through a tile they wait for instructions (424 us against 311).
//
// With e4m3 codes S = (Q_hi + Q_lo) K^T takes the codes of K as they lie in the
// cache: a query row, scaled by a power of two to at most 256, is the sum of two
// e4m3 values (4 + 4 significant bits hold bf16's 8 exactly, down to 2^-11 of the
// row's largest channel, where the quantum 2^-9 of the small part ends it: an
// error below 2^-18 of the largest), and the two e4m3 products cost what one fp16
// product does; the softmax multiplies a score by its key's scale.  V is converted
// with its scale: fp16(code * scale * 2^(6 - F)), off by 2^-11, F a running
// exponent of a piece's value scales (O is rescaled when it grows).  P is
// fp16(2^7 p): 2^-11, and 2^-32 absolute for the smallest.
//
// One F for all rows serves while the scales of the piece lie within 2^kSpread of each
// other.  From the tile on where they do not (a hidden draft with huge values, a token
// with tiny ones that takes nearly all the weight) V is the codes alone and P takes the
// scales: fp16(2^(13 - F) p scale), F each row's own, from the largest p scale that it
// sees.  Such a tile takes a third pass over the scores.
#pragma once

#include <climits>
#include <cstddef>

#include "attn_tree_work.cuh"

namespace attn {
namespace tree {

constexpr int kBigTile = 128;  // keys
constexpr int kLogBigTile = 7;
constexpr int kBigRows = 128;
constexpr int kBigThreads = 512;
// Registers after setmaxnreg; 128 threads each: two softmax groups, operands, the
// rest.  Their sum is the launch's 512 x 128, and with them nothing spills (192, 80
// and 48 spilled 260 bytes: 340 us against 313).
constexpr int kSoftmaxRegs = 176, kOperandRegs = 80, kRestRegs = 80;
constexpr int kRing = 8;  // segments whose flags are kept
constexpr float kPLog2 = 7.f;  // P is stored as fp16(2^7 p), room for 2^kLazy above
constexpr int kSpread = 12;       // log2
constexpr int kFar = INT_MAX;     // in place of a tile's F: the scales lie further apart
// Exponent of cache_write's smallest scale, in most cases a row of zeros': not counted
// among the scales that may lie far apart.  (Values below 2^-55, its others, count as
// zeros beside scales that are.)
constexpr int kScaleFloor = -64;

template <int D, bool kCodes, bool kPair>
struct BigCfg : Row<D, kCodes> {
  using Row<D, kCodes>::kRowBytes;
  static constexpr int kMat = kBigTile * kRowBytes;             // K or V of a tile, as in the cache
  static constexpr int kChunk = kBigTile * 128;                 // 128 rows of 128 bytes
  static constexpr int kConv = kCodes ? kBigTile * D * 2 : 0;   // V in fp16
  static constexpr int kQ1 = kBigRows * D * 2;                  // bf16, or the two e4m3 parts
  static constexpr int kQ = (kPair ? 2 : 1) * kQ1;
  static constexpr int kRows = (kPair ? 2 : 1) * kBigRows;      // of a segment
  // stages
  static constexpr int kK = D == 64 ? 4 : kCodes ? (kPair ? 3 : 4) : (kPair ? 2 : 3);
  static constexpr int kV = D == 64 ? 4 : kCodes && kPair ? 2 : 3;
  static constexpr int kReady = kCodes ? 2 : kV;                // V operand buffers
  static constexpr int kMeta = kCodes ? 4 : 1;                  // tiles whose factors are kept
  static constexpr int kOffK = kQ;
  static constexpr int kOffV = kOffK + kK * kMat;
  static constexpr int kOffC = kOffV + kV * kMat;
  static constexpr int kOffScale = kOffC + kReady * kConv;            // [kK][2][128] raw scales
  static constexpr int kOffMeta = kOffScale + (kCodes ? kK * 1024 : 0);  // [kMeta][128] key factors
  static constexpr int kOffFar = kOffMeta + (kCodes ? kMeta * 512 : 0);  // [kMeta][128] log2 of value scales, where far apart
  static constexpr int kOffShared = kOffFar + (kCodes ? kMeta * 512 : 0);
  // barriers
  static constexpr int bKF = 0, bKE = bKF + kK, bVF = bKE + kK, bVE = bVF + kV, bRF = bVE + kV, bRE = bRF + kReady,
                       bMF = bRE + kReady, bME = bMF + kMeta, bSF = bME + kMeta, bPF = bSF + 2, bOF = bPF + 2,
                       bQF = bOF + 2, bQE = bQF + 1, bOFree = bQE + 1, bDrain = bOFree + 1, kBars = bDrain + 1;
};

// kind::f16 with fp16 A and B (formats 0), fp32 D; B MN-major.
__host__ __device__ constexpr uint32_t idesc_f16_mn(uint32_t M, uint32_t N) {
  return (1u << 4) | (1u << 16) | ((N >> 3) << 17) | ((M >> 4) << 24);
}
// kind::f8f6f4 with e4m3 A and B (formats 0), fp32 D, both K-major.
__host__ __device__ constexpr uint32_t idesc_e4m3(uint32_t M, uint32_t N) {
  return (1u << 4) | ((N >> 3) << 17) | ((M >> 4) << 24);
}
__device__ __forceinline__ void mma_e4m3(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n"
      "  .reg .pred p;\n"
      "  setp.ne.b32 p, %4, 0;\n"
      "  tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n"
      "}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Packed fp32 pairs.
__device__ __forceinline__ void pmul(float& a0, float& a1, float b0, float b1) {
  asm("{\n .reg .b64 x, y, r;\n mov.b64 x, {%0, %1};\n mov.b64 y, {%2, %3};\n mul.rn.f32x2 r, x, y;\n mov.b64 {%0, %1}, r;\n}"
      : "+f"(a0), "+f"(a1)
      : "f"(b0), "f"(b1));
}
__device__ __forceinline__ void padd(float& a0, float& a1, float b0, float b1) {
  asm("{\n .reg .b64 x, y, r;\n mov.b64 x, {%0, %1};\n mov.b64 y, {%2, %3};\n add.rn.f32x2 r, x, y;\n mov.b64 {%0, %1}, r;\n}"
      : "+f"(a0), "+f"(a1)
      : "f"(b0), "f"(b1));
}
// (d0, d1) = (a0, a1) * b + (c0, c1)
__device__ __forceinline__ void pfma(float& d0, float& d1, float a0, float a1, float b, float c0, float c1) {
  asm("{\n .reg .b64 x, y, z, r;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %4};\n mov.b64 z, {%5, %6};\n"
      " fma.rn.f32x2 r, x, y, z;\n mov.b64 {%0, %1}, r;\n}"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b), "f"(c0), "f"(c1));
}
__device__ __forceinline__ float max3f(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Behind the tiles in dynamic shared memory (there is no static one, so the
// dynamic one begins at an address that is a multiple of 1024; the kernel checks).
struct BigShared {
  uint64_t bars[48];
  uint32_t tmem;
  int abort;                  // a wait ran out
  int bad[kRing];             // the segment reads a page outside the cache
  uint32_t hidden[kRing][2];  // its new tokens with values that are not finite
  float2 ml[2][kBigRows];     // [group]: maxima and sums
  __nv_bfloat16 fix[2][kBigRows];  // [group]: bf16: what rounding the largest probabilities adds to the sum
  // for codes
  int4 vexp[2];               // [tile's parity], of the four operand warps: exponents of value scales,
                              // the largest (low half) and minus the smallest
  int vref[4];                // by tile: the exponent F of its values, or kFar
  int fend[2][kBigRows];      // [group]: F of a row's O
  float rc[2][2 * kBigRows];  // [segment's parity]: log2 units of a row's raw score
};
template <int D, bool kCodes, bool kPair>
__host__ __device__ constexpr int big_smem() {
  return BigCfg<D, kCodes, kPair>::kOffShared + (kCodes ? (int)sizeof(BigShared) : (int)offsetof(BigShared, vexp));
}

__device__ __forceinline__ uint32_t half_mul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t half_fma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
// 2^e for e in -126 .. 127, 0 below.
__device__ __forceinline__ float pow2(int e) { return e < -126 ? 0.f : __uint_as_float((uint32_t)(127 + min(e, 127)) << 23); }

template <int D, bool kCodes, bool kPair>
struct Big {
  using C = BigCfg<D, kCodes, kPair>;
  const Params& p;
  const Work& w;
  BigShared& ss;
  uint8_t* smem_ptr;  // 1024-byte aligned
  uint32_t smem, tmem;

  __device__ __forceinline__ uint32_t bar(int i) const { return smem_u32(&ss.bars[i]); }
  // Bounded; once one wait of a CTA has run out no thread waits twice more, every
  // role goes through its loops to the end, and the rows come out as NaN.  (The
  // flag is looked at only when a barrier is not there yet: the thread that issues
  // the products passes three barriers a tile.)
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
  __device__ __forceinline__ int head(const Walk& k) const { return k.seg / (k.segs / p.H); }
  __device__ __forceinline__ int row0(const Walk& k) const { return k.seg % (k.segs / p.H) * C::kRows; }

  // ------------------------------------------------------------- producers --
  // One warp copies the keys (and the scales), another the values, each as far
  // ahead as its stages reach.
  template <bool kKeys>
  __device__ __forceinline__ void produce(Walk k, const CUtensorMap* map) {
    constexpr int kN = kKeys ? C::kK : C::kV, kFull = kKeys ? C::bKF : C::bVF, kEmpty = kKeys ? C::bKE : C::bVE;
    constexpr int kElems = kCodes ? C::kBox : C::kBox / 2;
    const int lane = threadIdx.x % 32;
    const int page = 1 << p.log_page;
    const int box = min(page, kBigTile), per = kBigTile / box;  // rows of a copy, copies of a tile
    const int batch = 32 / per;  // tiles whose page numbers one load fetches
    int s = 0, round = 0, seg = 0;
    do {
      const int h = head(k), len = k.s.len, end = k.tile + k.piece();
      const int* table = p.table + (int64_t)k.b * p.stride;
      auto fetch = [&](int tile) {
        const int64_t pos = (int64_t)tile * kBigTile + lane * box;
        return pos < len ? table[pos >> p.log_page] : 0;
      };
      int ids = fetch(k.tile);
      for (int t0 = k.tile; t0 < end; t0 += batch) {
        const int next = t0 + batch < end ? fetch(t0 + batch) : 0;
        const bool wrong = (unsigned)ids >= (unsigned)p.pages;
        if (wrong) ids = 0;
        const uint32_t wrongs = __ballot_sync(0xffffffffu, wrong);
        for (int t = t0; t < min(t0 + batch, end); ++t) {
          const int key0 = t * kBigTile, n = min(per, (len - key0 + box - 1) / box);
          const int id = __shfl_sync(0xffffffffu, ids, (t - t0) * per + lane % per);
          if (round > 0) wait(kEmpty + s, (round & 1) ^ 1);
          __syncwarp();
          if (!__any_sync(0xffffffffu, dead)) {
            const uint32_t full = bar(kFull + s);
            if (lane == 0) {
              if (kKeys && (wrongs >> ((t - t0) * per) & ((1u << per) - 1))) {
                ss.bad[seg % kRing] = 1;
                atomicOr(p.err, rows::kBadIndex);
              }
              mbar_arrive_expect_tx(full, n * box * C::kRowBytes);
            }
            __syncwarp();
            if (lane < n) {
              const int row = (id << p.log_page) + ((key0 + lane * box) & (page - 1));
              const uint32_t dst = smem + (kKeys ? C::kOffK : C::kOffV) + s * C::kMat + lane * box * C::kBox;
#pragma unroll
              for (int f = 0; f < C::kHalves; ++f)
                tma_load_3d(dst + f * kBigTile * C::kBox, map, full, f * kElems, h, row);
            }
            if (kKeys && kCodes) {  // each lane: four key scales and four value scales
              const int key = key0 + 4 * lane;
              const int sid = __shfl_sync(0xffffffffu, id, 4 * lane / box);
              if (key < len) {
                const int64_t at = (((int64_t)sid * p.H + h) << p.log_page) + (key & (page - 1));
                const uint32_t sd = smem + C::kOffScale + s * 1024 + 16 * lane;
                cp_async16(sd, p.kscale + at);
                cp_async16(sd + 512, p.vscale + at);
              }
              cp_async_arrive(full);
            }
          }
          if (++s == kN) s = 0, ++round;
        }
        ids = next;
      }
      ++seg;
    } while (k.next(p, w));
    if (kKeys && kCodes) asm volatile("cp.async.wait_all;" ::: "memory");
  }

  // -------------------------------------------------------------- products --
  __device__ __forceinline__ void scores(uint32_t tmem, int g, int ks) {
    const uint32_t k = smem + C::kOffK + ks * C::kMat, d = tmem + 128 * g, q = smem + (kPair ? g * C::kQ1 : 0);
    if (kCodes) {
      constexpr uint32_t kSwz = C::kBox == 128 ? 2 : 4;  // 128- or 64-byte swizzle
      const uint64_t hi = make_sdesc(q, 16, 8 * C::kBox, kSwz);
      const uint64_t lo = make_sdesc(q + kBigRows * C::kBox, 16, 8 * C::kBox, kSwz);
      const uint64_t b = make_sdesc(k, 16, 8 * C::kBox, kSwz);
#pragma unroll
      for (int part = 0; part < 2; ++part) {
        const uint64_t a = part ? lo : hi;
#pragma unroll
        for (int kk = 0; kk < D / 32; ++kk) mma_e4m3(d, a + 2 * kk, b + 2 * kk, idesc_e4m3(128, 128), part | kk);
      }
    } else {
      const uint64_t a = make_sdesc(q, 16, 1024, kSwizzle128B), b = make_sdesc(k, 16, 1024, kSwizzle128B);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint64_t off = (uint64_t)(((kk / 4) * C::kChunk + (kk % 4) * 32) >> 4);
        mma_ss(d, a + off, b + off, make_idesc_bf16(128, 128, false), kk > 0);
      }
    }
  }
  __device__ __forceinline__ void values(uint32_t tmem, int g, int r, bool accumulate) {
    const uint32_t v = kCodes ? smem + C::kOffC + r * C::kConv : smem + C::kOffV + r * C::kMat;
    const uint64_t b = make_sdesc(v, C::kChunk, 1024, kSwizzle128B);
    constexpr uint32_t kI = kCodes ? idesc_f16_mn(128, D) : make_idesc_bf16(128, D, true);
#pragma unroll
    for (int kk = 0; kk < kBigTile / 16; ++kk)
      mma_ts(tmem + 256 + D * g, tmem + 128 * g + 8 * kk, b + (uint64_t)((kk * 2048) >> 4), kI, kk > 0 || accumulate);
  }
  // One thread issues every product, in the order of the steps (a step is a key tile,
  // or with kPair a key tile of one row tile): S(0), S(1), then for each step j its
  // P V and S(j + 2).  The warp's lanes look at the barriers of a step together: one
  // look is some 200 cycles (370 -> 340 us, and 299 -> 290 in one call).
  __device__ __forceinline__ void multiply(Walk k) {
    const int lane = threadIdx.x % 32;
    // Values that are the same in every lane, for the compiler to see: descriptors are
    // then made in uniform registers, and products follow each other faster (trees of
    // 64 drafts, bf16 cache 241 -> 225 us).  Over codes that takes shared memory from
    // the softmax and the conversions (285 -> 295).
    auto uniform = [](int x) { return kCodes ? x : __shfl_sync(0xffffffffu, x, 0); };
    const uint32_t tm = uniform(tmem);
    int ks = 0, kr = 0, rs = 0, rr = 0, seg = 0;
    uint32_t pcount = 0;  // bit g: parity of group g's next probabilities
    do {
      const int n = kPair ? 2 * k.piece() : k.piece();
#pragma unroll 1
      for (int i = 0; i < n + 2; ++i) {
        const int g = i & 1, j = i - 2;
        const bool first = !kPair || g == 0, last = !kPair || g == 1;  // of a key tile
        int on = -1, parity = 0;  // what this lane waits for
        if (lane == 0 && i < n && first) on = C::bKF + ks, parity = kr;
        if (lane == 1 && j >= 0 && first) on = C::bRF + rs, parity = rr;
        if (lane == 2 && j >= 0) on = C::bPF + g, parity = pcount >> g;
        if (lane == 3 && i == 0) on = C::bQF, parity = seg;
        if (lane == 4 && j == 0 && seg > 0) on = C::bOFree, parity = seg - 1;
        if (on >= 0) wait(on, parity & 1);
        dead = __any_sync(0xffffffffu, dead);
        tc_fence_after();
        const int gu = uniform(g), ku = uniform(ks), ru = uniform(rs);
        if (lane == 0 && !dead) {
          if (j >= 0) {
            values(tm, gu, ru, j > 1);
            if (last) mma_commit(bar(kCodes ? C::bRE + rs : C::bVE + rs));
            if (i >= n) mma_commit(bar(C::bOF + g));
          }
          if (i < n) {
            scores(tm, gu, ku);
            mma_commit(bar(C::bSF + g));
          }
        }
        __syncwarp();
        if (j >= 0) {
          pcount ^= 1u << g;
          if (last && ++rs == C::kReady) rs = 0, ++rr;
        }
        if (i < n && last && ++ks == C::kK) ks = 0, ++kr;
      }
      ++seg;
    } while (k.next(p, w));
    if (lane == 0) {
      mma_commit(bar(C::bDrain));
      mbar_wait(bar(C::bDrain), 0, 100000000ull);
    }
  }

  // -------------------------------------------------------------- operands --
  // This thread's query row of the segment (of each of its tiles) into the Q tile.
  __device__ __forceinline__ void write_query(const Walk& k, int seg) {
#pragma unroll 1
    for (int i = 0; i < C::kRows / kBigRows; ++i) write_row(k, seg, i);
    fence_async_smem();
    mbar_arrive(bar(C::bQF));
  }
  __device__ __forceinline__ void write_row(const Walk& k, int seg, int part) {
    const int r = threadIdx.x % 128;
    const int h = head(k), row = row0(k) + part * kBigRows + r, M = k.s.n * p.G;
    const uint32_t to = smem + part * C::kQ1;
    const bool live = row < M;
    const int tok = live ? row / p.G : 0;
    const __nv_bfloat16* q = p.q + (int64_t)(k.s.q0 + tok) * p.q_ts + (int64_t)(h * p.G + (live ? row - tok * p.G : 0)) * D;
    if (!kCodes) {
#pragma unroll 8
      for (int ch = 0; ch < D / 8; ++ch) {
        const uint4 x = live ? no_infinity(*reinterpret_cast<const uint4*>(q + 8 * ch)) : make_uint4(0, 0, 0, 0);
        sts128(to + (ch / 8) * C::kChunk + swz<128>(r, ch % 8), x.x, x.y, x.z, x.w);
      }
    } else {
      uint32_t top = 0;  // largest magnitude: bf16 bits order like the values
#pragma unroll 8
      for (int ch = 0; ch < D / 8; ++ch) {
        const uint4 x = live ? *reinterpret_cast<const uint4*>(q + 8 * ch) : make_uint4(0, 0, 0, 0);
        const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) top = max(top, max(u[i] & 0x7fffu, (u[i] >> 16) & 0x7fffu));
      }
      int e = (int)(top >> 7) - 127;
      e = top == 0 ? 0 : min(max(e, -119), 126);
      const float up = __uint_as_float((uint32_t)(127 + 7 - e) << 23);
      ss.rc[seg & 1][part * kBigRows + r] = __uint_as_float((uint32_t)(127 + e - 7) << 23);
#pragma unroll 2
      for (int ch = 0; ch < D / 16; ++ch) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint4 x =
              live ? no_infinity(*reinterpret_cast<const uint4*>(q + 16 * ch + 8 * half)) : make_uint4(0, 0, 0, 0);
          const uint32_t u[4] = {x.x, x.y, x.z, x.w};
          uint32_t hp[4], lp[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float a = __uint_as_float(u[i] << 16) * up, b = __uint_as_float(u[i] & 0xffff0000u) * up;
            hp[i] = e4m3_pair(a, b);
            const uint32_t back = codes_lo(hp[i]);
            float ha, hb;
            asm("{\n .reg .b16 x, y;\n mov.b32 {x, y}, %2;\n cvt.f32.f16 %0, x;\n cvt.f32.f16 %1, y;\n}\n"
                : "=f"(ha), "=f"(hb)
                : "r"(back));
            lp[i] = e4m3_pair(a - ha, b - hb);
          }
          hi[2 * half] = hp[0] | hp[1] << 16, hi[2 * half + 1] = hp[2] | hp[3] << 16;
          lo[2 * half] = lp[0] | lp[1] << 16, lo[2 * half + 1] = lp[2] | lp[3] << 16;
        }
        const uint32_t at = to + swz<C::kBox>(r, ch);
        sts128(at, hi[0], hi[1], hi[2], hi[3]);
        sts128(at + kBigRows * C::kBox, lo[0], lo[1], lo[2], lo[3]);
      }
    }
  }

  __device__ __forceinline__ void prepare(Walk k) {
    const int r = threadIdx.x % 128, lane = threadIdx.x % 32;  // thread r: key r of a tile
    int ks = 0, kr = 0, vs = 0, vr = 0, rs = 0, rr = 0, ms = 0, mr = 0, seg = 0, vref = 0, low = 0, tile_parity = 0;
    do {
      if (seg > 0) wait(C::bQE, (seg - 1) & 1);
      write_query(k, seg);
      const int len = k.s.len, ctx = len - k.s.n, end = k.tile + k.piece();
      uint32_t* hidden = ss.hidden[seg % kRing];
      for (int t = k.tile; t < end; ++t) {
        const int pos = t * kBigTile + r;
        bool cut = false;  // the value scale is not finite, for a key that rows may not see
        bool far = false;  // the piece's value scales so far lie too far apart for one F
        float vscale = 0.f;
        if (kCodes) {
          wait(C::bKF + ks, kr & 1);
          if (mr > 0) wait(C::bME + ms, (mr & 1) ^ 1);
          const uint32_t sc = smem + C::kOffScale + ks * 1024 + 4 * r;
          const float kscale = __uint_as_float(lds32(sc));
          vscale = __uint_as_float(lds32(sc + 512));
          if (pos >= ctx && !(fabsf(vscale) < INFINITY)) {
            cut = pos < len;
            vscale = 0.f;
          }
          if (pos >= len) vscale = 0.f;
          // F: the largest exponent so far, with room to grow by two before O is rescaled
          const uint32_t bits = __float_as_uint(vscale) & 0x7fffffffu;
          const int e = bits < 0x7f800000u ? (int)(bits >> 23) - 127 : -127;
          const int most = __reduce_max_sync(0xffffffffu, e);
          const int minus = __reduce_max_sync(0xffffffffu, e > kScaleFloor ? -e : -127);
          const int turn = tile_parity;
          tile_parity ^= 1;
          if (lane == 0)
            reinterpret_cast<uint32_t*>(&ss.vexp[turn])[threadIdx.x / 32 % 4] = (uint32_t)(most & 0xffff) | (uint32_t)minus << 16;
          asm volatile("bar.sync 3, 128;" ::: "memory");
          const int4 by = ss.vexp[turn];
          const uint32_t both = __vmaxs2(__vmaxs2(by.x, by.y), __vmaxs2(by.z, by.w));
          const int all = (int16_t)(both & 0xffff), least = -((int)both >> 16);
          if (t == k.tile || all > vref) vref = max(all, -100) + 2;
          low = t == k.tile ? least : min(low, least);
          far = vref - low > kSpread + 2;
          *reinterpret_cast<float*>(smem_ptr + C::kOffMeta + ms * 512 + 4 * r) = kscale * p.c;
          if (far) *reinterpret_cast<float*>(smem_ptr + C::kOffFar + ms * 512 + 4 * r) = lg2(vscale);
          if (r == 0) ss.vref[ms] = far ? kFar : vref;
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(bar(C::bMF + ms));
            mbar_arrive(bar(C::bKE + ks));
          }
          if (++ks == C::kK) ks = 0, ++kr;
          if (++ms == C::kMeta) ms = 0, ++mr;
        }
        wait(C::bVF + vs, vr & 1);
        const uint32_t v = smem + C::kOffV + vs * C::kMat;
        bool odd = cut;  // something of this key's row is hidden from the products
        if (kCodes) {
          if (rr > 0) wait(C::bRE + rs, (rr & 1) ^ 1);
          const uint32_t dst = smem + C::kOffC + rs * C::kConv;
          // the scale as a sum of two fp16: code * hi + code * lo, rounded once more
          const float f = far ? 1.f : vscale * pow2(6 - vref);
          const uint32_t hi = pack_half(f, f);
          float fh;
          asm("{\n .reg .b16 x, y;\n mov.b32 {x, y}, %1;\n cvt.f32.f16 %0, x;\n}\n" : "=f"(fh) : "r"(hi));
          const uint32_t lo = pack_half(f - fh, f - fh);
          auto times = [&](uint32_t v) { return half_fma2(v, hi, half_mul2(v, lo)); };
          auto put = [&](int ch, const uint32_t (&u)[4]) {
            const int o = 2 * ch;  // 16-byte chunk of the fp16 row
            const uint32_t base = dst + (o / 8) * C::kChunk;
            sts128(base + swz<128>(r, o % 8), times(codes_lo(u[0])), times(codes_hi(u[0])), times(codes_lo(u[1])),
                   times(codes_hi(u[1])));
            sts128(base + swz<128>(r, o % 8 + 1), times(codes_lo(u[2])), times(codes_hi(u[2])), times(codes_lo(u[3])),
                   times(codes_hi(u[3])));
          };
          uint4 ahead = lds128(v + swz<C::kBox>(r, 0));
#pragma unroll 1
          for (int ch = 0; ch < D / 16; ++ch) {
            uint32_t u[4] = {ahead.x, ahead.y, ahead.z, ahead.w};
            ahead = lds128(v + swz<C::kBox>(r, min(ch + 1, D / 16 - 1)));
            if (pos >= ctx) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                if (pos >= len) u[i] = 0;
#pragma unroll
                for (int b = 0; b < 4; ++b)
                  if (((u[i] >> (8 * b)) & 0x7fu) == 0x7fu) u[i] &= ~(0xffu << (8 * b)), odd = true;
              }
            }
            put(ch, u);
          }
        } else if (pos >= ctx) {
#pragma unroll 1
          for (int ch = 0; ch < D / 8; ++ch) {
            const uint32_t at = v + (ch / 8) * C::kChunk + swz<128>(r, ch % 8);
            const uint4 x = lds128(at);
            uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (pos >= len) u[i] = 0;
              if ((u[i] & 0x7f80u) == 0x7f80u) u[i] &= 0xffff0000u, odd = true;
              if ((u[i] & 0x7f800000u) == 0x7f800000u) u[i] &= 0xffffu, odd = true;
            }
            sts128(at, u[0], u[1], u[2], u[3]);
          }
        }
        if (odd) atomicOr(hidden + ((pos - ctx) >> 5), 1u << ((pos - ctx) & 31));
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(C::bRF + rs));
          if (kCodes) mbar_arrive(bar(C::bVE + vs));
        }
        if (++vs == C::kV) vs = 0, ++vr;
        if (++rs == C::kReady) rs = 0, ++rr;
      }
      ++seg;
    } while (k.next(p, w));
  }

  // --------------------------------------------------------------- softmax --
  __device__ __forceinline__ void softmax(Walk k, int g) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int r = 32 * (warp % 4) + lane;
    const uint32_t mine = tmem + ((uint32_t)(32 * (warp % 4)) << 16);  // this warp's lanes of TMEM
    const uint32_t colS = mine + 128 * g;
    uint32_t scount = 0, ocount[2] = {0, 0};
    int ms = 0, mr = 0, ks = 0, seg = 0;
    bool firstp = true;
    do {
      const Seq sq = k.s;
      const int M = sq.n * p.G, ctx = sq.len - sq.n, r0 = row0(k) + (kPair ? g * kBigRows : 0), h = head(k);
      const int row = r0 + r, n = k.piece();
      const bool live = row < M, busy = r0 + 32 * (warp % 4) < M;  // the thread; its warp
      const int tok = live ? row / p.G : 0;
      const uint64_t word = (live ? mask_word(p.mask, sq.q0 + tok, tok) : 0) &
                            (sq.n >= 64 ? ~0ull : (1ull << sq.n) - 1);
      float rc = p.c, m = -INFINITY, l = 0.f, fix = 0.f;
      int vref = 0;
      for (int j = 0; j < n; ++j) {
        if (kPair || (j & 1) == g) {
          wait(C::bSF + g, scount++ & 1);
          tc_fence_after();
          if (threadIdx.x % 128 == 0) {  // the product that read them is done
            mbar_arrive(bar(C::bKE + ks));
            if (j == n - 1) mbar_arrive(bar(C::bQE));
          }
          if (kCodes) wait(C::bMF + ms, mr & 1);
          if (__any_sync(0xffffffffu, busy)) {
            if (kCodes && j == (kPair ? 0 : g)) rc = ss.rc[seg & 1][(kPair ? g * kBigRows : 0) + r];
            const int f = kCodes ? ss.vref[ms] : 0;
            const bool more = j > (kPair ? 0 : 1);  // O holds something
            uint8_t* const meta = smem_ptr + C::kOffMeta + ms * 512;
            if (!kCodes || f != kFar) {
              const float shrink = more && f != vref ? pow2(vref - f) : 1.f;
              vref = f;
              tile(k.tile + j, g, more, ctx, word, rc, shrink, reinterpret_cast<const float4*>(meta), mine, colS, m, l,
                   fix);
            } else {
              tile_far(k.tile + j, g, more, ctx, word, rc, reinterpret_cast<const float*>(meta),
                       reinterpret_cast<const float*>(meta + C::kOffFar - C::kOffMeta), mine, colS, m, l, vref);
            }
          }
          tc_fence_before();
          mbar_arrive(bar(C::bPF + g));
          if (kCodes) {
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::bME + ms));
          }
        }
        if (++ms == C::kMeta) ms = 0, ++mr;
        if (++ks == C::kK) ks = 0;
      }
      // ------------------------------------------------- the segment's end --
      if (!kPair || g == 0) wait(C::bOF + 0, ocount[0]++ & 1);
      if (kPair ? g == 1 : n > 1) wait(C::bOF + 1, ocount[1]++ & 1);
      tc_fence_after();
      close_row(m, l);
      // (the other group has read the last segment's: O is free only when it has)
      ss.ml[g][r] = make_float2(m, l);
      if (kCodes) ss.fend[g][r] = vref;
      else if (!kPair) ss.fix[g][r] = __float2bfloat16(fix);
      asm volatile("bar.sync 2, 256;" ::: "memory");
      const bool poison = aborted() || *(volatile int*)&ss.bad[seg % kRing];
      const uint64_t hid = (uint64_t) * (volatile uint32_t*)&ss.hidden[seg % kRing][1] << 32 |
                           *(volatile uint32_t*)&ss.hidden[seg % kRing][0];
      if (threadIdx.x == 0) {  // the entry of the segment before, which every thread has read
        const int old = (seg + kRing - 1) % kRing;
        ss.bad[old] = 0;
        ss.hidden[old][0] = ss.hidden[old][1] = 0;
      }
      if (__any_sync(0xffffffffu, busy)) {
        const float2 a = kPair ? make_float2(m, l) : ss.ml[0][r];
        const float2 b = kPair ? make_float2(-INFINITY, 0.f) : ss.ml[1][r];
        const float mm = fmaxf(a.x, b.x);
        // a side counts unless it saw nothing: a NaN sum, or an infinite value, survives a weight of 0
        const bool sa = a.x != -INFINITY, sb = b.x != -INFINITY;
        const float wa = sa ? ex2(a.x - mm) : 0.f, wb = sb ? ex2(b.x - mm) : 0.f;
        const float ls = (sa ? wa * a.y : 0.f) + (sb ? wb * b.y : 0.f);
        // O's sum is of the probabilities as the products took them
        float lo = ls;
        if (!kCodes && kPair) lo += fix;
        if (!kCodes && !kPair) lo += wa * __bfloat162float(ss.fix[0][r]) + wb * __bfloat162float(ss.fix[1][r]);
        const float inv = ls != 0.f ? 1.f / lo : 0.f;
        // O's units: 2^(6 - F) of the values, 2^7 of the probabilities (in the sums too)
        const float ua = kCodes ? wa * pow2((kPair ? vref : ss.fend[0][r]) - 6) : wa;
        const float ub = kCodes ? wb * pow2((kPair ? vref : ss.fend[1][r]) - 6) : wb;
        const bool whole = k.tile == 0 && n == k.tiles;
        const int slot = whole ? -1 : 2 * (int)blockIdx.x + !firstp;
        const int64_t at = whole ? (int64_t)(sq.q0 + tok) * p.Hq + h * p.G + (row - tok * p.G) : (int64_t)slot * C::kRows + (row - row0(k));
        if (live && (kPair || g == 0)) {
          float lse = ls != 0.f ? (mm + lg2(ls) - (kCodes ? kPLog2 : 0.f)) * 0.69314718055994531f : -INFINITY;
          if (poison) lse = whole ? NAN : INFINITY;  // +inf makes the join of the pieces a NaN row
          (whole ? p.lse : p.lse_part)[at] = lse;
        }
#pragma unroll 1
        for (int col = kPair ? 0 : g * (D / 2); col < (kPair ? D : (g + 1) * (D / 2)); col += 32) {
          uint32_t xa[32], xb[32];
          tmem_ld_x32(mine + 256 + (kPair ? g * D : 0) + col, xa);
          if (!kPair) tmem_ld_x32(mine + 256 + D + col, xb);
          tmem_ld_wait_x32(xa);
          if (!kPair) tmem_ld_wait_x32(xb);
          float f[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            f[i] = sa ? ua * __uint_as_float(xa[i]) : 0.f;
            if (!kPair) f[i] += sb ? ub * __uint_as_float(xb[i]) : 0.f;
            f[i] = inv != 0.f ? f[i] * inv : 0.f;
            if (poison) f[i] = NAN;
          }
          if (live && hid) add_hidden(f, hid & word, k.b, h, ctx, col);
          if (live && whole) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              *reinterpret_cast<uint4*>(p.o + at * D + col + 8 * i) =
                  make_uint4(rows::pack2(f[8 * i], f[8 * i + 1]), rows::pack2(f[8 * i + 2], f[8 * i + 3]),
                             rows::pack2(f[8 * i + 4], f[8 * i + 5]), rows::pack2(f[8 * i + 6], f[8 * i + 7]));
          } else if (live) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              *reinterpret_cast<float4*>(p.o_part + at * D + col + 4 * i) =
                  make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
          }
        }
      }
      tc_fence_before();
      mbar_arrive(bar(C::bOFree));
      firstp = false;
      ++seg;
    } while (k.next(p, w));
  }

  // What cleaning took out of the products, for a row that sees it.
  __device__ __forceinline__ void add_hidden(float (&f)[32], uint64_t todo, int b, int h, int ctx, int col) {
    while (todo) {
      const int t = __ffsll((long long)todo) - 1;
      todo &= todo - 1;
      const int pos = ctx + t;
      const int id = p.table[(int64_t)b * p.stride + (pos >> p.log_page)];
      if ((unsigned)id >= (unsigned)p.pages) continue;
      const int in = pos & ((1 << p.log_page) - 1);
      const int64_t v = ((((int64_t)id << p.log_page) + in) * p.H + h) * D + col;
      const bool wild = kCodes && !(fabsf(p.vscale[(((int64_t)id * p.H + h) << p.log_page) + in]) < INFINITY);
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        if (kCodes) {
          if (wild || (reinterpret_cast<const uint8_t*>(p.v)[v + i] & 0x7f) == 0x7f) f[i] = NAN;
        } else {
          const float y = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p.v)[v + i]);
          if (!isfinite(y)) f[i] += y;
        }
      }
    }
  }

  // Softmax of this thread's row of key tile t: S from TMEM, P back to it, over S.
  // O (accumulate: it holds something) takes `shrink` and the growth of the maximum.
  __device__ __forceinline__ void tile(int t, int g, bool accumulate, int ctx, uint64_t word, float rc, float shrink,
                                       const float4* meta, uint32_t mine, uint32_t colS, float& m, float& l,
                                       float& fix) {
    const int d = t * kBigTile - ctx;  // new token of the tile's first key
    const bool edge = d + kBigTile > 0;
    float top0 = -INFINITY, top1 = -INFINITY, top2 = -INFINITY, top3 = -INFINITY;
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
      uint32_t x[32];
      float4 f[8];
      tmem_ld_x32(colS + 32 * c, x);
      if (kCodes) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = meta[8 * c + i];
      }
      tmem_ld_wait_x32(x);
      float y[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) y[i] = __uint_as_float(x[i]);
      if (kCodes) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          pmul(y[4 * i], y[4 * i + 1], f[i].x, f[i].y);
          pmul(y[4 * i + 2], y[4 * i + 3], f[i].z, f[i].w);
        }
      }
      if (edge) {
        const int d0 = d + 32 * c;
        const uint32_t vis = d0 <= -32 ? 0xffffffffu
                             : d0 < 0  ? (uint32_t)(word << -d0) | ((1u << -d0) - 1)
                             : d0 < 64 ? (uint32_t)(word >> d0)
                                       : 0u;
#pragma unroll
        for (int i = 0; i < 32; ++i) y[i] = (vis >> i) & 1 ? y[i] : -INFINITY;
      }
#pragma unroll
      for (int i = 0; i < 32; i += 8) {
        top0 = max3f(top0, y[i], y[i + 1]);
        top1 = max3f(top1, y[i + 2], y[i + 3]);
        top2 = max3f(top2, y[i + 4], y[i + 5]);
        top3 = max3f(top3, y[i + 6], y[i + 7]);
      }
      if (kCodes || edge) {
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] = __float_as_uint(y[i]);
        tmem_st_x32(colS + 32 * c, x);
      }
    }
    if (kCodes || edge) tmem_st_wait();
    const float raw = fmaxf(max3f(top0, top1, top2), top3), top = raw * rc;  // rc > 0: -inf stays
    const bool grow = top > m + kLazy;  // also the first finite one
    float alpha = 1.f;
    if (grow) {
      alpha = m == -INFINITY ? 0.f : ex2(m - top);
      m = top;
    }
    if (accumulate && __any_sync(0xffffffffu, grow || shrink != 1.f)) {
      const float f = alpha * shrink;
#pragma unroll 1
      for (int col = 0; col < D; col += 32) {
        uint32_t o[32];
        tmem_ld_x32(mine + 256 + D * g + col, o);
        tmem_ld_wait_x32(o);
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
        tmem_st_x32(mine + 256 + D * g + col, o);
      }
    }
    const float neg = (m == -INFINITY ? 0.f : -m) + (kCodes ? kPLog2 : 0.f);
    if (!kCodes) {  // the largest probability alone is worth it (2^-9 of it, near all of a peaked row's sum)
      const float pm = ex2(fmaf(raw, rc, neg));
      fix = fix * alpha + (__bfloat162float(__float2bfloat16(pm)) - pm);
    }
    float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
      uint32_t x[32], pw[16];
      tmem_ld_x32(colS + 32 * c, x);
      tmem_ld_wait_x32(x);
#pragma unroll
      for (int i = 0; i < 32; i += 4) {
        float e[4];
        pfma(e[0], e[1], __uint_as_float(x[i]), __uint_as_float(x[i + 1]), rc, neg, neg);
        pfma(e[2], e[3], __uint_as_float(x[i + 2]), __uint_as_float(x[i + 3]), rc, neg, neg);
#pragma unroll
        for (int q = 0; q < 4; ++q) e[q] = ex2(e[q]);
        padd(s0, s1, e[0], e[1]);
        padd(s2, s3, e[2], e[3]);
        pw[i / 2] = kCodes ? pack_half(e[0], e[1]) : rows::pack2(e[0], e[1]);
        pw[i / 2 + 1] = kCodes ? pack_half(e[2], e[3]) : rows::pack2(e[2], e[3]);
      }
      tmem_st_x16(colS + 16 * c, pw);
    }
    tmem_st_wait();
    l = l * alpha + ((s0 + s1) + (s2 + s3));
  }

  // tile() where the piece's value scales lie far apart: P takes them (their log2 in
  // `scales`), the row's F is `frame`.  Rare, and its code is kept small.
  __device__ __forceinline__ void tile_far(int t, int g, bool accumulate, int ctx, uint64_t word, float rc,
                                           const float* meta, const float* scales, uint32_t mine, uint32_t colS, float& m,
                                           float& l, int& frame) {
    const int d = t * kBigTile - ctx;
    float top = -INFINITY;
#pragma unroll 1
    for (int c = 0; c < 8; ++c) {  // scores in log2, masked
      uint32_t x[16];
      tmem_ld_x16(colS + 16 * c, x);
      tmem_ld_wait_x16(x);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int j = d + 16 * c + i;  // new token of the key
        const float y = __uint_as_float(x[i]) * meta[16 * c + i] * rc;
        x[i] = __float_as_uint(j < 0 || (j < 64 && sees(word, j)) ? y : -INFINITY);
        top = fmaxf(top, __uint_as_float(x[i]));
      }
      tmem_st_x16(colS + 16 * c, x);
    }
    tmem_st_wait();
    const float was = m;
    float alpha = 1.f;
    if (top > m + kLazy) {
      alpha = m == -INFINITY ? 0.f : ex2(m - top);
      m = top;
    }
    const float zero = m == -INFINITY ? 0.f : m;
    float heavy = -INFINITY, sum = 0.f;  // log2 of the largest p scale
#pragma unroll 1
    for (int c = 0; c < 8; ++c) {
      uint32_t x[16];
      tmem_ld_x16(colS + 16 * c, x);
      tmem_ld_wait_x16(x);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float y = __uint_as_float(x[i]) - zero;
        sum += ex2(y + kPLog2);
        heavy = fmaxf(heavy, y + scales[16 * c + i]);
      }
    }
    l = l * alpha + sum;
    int to = (int)ceilf(fminf(fmaxf(heavy, -100.f), 127.f));
    if (accumulate) {  // what O holds has shrunk with the growth of the maximum
      const float now = was == -INFINITY ? -INFINITY : (float)frame + (was - m);
      to = max(to, (int)ceilf(fmaxf(now, -100.f)));
      const float f = ex2(now - (float)to);
#pragma unroll 1
      for (int col = 0; col < D; col += 16) {
        uint32_t o[16];
        tmem_ld_x16(mine + 256 + D * g + col, o);
        tmem_ld_wait_x16(o);
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
        tmem_st_x16(mine + 256 + D * g + col, o);
      }
    }
    frame = to;
    const float neg = 6.f + kPLog2 - (float)to - zero;  // to fp16(2^(13 - F) p scale)
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
      uint32_t pw[16];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t x[16];
        tmem_ld_x16(colS + 32 * c + 16 * half, x);
        tmem_ld_wait_x16(x);
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          const float* s = scales + 32 * c + 16 * half + i;
          pw[8 * half + i / 2] = pack_half(ex2(__uint_as_float(x[i]) + s[0] + neg), ex2(__uint_as_float(x[i + 1]) + s[1] + neg));
        }
      }
      tmem_st_x16(colS + 16 * c, pw);
    }
    tmem_st_wait();
  }
};

template <int D, bool kCodes, bool kPair>
__global__ void __launch_bounds__(kBigThreads, 1)
tree_tile_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                 const __grid_constant__ Params p, const __grid_constant__ Work w) {
  using C = BigCfg<D, kCodes, kPair>;
  extern __shared__ __align__(1024) uint8_t smem_big[];
  static_assert(C::kBars <= 48, "barriers");
  static_assert(big_smem<D, kCodes, kPair>() <= 227 * 1024, "shared memory");
  BigShared& ss = *reinterpret_cast<BigShared*>(smem_big + C::kOffShared);
  const int warp = threadIdx.x / 32;
  grid_dep_wait();
  grid_dep_launch();
  if (smem_u32(smem_big) & 1023u) {  // the swizzled tiles would be read askew
    if (threadIdx.x == 0) atomicOr(p.err, kTimedOut);
    return;
  }
  Walk k;
  if (!find_place(p, w, blockIdx.x, blockIdx.x == 0 && warp == 0, k)) return;  // the whole CTA
  auto init = [&](int first, int n, int count) {
    for (int i = 0; i < n; ++i) mbar_init(smem_u32(&ss.bars[first + i]), count);
  };
  if (threadIdx.x == 0) {
    init(C::bKF, C::kK, kCodes ? 33 : 1);  // the copies' bytes, and 32 lanes' scales
    constexpr int kBoth = kPair ? 2 : 1;                   // softmax groups that take a key tile
    init(C::bKE, C::kK, kBoth + (kCodes ? 4 : 0));         // they, and the operand warps
    init(C::bVF, C::kV, 1);
    init(C::bVE, C::kV, kCodes ? 4 : 1);   // the operand warps, or the products
    init(C::bRF, C::kReady, 4);
    init(C::bRE, C::kReady, 1);
    init(C::bMF, C::kMeta, 4);
    init(C::bME, C::kMeta, 4 * kBoth);
    init(C::bSF, 2, 1);
    init(C::bPF, 2, 128);
    init(C::bOF, 2, 1);
    init(C::bQF, 1, 128);
    init(C::bQE, 1, kBoth);
    init(C::bOFree, 1, 256);
    init(C::bDrain, 1, 1);
    fence_mbar_init();
    ss.abort = 0;
    for (int i = 0; i < kRing; ++i) ss.bad[i] = ss.hidden[i][0] = ss.hidden[i][1] = 0;
  }
  if (warp == 13) {
    tmem_alloc(smem_u32(&ss.tmem), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  Big<D, kCodes, kPair> big{p, w, ss, smem_big, smem_u32(smem_big), ss.tmem};
  if (warp < 8) {
    regs_inc<kSoftmaxRegs>();
    big.softmax(k, warp / 4);
  } else if (warp < 12) {
    regs_dec<kOperandRegs>();
    big.prepare(k);
  } else {
    regs_dec<kRestRegs>();
    if (warp == 12) {
      big.template produce<true>(k, &map_k);
    } else if (warp == 14) {
      big.template produce<false>(k, &map_v);
    } else if (warp == 13) {
      big.multiply(k);
    }
    __syncwarp();
  }
  if (big.aborted()) {  // let copies in flight land before the CTA leaves
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 1000000ull) {
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 13) {
    tc_fence_after();
    tmem_dealloc(ss.tmem, 512);
  }
}

}  // namespace tree
}  // namespace attn
