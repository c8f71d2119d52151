// Attention of the newest tokens of every sequence (one, or a tree of drafted
// ones) over a paged key/value cache, on the warp-level tensor instructions.
//
// A work item is (sequence b, key head h, range of keys, tile of query rows);
// the rows of one key head are its G = Hq / H query heads for every new token,
// row = token * G + head, so that keys and values are read once for all of
// them.  Per key the products take 4 M d flops for M rows against 4 d bytes
// (bf16) or 2 d bytes (e4m3) of cache: reading the cache bounds the kernel
// while M is small.
//
// One CTA of four compute warps and a producer warp per item.  The producer
// walks the page table and copies 64-key tiles of K and V (and the scales) by
// TMA into a ring of stages; a tile's pages land in one swizzled tile, so
// pages may end anywhere in it.  The compute warps split the tile: kWM row
// groups of 16 rows times 4 / kWM key groups.  Scores and probabilities stay in
// registers (the score fragment of a product is the probability fragment of
// the next), each warp keeps the running maximum and sum of its keys, and the
// key groups merge in shared memory at the end.
//
// Codes become fp16 in registers (exact).  With e4m3 codes the products are
// fp16: a query row is divided by a power of two that brings its largest
// channel into [1, 2), which keeps its bf16 values exact down to 2^-14 of that;
// the key scale multiplies the score and the value scale the probability, and
// the running maximum is taken over log2(probability * value scale), so the
// fp16 operand stays in range whatever the scales.  Its rounding (2^-11) is
// below the output's (2^-8).  With a bf16 cache probabilities are rounded to
// bf16, the type of V (tensor products take one type).
#pragma once

#include "attn_rows.cuh"

namespace attn {
namespace tree {

constexpr int kWarps = 4;                   // compute warps
constexpr int kThreads = 32 * kWarps + 32;  // and the producer
constexpr int kTile = 64;                   // keys per stage
constexpr int kMaxNew = 64;                 // bits of a mask word
constexpr float kLazy = 8.f;                // growth (log2) of a row maximum that is worth a rescale
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr int kTimedOut = 1;  // bit of the library's error word

struct Params {
  const __nv_bfloat16* q;
  int64_t q_ts;
  const int *lens, *cu, *table;
  const int64_t* mask;
  const void* v;  // the cache's values, for non-finite ones a tree hides from some rows
  const float *kscale, *vscale;
  __nv_bfloat16* o;
  float* lse;
  float* o_part;    // [S][total][Hq][D]
  float* lse_part;  // [S][total][Hq]
  int B, total, Hq, H, G;
  int stride, pages, log_page;
  int max_new, max_len;
  int chunk;   // keys per range, a multiple of kTile
  int S;       // ranges of max_len
  int mtiles;  // row tiles of max_new * G rows
  float c;     // scale * log2 e (at least the smallest normal float)
  int* err;
};

// Bytes of a key's (or value's) row of one head, and how TMA boxes cut it.
template <int D, bool kCodes>
struct Row {
  static constexpr int kRowBytes = D * (kCodes ? 1 : 2);
  static constexpr int kBox = kRowBytes < 128 ? kRowBytes : 128;  // bytes of a swizzled row
  static constexpr int kHalves = kRowBytes / kBox;
};

template <int D, bool kCodes>
struct Cfg : Row<D, kCodes> {
  using Row<D, kCodes>::kRowBytes;
  static constexpr int kMatBytes = kTile * kRowBytes;
  static constexpr int kScaleBytes = kCodes ? kTile * 4 : 0;
  static constexpr int kStage = 2 * kMatBytes;
  // about 96 KB of ring, so that two CTAs share an SM; the scales behind it
  static constexpr int kStages = kStage > 24 * 1024 ? 3 : kStage > 12 * 1024 ? 5 : 8;
  static constexpr int kRing = kStages * kStage;
  static constexpr int kSmem = kRing + kStages * 2 * kScaleBytes + 1024;  // and the alignment of the ring
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Byte offset of 16-byte chunk `ch` of row `r` in a tile of kBox-byte rows, as
// TMA's 128-byte and 64-byte swizzles place it.
template <int kBox>
__device__ __forceinline__ uint32_t swz(int r, int ch) {
  return kBox == 128 ? r * 128 + ((ch ^ (r & 7)) << 4) : r * 64 + ((ch ^ ((r >> 1) & 3)) << 4);
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t r;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r) : "r"(a) : "memory");
  return r;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "r"(a)
               : "memory");
  return r;
}
__device__ __forceinline__ float2 lds_f2(uint32_t a) {
  float2 r;
  asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(r.x), "=f"(r.y) : "r"(a) : "memory");
  return r;
}

// acc += A (16 x 16, rows) * B (16 x 8, columns); bf16 or fp16, fp32 sums
template <bool kHalf>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (kHalf)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// The low / high two codes of a word as fp16x2.
__device__ __forceinline__ uint32_t codes_lo(uint32_t w) {
  uint32_t h;
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %1;\n cvt.rn.f16x2.e4m3x2 %0, a;\n}\n" : "=r"(h) : "r"(w));
  return h;
}
__device__ __forceinline__ uint32_t codes_hi(uint32_t w) {
  uint32_t h;
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %1;\n cvt.rn.f16x2.e4m3x2 %0, b;\n}\n" : "=r"(h) : "r"(w));
  return h;
}

__device__ __forceinline__ void compute_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// The rows and keys of a sequence; false if they are not what the caller's
// bounds allow.
struct Seq {
  int q0, n, len;
};
__device__ __forceinline__ bool load_seq(const Params& p, int b, Seq& s) {
  s.q0 = p.cu[b];
  const int end = p.cu[b + 1];
  s.len = p.lens[b];
  s.n = end - s.q0;
  return s.q0 >= 0 && end >= s.q0 && end <= p.total && s.n <= p.max_new && s.len >= s.n &&
         s.len <= p.max_len && s.len <= (int64_t)p.stride << p.log_page;
}

// Whether new token i (mask word `word`) sees new token t.
__device__ __forceinline__ bool sees(uint64_t word, int t) { return (word >> (t & 63)) & 1; }
__device__ __forceinline__ uint64_t mask_word(const int64_t* mask, int64_t tok, int i) {
  return mask ? (uint64_t)mask[tok] : i >= 63 ? ~0ull : (1ull << (i + 1)) - 1;
}

// A row's maximum and sum at the end: NaN scores alone (no maximum) are not an
// empty row, and an infinite score or value scale (no weight is left) makes it NaN.
__device__ __forceinline__ void close_row(float& m, float& l) {
  if (m == INFINITY) l = NAN;
  if (l != l) m = 0.f;
}

// Values of the new tokens' keys in a stage made harmless: rows behind the
// sequence become 0 (they hold whatever the page held), and so does every
// infinity and NaN of a new token, whose row may be hidden from some query rows
// (0 * inf); its bit in `hidden` has the epilogue add it where it is seen.
template <int D, bool kCodes, int kTile, int kThreads>
__device__ __forceinline__ void clean_values(uint8_t* v, int thread, int key0, int ctx, int len, uint32_t* hidden) {
  using C = Row<D, kCodes>;
  constexpr int kWords = C::kRowBytes / 4;
  for (int i = thread; i < kTile * kWords; i += kThreads) {
    const int r = i / kWords, w = i % kWords;
    const int pos = key0 + r;
    if (pos < ctx) continue;
    uint32_t* at = reinterpret_cast<uint32_t*>(
        v + (w * 4 / C::kBox) * (kTile * C::kBox) + swz<C::kBox>(r, (w * 4 % C::kBox) / 16) + (w * 4) % 16);
    if (pos >= len) {
      *at = 0;
      continue;
    }
    const uint32_t x = *at;
    uint32_t bad = 0;
    if (kCodes) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (((x >> (8 * k)) & 0x7fu) == 0x7fu) bad |= 0xffu << (8 * k);
    } else {
      if ((x & 0x7f80u) == 0x7f80u) bad |= 0xffffu;
      if ((x & 0x7f800000u) == 0x7f800000u) bad |= 0xffff0000u;
    }
    if (bad) {
      *at = x & ~bad;
      const int t = pos - ctx;
      atomicOr(hidden + (t >> 5), 1u << (t & 31));
    }
  }
}

// The end of an item: kParts partial results of kRows query rows (part k of row
// r: sums at buf[(k kRows + r) pad], maximum and sum at sm_m, sm_l[k kRows + r])
// merged and written by the 128 compute threads, as the result where the
// sequence has one range, else as this range's part.
template <int D, bool kCodes, int kRows, int kParts>
__device__ __forceinline__ void write_rows(const Params& p, const Seq& sq, int b, int h, int split, int ctx, int row0,
                                           int M, const float* buf, int pad, const float* sm_m, const float* sm_l,
                                           uint64_t hid, bool poison, int thread) {
  const bool only = sq.len <= p.chunk;
  constexpr int kVec = D / 4;  // threads of a row, four columns each
  for (int i = thread; i < kRows * kVec; i += 32 * kWarps) {
    const int r = i / kVec, col = 4 * (i % kVec);
    if (row0 + r >= M) continue;
    const int tok = (row0 + r) / p.G, head = h * p.G + (row0 + r) % p.G;
    float mm = -INFINITY;
#pragma unroll
    for (int k = 0; k < kParts; ++k) mm = fmaxf(mm, sm_m[k * kRows + r]);
    float ls = 0.f, f[4] = {0.f, 0.f, 0.f, 0.f};
    if (mm != -INFINITY) {
#pragma unroll
      for (int k = 0; k < kParts; ++k) {
        const int at = k * kRows + r;
        const float a = sm_m[at] == -INFINITY ? 0.f : ex2(sm_m[at] - mm);
        if (a == 0.f) continue;
        ls = fmaf(sm_l[at], a, ls);
        const float4 x = *reinterpret_cast<const float4*>(buf + at * pad + col);
        f[0] = fmaf(x.x, a, f[0]), f[1] = fmaf(x.y, a, f[1]);
        f[2] = fmaf(x.z, a, f[2]), f[3] = fmaf(x.w, a, f[3]);
      }
    }
    // a row of NaN sums keeps them; one that saw nothing is 0
    const float inv = ls != 0.f ? 1.f / ls : 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) f[k] *= inv;
    float lse = ls != 0.f ? (mm + lg2(ls)) * 0.69314718055994531f : -INFINITY;
    if (hid) {
      uint64_t todo = hid & mask_word(p.mask, sq.q0 + tok, tok);
      while (todo) {
        const int t = __ffsll((long long)todo) - 1;
        todo &= todo - 1;
        const int pos = ctx + t;
        const int id = p.table[(int64_t)b * p.stride + (pos >> p.log_page)];
        if ((unsigned)id >= (unsigned)p.pages) continue;
        const int64_t at = ((((int64_t)id << p.log_page) + (pos & ((1 << p.log_page) - 1))) * p.H + h) * D + col;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (kCodes) {
            const uint8_t x = reinterpret_cast<const uint8_t*>(p.v)[at + k];
            if ((x & 0x7f) == 0x7f) f[k] = NAN;
          } else {
            const float x = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p.v)[at + k]);
            if (!isfinite(x)) f[k] += x;
          }
        }
      }
    }
    if (poison) {  // a NaN row; +inf makes the merge of the ranges one
      f[0] = f[1] = f[2] = f[3] = NAN;
      lse = only ? NAN : INFINITY;
    }
    const int64_t out = (int64_t)(sq.q0 + tok) * p.Hq + head;
    if (only) {
      const uint2 v2 = make_uint2(rows::pack2(f[0], f[1]), rows::pack2(f[2], f[3]));
      *reinterpret_cast<uint2*>(p.o + out * D + col) = v2;
      if (col == 0) p.lse[out] = lse;
    } else {
      const int64_t at = (int64_t)split * p.total * p.Hq + out;
      *reinterpret_cast<float4*>(p.o_part + at * D + col) = make_float4(f[0], f[1], f[2], f[3]);
      if (col == 0) p.lse_part[at] = lse;
    }
  }
}

template <int D, bool kCodes, int kWM>
__global__ void __launch_bounds__(kThreads, 2)
tree_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
            const __grid_constant__ Params p) {
  using C = Cfg<D, kCodes>;
  constexpr int kWK = kWarps / kWM;   // key groups
  constexpr int kKeys = kTile / kWK;  // keys of a warp per tile
  constexpr int kNT = kKeys / 8;      // score fragments
  constexpr int kRows = 16 * kWM;
  constexpr int kQ = D / 16;  // k-steps of the score product
  constexpr int kOT = D / 8;  // output fragments
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[2 * C::kStages];
  __shared__ uint32_t hidden[2];
  __shared__ int flags[2];  // [0] a wait expired, [1] a page outside the cache
  __shared__ float sm_m[kWarps][16], sm_l[kWarps][16];
  const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* ring_ptr = smem_raw + (ring - smem_u32(smem_raw));
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  auto full = [&](int s) { return smem_u32(&bars[s]); };
  auto empty = [&](int s) { return smem_u32(&bars[C::kStages + s]); };
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), kWarps);
    }
    fence_mbar_init();
    hidden[0] = hidden[1] = 0;
    flags[0] = flags[1] = 0;
  }
  __syncthreads();
  grid_dep_wait();
  grid_dep_launch();

  int item = blockIdx.x;
  const int mt = item % p.mtiles;
  item /= p.mtiles;
  const int h = item % p.H;
  item /= p.H;
  const int split = item % p.S;
  const int b = item / p.S;
  Seq sq;
  if (!load_seq(p, b, sq)) {
    if (threadIdx.x == 0) atomicOr(p.err, rows::kBadSeqlens);
    return;
  }
  const int M = sq.n * p.G;
  const int row0 = mt * kRows;
  const int k_lo = split * p.chunk;
  if (row0 >= M || k_lo >= sq.len) return;
  const int k_hi = min(sq.len, k_lo + p.chunk);
  const int ctx = sq.len - sq.n;
  const int tiles = (k_hi - k_lo + kTile - 1) / kTile;
  volatile int* vflags = flags;

  if (warp == kWarps) {
    // ------------------------------------------------------------ producer --
    const int page = 1 << p.log_page;
    const int box = min(page, kTile);  // rows of one copy
    const int per = kTile / box;       // copies per tile (of each matrix)
    const int batch = 32 / per;        // tiles whose page numbers one load fetches
    const int* table = p.table + (int64_t)b * p.stride;
    auto fetch = [&](int tile) {  // this lane's copy of the batch that starts at `tile`
      const int64_t pos = k_lo + (int64_t)tile * kTile + lane * box;
      return pos < k_hi ? table[pos >> p.log_page] : 0;
    };
    int ids = fetch(0);
    for (int t0 = 0; t0 < tiles; t0 += batch) {
      const int next = t0 + batch < tiles ? fetch(t0 + batch) : 0;
      if ((unsigned)ids >= (unsigned)p.pages) {
        flags[1] = 1;
        atomicOr(p.err, rows::kBadIndex);
        ids = 0;
      }
      for (int t = t0; t < min(t0 + batch, tiles); ++t) {
        const int s = t % C::kStages;
        if (t >= C::kStages && !vflags[0] &&
            !mbar_wait(empty(s), ((t / C::kStages) & 1) ^ 1, kWaitNs)) {
          vflags[0] = 1;
          atomicOr(p.err, kTimedOut);
        }
        __syncwarp();
        const int id = __shfl_sync(0xffffffffu, ids, (t - t0) * per + lane % per);
        if (__any_sync(0xffffffffu, vflags[0])) continue;  // nothing more is copied
        const int key0 = k_lo + t * kTile;
        const int n = min(per, (k_hi - key0 + box - 1) / box);
        if (lane == 0) mbar_arrive_expect_tx(full(s), n * box * 2 * (C::kRowBytes + (kCodes ? 4 : 0)));
        __syncwarp();
        if (lane < n) {
          const int in = (key0 + lane * box) & (page - 1);
          const int row = (id << p.log_page) + in;
          const uint32_t dst = ring + s * C::kStage + lane * box * C::kBox;
          constexpr int kElems = kCodes ? C::kBox : C::kBox / 2;
#pragma unroll
          for (int f = 0; f < C::kHalves; ++f) {
            tma_load_3d(dst + f * kTile * C::kBox, &map_k, full(s), f * kElems, h, row);
            tma_load_3d(dst + C::kMatBytes + f * kTile * C::kBox, &map_v, full(s), f * kElems, h, row);
          }
          if (kCodes) {
            const int64_t at = (((int64_t)id * p.H + h) << p.log_page) + in;
            const uint32_t sd = ring + C::kRing + s * 2 * C::kScaleBytes + lane * box * 4;
            bulk_load(sd, p.kscale + at, box * 4, full(s));
            bulk_load(sd + C::kScaleBytes, p.vscale + at, box * 4, full(s));
          }
        }
      }
      ids = next;
    }
    __syncwarp();
    if (vflags[0]) {  // let copies in flight land before the CTA leaves
      const uint64_t t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < 1000000ull) {
      }
    }
  } else {
    // ------------------------------------------------------------- compute --
    const int rg = warp % kWM, kg = warp / kWM;
    const int c = lane % 4, n = lane / 4;
    const bool active = row0 + rg * 16 < M;  // the whole warp
    const __nv_bfloat16* qrow[2];
    bool live[2];
    uint64_t word[2];
    float rc[2] = {p.c, p.c};  // factor of a raw score (log2 units)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = row0 + rg * 16 + n + 8 * i;
      live[i] = r < M;
      const int tok = live[i] ? r / p.G : 0, g = live[i] ? r % p.G : 0;
      qrow[i] = p.q + (int64_t)(sq.q0 + tok) * p.q_ts + (int64_t)(h * p.G + g) * D;
      word[i] = live[i] ? mask_word(p.mask, sq.q0 + tok, tok) : 0;
    }
    uint32_t qa[kQ][4];
    if (active) {
      if (!kCodes) {
#pragma unroll
        for (int s = 0; s < kQ; ++s)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            qa[s][i] = live[i & 1] ? *reinterpret_cast<const uint32_t*>(qrow[i & 1] + 16 * s + 2 * c + 8 * (i >> 1)) : 0u;
      } else {
        // lane c's channels of k-step s: the four that its 16 bytes of a key's
        // codes (chunk kHH c + s / 4) hold at 4 (s % 4)
        constexpr int kHH = D / 64;
        float amax[2] = {0.f, 0.f};
        uint2 raw[kQ][2];
#pragma unroll
        for (int s = 0; s < kQ; ++s)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int ch = 16 * (kHH * c + s / 4) + 4 * (s % 4);
            raw[s][i] = live[i] ? *reinterpret_cast<const uint2*>(qrow[i] + ch) : make_uint2(0, 0);
            const uint32_t u[2] = {raw[s][i].x, raw[s][i].y};
#pragma unroll
            for (int k = 0; k < 2; ++k)
              amax[i] = fmaxf(amax[i], fmaxf(fabsf(__uint_as_float(u[k] << 16)),
                                             fabsf(__uint_as_float(u[k] & 0xffff0000u))));
          }
        float down[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          amax[i] = fmaxf(amax[i], __shfl_xor_sync(0xffffffffu, amax[i], 1));
          amax[i] = fmaxf(amax[i], __shfl_xor_sync(0xffffffffu, amax[i], 2));
          int e = (int)(__float_as_uint(amax[i]) >> 23) - 127;
          e = amax[i] == 0.f ? 0 : min(max(e, -126), 126);
          down[i] = __uint_as_float((uint32_t)(127 - e) << 23);
          rc[i] = p.c * __uint_as_float((uint32_t)(127 + e) << 23);
        }
#pragma unroll
        for (int s = 0; s < kQ; ++s)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t u[2] = {raw[s][i].x, raw[s][i].y};
#pragma unroll
            for (int k = 0; k < 2; ++k)
              qa[s][2 * k + i] = pack_half(__uint_as_float(u[k] << 16) * down[i],
                                           __uint_as_float(u[k] & 0xffff0000u) * down[i]);
          }
      }
    }
    float o[kOT][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int t = 0; t < kOT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[t][i] = 0.f;

    for (int t = 0; t < tiles; ++t) {
      const int s = t % C::kStages;
      if (!vflags[0] && !mbar_wait(full(s), (t / C::kStages) & 1, kWaitNs)) {
        vflags[0] = 1;
        atomicOr(p.err, kTimedOut);
      }
      __syncwarp();
      const int key0 = k_lo + t * kTile;
      const uint32_t kt = ring + s * C::kStage, vt = kt + C::kMatBytes;
      const uint32_t ks = ring + C::kRing + s * 2 * C::kScaleBytes, vs = ks + C::kScaleBytes;
      const bool edge = key0 + kTile > ctx;
      if (edge) {  // the same for every warp
        clean_values<D, kCodes, kTile, 32 * kWarps>(ring_ptr + s * C::kStage + C::kMatBytes, threadIdx.x, key0, ctx,
                                                    sq.len, hidden);
        compute_sync();
      }
      if (active) {
        float sc[kNT][4];
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) {
          sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.f;
          const int key = kg * kKeys + nt * 8;
          if (!kCodes) {
#pragma unroll
            for (int q2 = 0; q2 < kQ; q2 += 2) {
              uint32_t kb[4];
              const int ch = 2 * q2 + lane / 8;  // 16-byte chunk of the key row
              ldsm4(kb, kt + (ch / 8) * (kTile * 128) + swz<128>(key + lane % 8, ch % 8));
              mma<false>(sc[nt], qa[q2], kb[0], kb[1]);
              mma<false>(sc[nt], qa[q2 + 1], kb[2], kb[3]);
            }
          } else {
            constexpr int kHH = D / 64;
#pragma unroll
            for (int hh = 0; hh < kHH; ++hh) {
              const uint4 w = lds128(kt + swz<C::kBox>(key + n, kHH * c + hh));
              mma<true>(sc[nt], qa[4 * hh], codes_lo(w.x), codes_hi(w.x));
              mma<true>(sc[nt], qa[4 * hh + 1], codes_lo(w.y), codes_hi(w.y));
              mma<true>(sc[nt], qa[4 * hh + 2], codes_lo(w.z), codes_hi(w.z));
              mma<true>(sc[nt], qa[4 * hh + 3], codes_lo(w.w), codes_hi(w.w));
            }
          }
        }
        // log2 scores, masked; their maxima (with the value scale for codes)
        float2 vsc[kNT];
        float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) {
          const int key = kg * kKeys + nt * 8 + 2 * c;
          float2 ksc = make_float2(1.f, 1.f), lg = make_float2(0.f, 0.f);
          if (kCodes) {
            ksc = lds_f2(ks + key * 4);
            vsc[nt] = lds_f2(vs + key * 4);
            lg = make_float2(lg2(fmaxf(vsc[nt].x, 0x1p-64f)), lg2(fmaxf(vsc[nt].y, 0x1p-64f)));
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = i >> 1;
            float x = sc[nt][i] * rc[r];
            if (kCodes) x *= (i & 1) ? ksc.y : ksc.x;
            if (edge) {
              const int d = key0 + key + (i & 1) - ctx;
              if (d >= sq.n || (d >= 0 && !sees(word[r], d))) x = -INFINITY;
            }
            sc[nt][i] = x;
            // a masked score stays -inf whatever the scale of its key holds
            top[r] = fmaxf(top[r], kCodes && x != -INFINITY ? x + ((i & 1) ? lg.y : lg.x) : x);
          }
        }
        float ref[2];
        bool grow = false;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 1));
          top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 2));
          grow |= top[r] > m[r] + kLazy;  // also the first finite one: m is -inf
        }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float mn = fmaxf(m[r], top[r]);
            const float a = m[r] == -INFINITY ? 0.f : ex2(m[r] - mn);
            m[r] = mn;
            l[r] *= a;
#pragma unroll
            for (int ot = 0; ot < kOT; ++ot) {
              o[ot][2 * r] *= a;
              o[ot][2 * r + 1] *= a;
            }
          }
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) ref[r] = m[r] == -INFINITY ? 0.f : m[r];
        uint32_t pa[kNT / 2][4];
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) {
          float w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float pr = ex2(sc[nt][i] - ref[i >> 1]);
            l[i >> 1] += pr;
            w[i] = pr;
            if (kCodes) w[i] = sc[nt][i] == -INFINITY ? 0.f : pr * ((i & 1) ? vsc[nt].y : vsc[nt].x);
          }
          pa[nt / 2][2 * (nt & 1)] = kCodes ? pack_half(w[0], w[1]) : rows::pack2(w[0], w[1]);
          pa[nt / 2][2 * (nt & 1) + 1] = kCodes ? pack_half(w[2], w[3]) : rows::pack2(w[2], w[3]);
        }
#pragma unroll
        for (int k2 = 0; k2 < kNT / 2; ++k2) {
          const int key = kg * kKeys + k2 * 16;
          if (!kCodes) {
#pragma unroll
            for (int o2 = 0; o2 < kOT; o2 += 2) {
              uint32_t vb[4];
              const int ch = o2 + lane / 16;
              ldsm4t(vb, vt + (ch / 8) * (kTile * 128) + swz<128>(key + lane % 16, ch % 8));
              mma<false>(o[o2], pa[k2], vb[0], vb[1]);
              mma<false>(o[o2 + 1], pa[k2], vb[2], vb[3]);
            }
          } else {
            // lane (n, c): four neighbouring columns of keys 2c, 2c+1, 2c+8, 2c+9;
            // fragment 4 g + j takes column 32 g + 4 n + j
#pragma unroll
            for (int g = 0; g < D / 32; ++g) {
              const int ch = 2 * g + n / 4, in = 4 * (n % 4);
              const uint32_t w0 = lds32(vt + swz<C::kBox>(key + 2 * c, ch) + in);
              const uint32_t w1 = lds32(vt + swz<C::kBox>(key + 2 * c + 1, ch) + in);
              const uint32_t w2 = lds32(vt + swz<C::kBox>(key + 2 * c + 8, ch) + in);
              const uint32_t w3 = lds32(vt + swz<C::kBox>(key + 2 * c + 9, ch) + in);
              const uint32_t a01 = __byte_perm(w0, w1, 0x5140), b01 = __byte_perm(w0, w1, 0x7362);
              const uint32_t a23 = __byte_perm(w2, w3, 0x5140), b23 = __byte_perm(w2, w3, 0x7362);
              mma<true>(o[4 * g], pa[k2], codes_lo(a01), codes_lo(a23));
              mma<true>(o[4 * g + 1], pa[k2], codes_hi(a01), codes_hi(a23));
              mma<true>(o[4 * g + 2], pa[k2], codes_lo(b01), codes_lo(b23));
              mma<true>(o[4 * g + 3], pa[k2], codes_hi(b01), codes_hi(b23));
            }
          }
        }
      }
      if (edge) fence_async_smem();  // this thread wrote to the stage; a copy may follow
      __syncwarp();
      if (lane == 0) mbar_arrive(empty(s));
    }

    // ------------------------------------------------ merge the key groups --
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
      close_row(m[r], l[r]);
      if (c == 0) {
        sm_m[warp][n + 8 * r] = active ? m[r] : -INFINITY;
        sm_l[warp][n + 8 * r] = l[r];
      }
    }
    compute_sync();  // every warp is through with the ring
    constexpr int kPad = D + 4;
    float* buf = reinterpret_cast<float*>(ring_ptr) + warp * 16 * kPad;
    if (active) {
#pragma unroll
      for (int ot = 0; ot < kOT; ++ot)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int col = kCodes ? 32 * (ot / 4) + 8 * c + 4 * (i & 1) + ot % 4 : 8 * ot + 2 * c + (i & 1);
          buf[(n + 8 * (i >> 1)) * kPad + col] = o[ot][i];
        }
    }
    compute_sync();
    write_rows<D, kCodes, kRows, kWK>(p, sq, b, h, split, ctx, row0, M, reinterpret_cast<const float*>(ring_ptr), kPad,
                                      &sm_m[0][0], &sm_l[0][0], (uint64_t)hidden[1] << 32 | hidden[0],
                                      vflags[0] || vflags[1], threadIdx.x);
  }
  __syncthreads();
}

// Ranges of a row joined: weights e^(LSE_s - max), as for split keys elsewhere
// in the library.  One warp per (new token, query head); lanes first take the
// ranges' LSE, then d / 32 columns each.  Rows of a sequence with one range (or
// with lengths that the attention refused) are left as they are.
template <int D>
__global__ void __launch_bounds__(256) tree_combine_kernel(const __grid_constant__ Params p) {
  constexpr int kPer = D / 32;
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x % 32;
  const int64_t rowi = (int64_t)blockIdx.x * 8 + threadIdx.x / 32;
  if (rowi >= (int64_t)p.total * p.Hq) return;
  const int t = (int)(rowi / p.Hq);
  const int b = rows::find_sequence(p.cu, p.B, t);
  if (b >= p.B) return;
  Seq sq;
  if (!load_seq(p, b, sq) || t < sq.q0 || t >= sq.q0 + sq.n) return;
  const int S = (int)(((int64_t)sq.len + p.chunk - 1) / p.chunk);
  if (S <= 1) return;
  const int64_t step = (int64_t)p.total * p.Hq;
  float top = -INFINITY;
  for (int s = lane; s < S; s += 32) top = fmaxf(top, p.lse_part[s * step + rowi]);
#pragma unroll
  for (int off = 16; off; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
  bool nan = false;  // fmaxf passes a NaN over
  float acc[kPer], sum = 0.f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) acc[i] = 0.f;
  for (int s = 0; s < S; ++s) {
    const float ls = p.lse_part[s * step + rowi];
    nan |= ls != ls;
    if (ls == -INFINITY) continue;
    const float w = __expf(ls - top);
    sum += w;
    const float* src = p.o_part + (s * step + rowi) * D + lane * kPer;
#pragma unroll
    for (int i = 0; i < kPer; ++i) acc[i] = fmaf(w, src[i], acc[i]);
  }
  if (nan) sum = NAN;
  const float inv = sum != 0.f ? 1.f / sum : 0.f;
  __nv_bfloat16* dst = p.o + rowi * D + lane * kPer;
#pragma unroll
  for (int i = 0; i < kPer; i += 2)
    *reinterpret_cast<uint32_t*>(dst + i) = rows::pack2(acc[i] * inv, acc[i + 1] * inv);
  if (lane == 0) p.lse[rowi] = sum != 0.f ? top + __logf(sum) : -INFINITY;
}

}  // namespace tree
}  // namespace attn
