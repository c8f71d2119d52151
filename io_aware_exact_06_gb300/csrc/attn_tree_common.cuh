// Attention of the newest tokens of every sequence (one, or a tree of drafted
// ones) over a paged key/value cache: what its kernels share.
//
//   O_i = sum_j softmax_j(scale q_i . k_j) v_j
// over the context and the new tokens that row i sees.  The rows of one key head
// are its G = Hq / H query heads for every new token, row = token * G + head, so
// that keys and values are read once for all of them: per key the products take
// 4 M d flops for M rows against 4 d bytes (bf16) or 2 d bytes (e4m3) of cache.
// Up to 8 rows (16, but for bf16 with d = 128) run on the warp-level products
// (attn_tree_few_kernel.cuh), more on tcgen05 (attn_tree_tile_kernel.cuh);
// attn_tree_work.cuh cuts the work.
//
// With e4m3 codes a score is code . q times the key's scale, and the products with V
// take fp16 operands, whose rounding (2^-11) is below the output's (2^-8); each
// kernel says which of them takes the value's scale.  With a bf16 cache
// probabilities are bf16, the type of V (tensor products take one type): few rows take
// them as the sum of two (2^-16 of each is lost), many rows round once (2^-8) and divide
// O by the sum with the largest of each tile rounded; LSE is of the sum before.
// Sums, maxima and scores are fp32.
#pragma once

#include "attn_rows.cuh"

namespace attn {
namespace tree {

constexpr int kMaxNew = 64;   // bits of a mask word
constexpr float kLazy = 8.f;  // growth (log2) of a row maximum that is worth a rescale
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
  float* o_part;    // the workspace's parts [slots][D]
  float* lse_part;  // [slots]
  int B, total, Hq, H, G;
  int stride, pages, log_page;
  int max_new, max_len;
  float c;  // scale * log2 e (at least the smallest normal float)
  int* err;
};

// Bytes of a key's (or value's) row of one head, and how TMA boxes cut it.
template <int D, bool kCodes>
struct Row {
  static constexpr int kRowBytes = D * (kCodes ? 1 : 2);
  static constexpr int kBox = kRowBytes < 128 ? kRowBytes : 128;  // bytes of a swizzled row
  static constexpr int kHalves = kRowBytes / kBox;
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

// Two bf16 channels of a query, an infinity as a NaN: every score of the row is NaN
// then, and so is the row wherever it sees a key.  (An infinity itself could make all
// its scores -inf, an empty row's, and saturates where a query is split into codes.)
__device__ __forceinline__ uint32_t no_infinity(uint32_t x) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %1;" : "=r"(r) : "r"(x), "r"(0u));  // x 0 + x
  return r;
}
__device__ __forceinline__ uint4 no_infinity(uint4 x) {
  return make_uint4(no_infinity(x.x), no_infinity(x.y), no_infinity(x.z), no_infinity(x.w));
}

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

}  // namespace tree
}  // namespace attn
