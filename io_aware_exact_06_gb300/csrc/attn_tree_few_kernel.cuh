// Attention of the newest tokens over the paged cache for few query rows of a key
// head, on the warp-level tensor instructions.  Codes become fp16 in registers; a
// query row is divided by a power of two that brings its largest channel into
// [1, 2), which keeps its bf16 values exact in fp16 down to 2^-14 of that.  A
// probability takes its value's scale before it meets the codes of V; the running
// maximum is taken over log2(probability * value scale), so that this fp16 operand
// stays in range whatever the scales.  Over a bf16 cache a probability is two bf16,
// its rounding and what that leaves, each with its product with V (12 drafts 51.4 ->
// 52.4 us; 0.00227 -> 0.00166 off fp64, which is the rounding of O alone).
#pragma once

#include "attn_tree_work.cuh"

namespace attn {
namespace tree {

// Up to 8 kNT rows (one token, or a few drafts, of a key head's group): keys
// take the 16-row side of the products and queries the 8-column side,
//   S^T = K Q^T,   O^T += V^T P^T,
// so a fragment holds 8 queries, not 16, and a warp takes whole tiles of one
// head: no key or value is read or converted twice.  P^T is the score fragment
// transposed in registers (movmatrix).
//
// Every warp works alone: it finds its place in the line, copies its tiles by
// TMA into stages of its own (the copies of a later tile go out as soon as a
// stage is free, across the ends of segments), keeps its softmax and writes its
// pieces; the CTA is only where four warps live.  A segment is a
// group of `heads` neighbouring heads, one to a warp, which so read neighbouring
// lines of the cache's token rows at about the same time: with 128-byte head
// rows (e4m3, d = 128) four warps on four heads read 512 contiguous bytes.
// (One head to a CTA, its tiles dealt to the warps: 4.4 TB/s on 64 ragged
// sequences of 8 heads against 5.4 TB/s on the same bytes with one head.  A
// producer warp for the CTA instead spent about 1000 cycles on a 32-key tile's
// issue, against 365 that HBM needs for the tiles of twelve warps.)
constexpr int kWarps = 4;     // of a CTA
constexpr int kFewTile = 32;  // keys per stage
constexpr int kLogFewTile = 5;
constexpr int kFewThreads = 32 * kWarps;
// CTAs per SM.  Two leave a lane 255 registers and DRAM fewer streams; d = 64 codes
// are bound by their arithmetic and want three (64 ragged sequences of up to 8192
// keys, one token, 32 + 8 heads, two : three CTAs: d = 128 e4m3 144 : 145 us, bf16
// 247 : 246, d = 64 bf16 132 : 136, e4m3 142 : 104).
__host__ __device__ constexpr int few_ctas(int d, bool codes) { return d == 64 && codes ? 3 : 2; }
// For the registers: d = 128 bf16 does better held to three CTAs' where sequences are
// short (one token for four of them 12.0 against 12.8 us, the long batch 243 against
// 241), e4m3 does not (184 : 143).
__host__ __device__ constexpr int few_bound(int d, bool codes) { return (d == 128) != codes ? 3 : 2; }
constexpr int kFewRing = 16384;  // bytes of a warp's stages (24576: d = 64 bf16 135 us against 129)

template <int D, bool kCodes, int kNT>
struct FewCfg : Row<D, kCodes> {
  using Row<D, kCodes>::kRowBytes;
  static constexpr int kMatBytes = kFewTile * kRowBytes;
  static constexpr int kScaleBytes = kCodes ? kFewTile * 4 : 0;
  static constexpr int kStage = 2 * kMatBytes;
  static constexpr int kOwn = kFewRing / kStage < 3 ? kFewRing / kStage : 3;  // stages of a warp
  static constexpr int kStages = kOwn * kWarps;
  static constexpr int kRing = kStages * kStage;
  static constexpr int kTurn = 32;  // columns of the output turned to rows at a time
  static constexpr int kPad = kTurn + 4;
  static constexpr int kTurnBytes = kWarps * 8 * kNT * kPad * 4;
  static constexpr int kSmem = kRing + kStages * 2 * kScaleBytes + kTurnBytes + 1024;
};

__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

template <int D, bool kCodes, int kNT>
__global__ void __launch_bounds__(kFewThreads, few_bound(D, kCodes))
tree_few_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                const __grid_constant__ Params p, const __grid_constant__ Work w) {
  using C = FewCfg<D, kCodes, kNT>;
  constexpr int kQ = D / 16;  // k-steps of the score product
  constexpr int kMT = D / 16;  // 16-column tiles of the output
  constexpr int kHH = D / 64;  // 16-byte chunks of a lane's codes
  constexpr int kRows = 8 * kNT;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[C::kStages];
  __shared__ uint32_t hidden_all[kWarps][2];
  __shared__ float sm_m[kWarps][kRows], sm_l[kWarps][kRows];
  const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* ring_ptr = smem_raw + (ring - smem_u32(smem_raw));
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  float* turn = reinterpret_cast<float*>(ring_ptr + C::kRing + C::kStages * 2 * C::kScaleBytes) +
                warp * kRows * C::kPad;
  uint32_t* hidden = hidden_all[warp];
  auto full = [&](int s) { return smem_u32(&bars[s]); };
  if (lane == 0) {
    for (int s = 0; s < C::kOwn; ++s)
      mbar_init(full(warp * C::kOwn + s), kCodes ? 17 : 1);  // the copies' bytes, and 16 lanes' scales
    fence_mbar_init();
    hidden[0] = hidden[1] = 0;
  }
  __syncwarp();
  grid_dep_wait();
  grid_dep_launch();
  const int units = kWarps / w.heads;  // of the CTA
  const int unit = blockIdx.x * units + warp / w.heads, sub = warp % w.heads;
  Walk wk;
  if (!find_place(p, w, unit, threadIdx.x < 32 && blockIdx.x == 0, wk)) return;
  bool expired = false;  // a wait ran out: nothing more is copied, the rows come out as NaN

  // ------------------------------------------------------- the warp's copies --
  const int page = 1 << p.log_page;
  const int box = min(page, kFewTile);  // rows of one copy
  const int per = kFewTile / box;       // copies per tile (of each matrix)
  const int batch = 32 / per;           // tiles whose page numbers one load fetches
  Walk fw = wk;                         // runs ahead of wk
  int f_tile, f_end, f_at = 0, f_head, f_ids, f_next, f_stage = 0;
  bool f_more = true;
  uint32_t bad = 0;  // bit s: the tile in stage s reads a page outside the cache
  auto fetch = [&](int tile) {  // this lane's copy of the `batch` tiles from `tile` on
    const int64_t pos = (int64_t)tile * kFewTile + lane * box;
    return pos < fw.s.len ? p.table[(int64_t)fw.b * p.stride + (pos >> p.log_page)] : 0;
  };
  auto enter = [&]() {
    f_tile = fw.tile;
    f_end = fw.tile + fw.piece();
    f_head = fw.seg / (fw.segs / (p.H / w.heads)) * w.heads + sub;
    f_at = 0;
    f_ids = fetch(f_tile);
    f_next = fetch(f_tile + batch);
  };
  auto feed = [&]() {  // copies of the warp's next tile into its stage f_stage
    if (f_more && f_tile >= f_end) {
      f_more = fw.next(p, w);
      if (f_more) enter();
    }
    if (!f_more || expired) return;
    const int s = warp * C::kOwn + f_stage, key0 = f_tile * kFewTile, len = fw.s.len;
    int id = __shfl_sync(0xffffffffu, f_ids, f_at * per + lane % per);
    const bool wrong = (unsigned)id >= (unsigned)p.pages;
    if (wrong) id = 0;
    const int n = min(per, (len - key0 + box - 1) / box);
    bad &= ~(1u << f_stage);
    if (__any_sync(0xffffffffu, wrong)) {
      bad |= 1u << f_stage;
      if (lane == 0) atomicOr(p.err, rows::kBadIndex);
    }
    if (lane == 0) mbar_arrive_expect_tx(full(s), n * box * 2 * C::kRowBytes);
    __syncwarp();
    if (lane < n) {
      const int row = (id << p.log_page) + ((key0 + lane * box) & (page - 1));
      const uint32_t dst = ring + s * C::kStage + lane * box * C::kBox;
      constexpr int kElems = kCodes ? C::kBox : C::kBox / 2;
#pragma unroll
      for (int f = 0; f < C::kHalves; ++f) {
        tma_load_3d(dst + f * kFewTile * C::kBox, &map_k, full(s), f * kElems, f_head, row);
        tma_load_3d(dst + C::kMatBytes + f * kFewTile * C::kBox, &map_v, full(s), f * kElems, f_head, row);
      }
    }
    if (kCodes) {  // lanes 0-7: four key scales each, 8-15: value scales
      const int key = (lane & 7) * 4;
      const int sid = __shfl_sync(0xffffffffu, id, per == 1 ? 0 : key / 16);
      if (lane < 16) {
        if (key0 + key < len) {
          const int64_t at = (((int64_t)sid * p.H + f_head) << p.log_page) + ((key0 + key) & (page - 1));
          cp_async16(ring + C::kRing + (2 * s + lane / 8) * C::kScaleBytes + key * 4,
                     (lane < 8 ? p.kscale : p.vscale) + at);
        }
        cp_async_arrive(full(s));
      }
    }
    if (++f_stage == C::kOwn) f_stage = 0;
    ++f_tile;
    if (++f_at == batch) {
      f_at = 0;
      f_ids = f_next;
      f_next = fetch(f_tile + batch);
    }
  };
  enter();
#pragma unroll 1
  for (int i = 0; i < C::kOwn; ++i) feed();

  // --------------------------------------------------------------- compute --
  const int c = lane % 4, n = lane / 4;
  int stage = 0, parity = 0;
  bool first = true;
  do {
    const Seq sq = wk.s;
    const int M = sq.n * p.G, ctx = sq.len - sq.n;
    const int mtiles = wk.segs / (p.H / w.heads), group = wk.seg / mtiles;
    const int h = group * w.heads + sub, row0 = (wk.seg - group * mtiles) * kRows;
    const int t_begin = wk.tile, t_end = wk.tile + wk.piece();
    bool poison = false;
    uint64_t word[kNT][2];  // masks and score factors (log2 units) of queries 2c, 2c + 1
    float rc[kNT][2];
    uint32_t qb[kNT][kQ][2];  // query n's channels
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
      const int r = row0 + 8 * nt + n;
      const bool live = r < M;
      const int tok = live ? r / p.G : 0, g = live ? r % p.G : 0;
      const __nv_bfloat16* q = p.q + (int64_t)(sq.q0 + tok) * p.q_ts + (int64_t)(h * p.G + g) * D;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int ri = row0 + 8 * nt + 2 * c + i;
        word[nt][i] = ri < M ? mask_word(p.mask, sq.q0 + ri / p.G, ri / p.G) : 0;
        rc[nt][i] = p.c;
      }
      if (!kCodes) {
#pragma unroll
        for (int s = 0; s < kQ; ++s)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            qb[nt][s][i] = live ? no_infinity(*reinterpret_cast<const uint32_t*>(q + 16 * s + 2 * c + 8 * i)) : 0u;
      } else {
        // lane c's channels of k-step s: the four that its 16 bytes of a key's
        // codes (chunk kHH c + s / 4) hold at 4 (s % 4)
        float amax = 0.f;
#pragma unroll
        for (int s = 0; s < kQ; ++s) {
          const int ch = 16 * (kHH * c + s / 4) + 4 * (s % 4);
          const uint2 raw = live ? *reinterpret_cast<const uint2*>(q + ch) : make_uint2(0, 0);
          qb[nt][s][0] = no_infinity(raw.x), qb[nt][s][1] = no_infinity(raw.y);
#pragma unroll
          for (int k = 0; k < 2; ++k)
            amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(qb[nt][s][k] << 16)),
                                     fabsf(__uint_as_float(qb[nt][s][k] & 0xffff0000u))));
        }
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        int e = (int)(__float_as_uint(amax) >> 23) - 127;
        e = amax == 0.f ? 0 : min(max(e, -126), 126);
        const float down = __uint_as_float((uint32_t)(127 - e) << 23);
        const float up = p.c * __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
        for (int i = 0; i < 2; ++i) rc[nt][i] = __shfl_sync(0xffffffffu, up, 4 * (2 * c + i));
#pragma unroll
        for (int s = 0; s < kQ; ++s)
#pragma unroll
          for (int k = 0; k < 2; ++k)
            qb[nt][s][k] = pack_half(__uint_as_float(qb[nt][s][k] << 16) * down,
                                     __uint_as_float(qb[nt][s][k] & 0xffff0000u) * down);
      }
    }
    float o[kMT][kNT][4], m[kNT][2], l[kNT][2];
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[mt][nt][i] = 0.f;
    }

    for (int t = t_begin; t < t_end; ++t) {
      const int mine = warp * C::kOwn + stage;
      if (!expired) {
        expired = __any_sync(0xffffffffu, !mbar_wait(full(mine), parity, kWaitNs));
        if (expired && lane == 0) atomicOr(p.err, kTimedOut);
      }
      poison |= bad >> stage & 1;
      const int key0 = t * kFewTile;
      const uint32_t kt = ring + mine * C::kStage, vt = kt + C::kMatBytes;
      const uint32_t ks = ring + C::kRing + mine * 2 * C::kScaleBytes, vs = ks + C::kScaleBytes;
      const bool edge = key0 + kFewTile > ctx;
      if (edge) {
        clean_values<D, kCodes, kFewTile, 32>(ring_ptr + mine * C::kStage + C::kMatBytes, lane, key0, ctx, sq.len,
                                              hidden);
        __syncwarp();
      }
      float sc[2][kNT][4];  // [16-key half][query tile]: keys n, n + 8 x queries 2c, 2c + 1
#pragma unroll
      for (int ksub = 0; ksub < 2; ++ksub) {
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) sc[ksub][nt][0] = sc[ksub][nt][1] = sc[ksub][nt][2] = sc[ksub][nt][3] = 0.f;
        if (!kCodes) {
#pragma unroll
          for (int q2 = 0; q2 < kQ; ++q2) {
            uint32_t ka[4];
            const int ch = 2 * q2 + lane / 16;  // 16-byte chunk of the key row
            ldsm4(ka, kt + (ch / 8) * (kFewTile * 128) + swz<128>(16 * ksub + lane % 16, ch % 8));
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt) mma<false>(sc[ksub][nt], ka, qb[nt][q2][0], qb[nt][q2][1]);
          }
        } else {
#pragma unroll
          for (int hh = 0; hh < kHH; ++hh) {
            const uint4 w0 = lds128(kt + swz<C::kBox>(16 * ksub + n, kHH * c + hh));
            const uint4 w1 = lds128(kt + swz<C::kBox>(16 * ksub + n + 8, kHH * c + hh));
            const uint32_t x0[4] = {w0.x, w0.y, w0.z, w0.w}, x1[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t ka[4] = {codes_lo(x0[j]), codes_lo(x1[j]), codes_hi(x0[j]), codes_hi(x1[j])};
#pragma unroll
              for (int nt = 0; nt < kNT; ++nt)
                mma<true>(sc[ksub][nt], ka, qb[nt][4 * hh + j][0], qb[nt][4 * hh + j][1]);
            }
          }
        }
      }
      // log2 scores, masked; their maxima (with the value scale for codes)
      float vsc[2][2];
      float top[kNT][2];
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt) top[nt][0] = top[nt][1] = -INFINITY;
#pragma unroll
      for (int ksub = 0; ksub < 2; ++ksub)
#pragma unroll
        for (int kh = 0; kh < 2; ++kh) {
          const int key = 16 * ksub + 8 * kh + n;
          float ksc = 1.f, lg = 0.f;
          if (kCodes) {
            ksc = __uint_as_float(lds32(ks + key * 4));
            vsc[ksub][kh] = __uint_as_float(lds32(vs + key * 4));
            lg = lg2(fmaxf(vsc[ksub][kh], 0x1p-64f));
          }
#pragma unroll
          for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float x = sc[ksub][nt][2 * kh + i] * rc[nt][i];
              if (kCodes) x *= ksc;
              if (edge) {
                const int d = key0 + key - ctx;
                if (d >= sq.n || (d >= 0 && !sees(word[nt][i], d))) x = -INFINITY;
              }
              sc[ksub][nt][2 * kh + i] = x;
              // a masked score stays -inf whatever the scale of its key holds
              top[nt][i] = fmaxf(top[nt][i], kCodes && x != -INFINITY ? x + lg : x);
            }
        }
      bool grow = false;
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
          for (int off = 4; off < 32; off <<= 1)
            top[nt][i] = fmaxf(top[nt][i], __shfl_xor_sync(0xffffffffu, top[nt][i], off));
          grow |= top[nt][i] > m[nt][i] + kLazy;  // also the first finite one: m is -inf
        }
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float mn = fmaxf(m[nt][i], top[nt][i]);
            const float a = m[nt][i] == -INFINITY ? 0.f : ex2(m[nt][i] - mn);
            m[nt][i] = mn;
            l[nt][i] *= a;
#pragma unroll
            for (int mt = 0; mt < kMT; ++mt) {
              o[mt][nt][i] *= a;
              o[mt][nt][2 + i] *= a;
            }
          }
      }
#pragma unroll
      for (int ksub = 0; ksub < 2; ++ksub) {
        uint32_t pb[kNT][2], pl[kNT][2];
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
          for (int kh = 0; kh < 2; ++kh) {
            float w[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float x = sc[ksub][nt][2 * kh + i];
              const float pr = ex2(x - (m[nt][i] == -INFINITY ? 0.f : m[nt][i]));
              l[nt][i] += pr;
              w[i] = kCodes ? (x == -INFINITY ? 0.f : pr * vsc[ksub][kh]) : pr;
            }
            const uint32_t both = kCodes ? pack_half(w[0], w[1]) : rows::pack2(w[0], w[1]);
            pb[nt][kh] = transposed(both);
            if (!kCodes)
              pl[nt][kh] = transposed(rows::pack2(w[0] - __uint_as_float(both << 16), w[1] - __uint_as_float(both & 0xffff0000u)));
          }
        if (!kCodes) {
#pragma unroll
          for (int mt = 0; mt < kMT; ++mt) {
            uint32_t va[4];
            const int ch = 2 * mt + ((lane / 8) & 1);
            ldsm4t(va, vt + (ch / 8) * (kFewTile * 128) + swz<128>(16 * ksub + lane % 8 + 8 * (lane / 16), ch % 8));
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt) {
              mma<false>(o[mt][nt], va, pb[nt][0], pb[nt][1]);
              mma<false>(o[mt][nt], va, pl[nt][0], pl[nt][1]);
            }
          }
        } else {
          // lane (n, c): columns 32 g + 4 n .. + 3 of keys 2c, 2c+1, 2c+8, 2c+9; the
          // first two are rows n, n + 8 of output tile 2 g, the others of 2 g + 1
#pragma unroll
          for (int g = 0; g < D / 32; ++g) {
            const int ch = 2 * g + n / 4, in = 4 * (n % 4), key = 16 * ksub + 2 * c;
            const uint32_t w0 = lds32(vt + swz<C::kBox>(key, ch) + in);
            const uint32_t w1 = lds32(vt + swz<C::kBox>(key + 1, ch) + in);
            const uint32_t w2 = lds32(vt + swz<C::kBox>(key + 8, ch) + in);
            const uint32_t w3 = lds32(vt + swz<C::kBox>(key + 9, ch) + in);
            const uint32_t a01 = __byte_perm(w0, w1, 0x5140), b01 = __byte_perm(w0, w1, 0x7362);
            const uint32_t a23 = __byte_perm(w2, w3, 0x5140), b23 = __byte_perm(w2, w3, 0x7362);
            const uint32_t va[4] = {codes_lo(a01), codes_hi(a01), codes_lo(a23), codes_hi(a23)};
            const uint32_t vb[4] = {codes_lo(b01), codes_hi(b01), codes_lo(b23), codes_hi(b23)};
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt) {
              mma<true>(o[2 * g][nt], va, pb[nt][0], pb[nt][1]);
              mma<true>(o[2 * g + 1][nt], vb, pb[nt][0], pb[nt][1]);
            }
          }
        }
      }
      if (edge) fence_async_smem();  // this thread wrote to the stage; a copy follows
      __syncwarp();
      feed();
      if (++stage == C::kOwn) stage = 0, parity ^= 1;
    }

    // ------------------------------------------------------ the piece's end --
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) l[nt][i] += __shfl_xor_sync(0xffffffffu, l[nt][i], off);
        close_row(m[nt][i], l[nt][i]);
        if (n == 0) {
          sm_m[warp][8 * nt + 2 * c + i] = m[nt][i];
          sm_l[warp][8 * nt + 2 * c + i] = l[nt][i];
        }
      }
    const bool whole = t_begin == 0 && t_end == wk.tiles;
    const int slot = whole ? -1 : (2 * unit + !first) * w.heads + sub;
    __syncwarp();
    PieceEnd<D, kCodes, kRows> end;
    end.rows_of(p, sq, h, row0, slot, sm_m[warp], sm_l[warp], (uint64_t)hidden[1] << 32 | hidden[0],
                poison || expired, lane);
#pragma unroll
    for (int g = 0; g < D / C::kTurn; ++g) {
#pragma unroll
      for (int mt = 2 * g; mt < 2 * g + 2; ++mt)
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int col = kCodes ? 4 * n + 2 * (mt & 1) + (i >> 1) : 16 * (mt & 1) + n + 8 * (i >> 1);
            turn[(8 * nt + 2 * c + (i & 1)) * C::kPad + col] = o[mt][nt][i];
          }
      __syncwarp();
      end.columns(p, sq, wk.b, h, turn, C::kPad, C::kTurn * g, lane);
      __syncwarp();
    }
    if (lane == 0) hidden[0] = hidden[1] = 0;
    __syncwarp();
    first = false;
  } while (wk.next(p, w));
  if (kCodes) asm volatile("cp.async.wait_all;" ::: "memory");
  if (expired) {  // let copies in flight land before the CTA leaves
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 1000000ull) {
    }
  }
}

}  // namespace tree
}  // namespace attn
