// How attention over the paged cache is cut for a launch: query rows of a tile, the
// kernel, the line's units and the workspace.
#pragma once

#include "attn_serve_host.h"
#include "attn_tree_few_kernel.cuh"
#include "attn_tree_tile_kernel.cuh"

namespace attn_serve {

struct Plan {
  int rows;  // query rows of a segment: 8 or 16 (few rows), 128 or 256
  attn::tree::Work work;
  int64_t ctas;
  int64_t slots;  // parts in the workspace, `rows` rows each
  bool many;      // eight warps join a row's pieces
  bool fits;      // the line's tiles are a 32-bit number
};

inline bool few(const Plan& pl) { return pl.rows <= 16; }

// Query rows of a segment: the smallest tile that holds max_new * G of them.
// Few rows: as many persistent warps as fit the SMs; more: a persistent CTA an SM
// with tcgen05 products.  9 to 16 rows take the former but for a bf16 cache with
// d = 128, where HBM outruns its arithmetic (us, few : many; 12 rows, 16 sequences of
// 4096 keys: d = 128 bf16 104 : 82, e4m3 69 : 84, d = 64 52 : 63 and 54 : 75; 16 rows,
// 64 sequences of 8192 keys: d = 128 bf16 284 : 254, e4m3 192 : 247).  num_splits caps
// the pieces of a segment instead.
inline Plan tree_plan(int B, int total, int Hq, int H, int d, int max_new, int max_len, int num_splits, bool codes,
                      bool shared = false) {
  Plan pl{};
  const int64_t M = (int64_t)max_new * (Hq / H);
  constexpr int kBig = attn::tree::kBigRows;
  pl.rows = M <= 8 ? 8 : M <= 16 && (d == 64 || codes) ? 16 : M <= kBig ? kBig : 2 * kBig;
  const int64_t T = few(pl) ? attn::tree::kFewTile : attn::tree::kBigTile;
  const int64_t tiles = (std::max<int64_t>(max_len, 1) + T - 1) / T;
  const int heads = !few(pl) ? 1 : H % 4 == 0 ? 4 : H % 2 == 0 ? 2 : 1;  // of a segment, one a warp
  const int64_t segments = (int64_t)B * (H / heads) * ((M + pl.rows - 1) / pl.rows);
  const int per_cta = few(pl) ? attn::tree::few_warps(shared, pl.rows) / heads : 1;
  pl.work.rows = pl.rows;
  pl.work.heads = heads;
  pl.work.log_tile = few(pl) ? attn::tree::kLogFewTile : attn::tree::kLogBigTile;
  pl.work.min_share = num_splits > 0 ? (int)((tiles + num_splits - 1) / num_splits) : 1;
  const int64_t most = (int64_t)std::min((double)segments * (double)tiles / pl.work.min_share + 1, 1e9);
  pl.ctas = std::min<int64_t>((most + per_cta - 1) / per_cta, kPlanSms * (few(pl) && !shared ? attn::tree::few_ctas(d, codes) : 1));
  pl.work.units = (int)(pl.ctas * per_cta);
  pl.slots = 2 * (int64_t)pl.work.units * heads;
  // eight warps to a row where segments are cut into many pieces, and where the
  // rows leave the SMs idle anyway
  pl.many = pl.work.units > 32 * segments || (int64_t)total * Hq <= 8 * kPlanSms;
  pl.fits = (double)segments * (double)tiles <= INT32_MAX - (shared ? 1 << 16 : 0);  // (segments may be padded)
  return pl;
}

inline size_t tree_rows(const Plan& pl) { return (size_t)pl.slots * pl.rows; }
inline size_t tree_bytes(const Plan& pl, int d) { return tree_rows(pl) * (d + 1) * sizeof(float); }

inline int check_tree(int B, int total, int Hq, int H, int d, int max_new, int max_len, int num_splits) {
  if (d != 64 && d != 128) return ATTN_ERR_HEADDIM;
  if (B < 0 || total < 0 || Hq < 1 || H < 1 || Hq % H || (int64_t)Hq * d > (1 << 20)) return ATTN_ERR_SHAPE;
  if (max_new < 0 || max_new > attn::tree::kMaxNew || max_len < max_new || num_splits < 0 || num_splits > 256)
    return ATTN_ERR_SHAPE;
  if (max_len > INT32_MAX - 256) return ATTN_ERR_SHAPE;
  return ATTN_OK;
}

// The kernel of a plan over one line of work.
template <int D, bool kCodes, bool kShared>
int launch_line(const Plan& pl, const CUtensorMap& mk, const CUtensorMap& mv, const attn::tree::Params& p,
                cudaStream_t s) {
  using namespace attn::tree;
  constexpr int kTwo = D == 64 || kCodes ? 2 : 1;  // no plan has 16 rows of the other kind
  auto kernel = pl.rows == 8          ? tree_few_kernel<D, kCodes, 1, kShared>
                : pl.rows == 16       ? tree_few_kernel<D, kCodes, kTwo, kShared>
                : pl.rows == kBigRows ? tree_tile_kernel<D, kCodes, false, kShared>
                                      : tree_tile_kernel<D, kCodes, true, kShared>;
  const int smem = pl.rows == 8          ? FewCfg<D, kCodes, 1, kShared>::kSmem
                   : pl.rows == 16       ? FewCfg<D, kCodes, kTwo, kShared>::kSmem
                   : pl.rows == kBigRows ? big_smem<D, kCodes, false>()
                                         : big_smem<D, kCodes, true>();
  const int st = allow_smem(reinterpret_cast<const void*>(kernel), smem);
  if (st != ATTN_OK) return st;
  return launch(kernel, pl.ctas, few(pl) ? 32 * few_warps(kShared, pl.rows) : kBigThreads, smem, s, mk, mv, p, pl.work);
}

}  // namespace attn_serve
