/*
 * C ABI of the paged key/value cache on GB300 (sm_103a): writing new tokens
 * into it, reading it back, and attention over it for the newest token or a
 * tree of drafted tokens of every sequence.
 *
 * The cache holds num_pages pages of page_size token rows.  Position p of
 * sequence b is row p % page_size of page page_table[b][p / page_size].  Keys
 * and values are bf16, or e4m3 codes with one fp32 scale per token and head
 * (scale = max(max_c |x_c| / 448, 2^-64), code_c = e4m3(x_c * (1 / scale)) in
 * fp32, round to nearest even; a row with a NaN or an infinity reads back as
 * NaN).
 *
 * A batch of B sequences adds the tokens cu_seqlens[b] .. cu_seqlens[b+1]-1
 * of packed tensors to sequence b, at its last positions: seqlens[b] is its
 * length with them.  Packed rows from cu_seqlens[B] on belong to no sequence:
 * they have no effect and are not written (padded batches).
 *
 * Lengths, positions and pages are checked on the device, where they are
 * used; nothing outside the caller's tensors is read or written whatever they
 * hold.  Conventions as in attn_fwd.h.
 */
#ifndef IO_AWARE_EXACT_06_ATTN_CACHE_H
#define IO_AWARE_EXACT_06_ATTN_CACHE_H

#include <stddef.h>
#include <stdint.h>

#include "attn_fwd.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
    void *k, *v;              /* [num_pages, page_size, H, d] bf16, or uint8 e4m3 codes */
    float *k_scale, *v_scale; /* [num_pages, H, page_size] fp32 for codes; both NULL for bf16 */
    const int32_t *page_table; /* [B, page_table_stride] on the device */
    int page_table_stride;     /* pages of the longest sequence the table has room for */
    int num_pages;
    int page_size; /* 16, 32, 64, 128 or 256 */
    int H;         /* heads of keys and values */
    int d;         /* 64 or 128 */
} attn_paged_cache;

/*
 * attn_cache_write: k, v [total, H, d] bf16 (token strides in elements,
 * multiples of 8, at least H * d) into the cache.  Two sequences whose tables
 * share a page must not both write to it.
 * Errors in the error word: ATTN_ERR_SEQLENS and ATTN_ERR_INDEX (a page outside
 * the cache; its tokens are not written).  ATTN_ERR_SEQLENS: cu_seqlens decreases
 * somewhere, which places no token: nothing is written; or a sequence that begins
 * below 0 (the first: anywhere but at 0), ends past total, is shorter than its new
 * tokens or longer than its table: its tokens are not written.
 */
int attn_cache_write(const attn_paged_cache *cache, const void *k, int64_t k_stride, const void *v,
                     int64_t v_stride, const int32_t *seqlens, const int32_t *cu_seqlens, int B,
                     int total, attn_stream_t stream);

/*
 * attn_cache_read: positions 0 .. cu_seqlens[b+1] - cu_seqlens[b] - 1 of every
 * sequence into the packed rows cu_seqlens[b] .. of k, v [total, H, d] bf16
 * (contiguous), the layout attn_fwd and attn_fwd_decode take.  (Those have as
 * many key heads as query heads: heads that queries share are repeated for
 * them first; attn_fwd_tree reads shared heads as they are.)  Codes read back
 * as bf16(code * scale).  Errors as for attn_cache_write; the rows concerned
 * are not written.
 */
int attn_cache_read(const attn_paged_cache *cache, void *k, void *v, const int32_t *cu_seqlens, int B,
                    int total, attn_stream_t stream);

/*
 * attn_fwd_tree: attention of the new tokens of every sequence over its cached
 * keys and values, the new tokens' own included (written before):
 *     O_i = sum_j softmax_j(scale q_i . k_j) v_j,  LSE_i as in attn_fwd.h,
 * over the keys j < seqlens[b] - n_b (n_b its new tokens) and those new tokens
 * whose bit is set in mask[i]: bit t of the 64-bit word of new token i stands
 * for new token t of the same sequence (a tree of drafted tokens: itself and
 * its ancestors).  mask == NULL: every new token sees itself and the ones
 * before it (n_b = 1: decoding).  A row that sees no key gets O = 0 and
 * LSE = -inf; what keys and values hold where a row does not see them,
 * infinities and NaN included, does not reach it.  A query with an infinity or a
 * NaN gives a row of NaN (LSE too) wherever it sees a key.  Over codes, where
 * more than 16 query rows share a key head, values whose scale is 2^-64 or less
 * may count as 0 beside scales that are 2^12 times larger and more.
 * q: [total, Hq, d] bf16, token stride in elements (multiple of 8, at least
 * Hq * d); Hq a multiple of cache->H, head h reads key head h / (Hq / H).
 * o: [total, Hq, d] bf16, lse: [total, Hq] fp32, contiguous.  mask: int64
 * [total] on the device.
 * max_new >= every n_b, at most 64; max_len >= every seqlens[b] (they size the
 * launch; larger values on the device are an error).  All sequences' keys, taken
 * together, are cut into equal shares for the GPU; num_splits, 1..256, bounds the
 * pieces that the keys of a sequence of max_len fall into (num_splits + 1 at most;
 * shorter sequences fall into fewer), 0 leaves them to the launch.  Results depend
 * on it, on the lengths and on the sizes by rounding alone, and repeat bit for bit.
 * workspace: attn_fwd_tree_workspace(...) bytes of the caller's device memory, for
 * the pieces (it does not grow with the lengths beyond a launch's pieces), 16-byte
 * aligned, not initialised, in use until the call's work on stream has finished;
 * calls that may run at the same time need one each.  Missing or too small:
 * ATTN_ERR_SCRATCH.
 * ATTN_ERR_SHAPE also where the key tiles of a batch (at most B * H * max_len / 32,
 * times max_new * Hq / H / 256 rounded up) could be more than 2^31 - 1.
 * Errors in the error word: ATTN_ERR_SEQLENS (offsets and lengths as for
 * attn_cache_write, and the bounds max_new and max_len; the rows of that sequence,
 * with offsets that decrease all rows, are not written), ATTN_ERR_INDEX (a page
 * outside the cache; the rows that read it come out as NaN),
 * ATTN_ERR_DEVICE_TIMEOUT (NaN as well).
 */
int attn_fwd_tree(const void *q, int64_t q_stride, const attn_paged_cache *cache,
                  const int32_t *seqlens, const int32_t *cu_seqlens, const int64_t *mask, void *o,
                  float *lse, int B, int total, int Hq, int max_new, int max_len, float scale,
                  int num_splits, void *workspace, size_t workspace_bytes, attn_stream_t stream);

size_t attn_fwd_tree_workspace(int B, int total, int Hq, int H, int d, int max_new, int max_len,
                               int num_splits);

#ifdef __cplusplus
}
#endif

#endif /* IO_AWARE_EXACT_06_ATTN_CACHE_H */
