/*
 * C ABI of the paged key/value cache on GB300 (sm_103a): writing new tokens
 * into it, reading it back, attention over it for the newest token or a
 * tree of drafted tokens of every sequence (sequences that share a prefix
 * included), and its pages between steps: forked, copied, given back, accepted
 * drafts moved together.
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

/*
 * attn_fwd_prefix: attn_fwd_tree for groups of sequences that share a prefix
 * (samples of one prompt), whose keys and values are read once for all rows of
 * the group.  Sequences cu_groups[g] .. cu_groups[g+1]-1 are group g (cu_groups:
 * int32[groups+1], prefix_lens: int32[groups], on the device); their tables name
 * the same pages for the first prefix_lens[g] positions, as far as these fill
 * pages, and those are read by the first of these tables.  (What follows in a
 * page that is not filled is each sequence's own.)  A prefix ends before the new
 * tokens of its sequences.  A sequence in no group shares nothing; one without new
 * tokens has no rows, and neither its table nor its length's place behind the prefix
 * counts (nor the prefix of a group without them); groups may be empty, groups may be 0.  Everything else as for attn_fwd_tree; results differ
 * from its by rounding alone, and where max_new tokens have at most 8 rows a key head (16 with
 * d = 64) over a bf16 cache both hold a probability as the sum of two bf16, else as one.
 * Over codes the rows of a group count together for what is said there of more than 16.
 * It has two launches more than attn_fwd_tree, which is faster where little is shared: groups of
 * less than some eight sequences, or (sequences - groups) * prefix below some 30000 positions (8
 * sequences: 15 us against 24 with a prefix of 512, 38 against 31 with 8192).
 * max_group >= the new tokens of every group together, max_prefix >= every
 * prefix_lens[g], at most max_len: they size the launch (close bounds pick the
 * kernels that fit).
 * workspace: attn_fwd_prefix_workspace(...) bytes, as for attn_fwd_tree.
 * Errors in the error word: those of attn_fwd_tree, and ATTN_ERR_SEQLENS where
 * cu_groups decreases (no row is written), where a group lies outside the batch or
 * exceeds the bounds (no row of its sequences is), or a prefix reaches into a
 * sequence's new tokens (no row of that sequence is).  A page of a prefix outside
 * the cache makes the group's rows NaN.
 */
int attn_fwd_prefix(const void *q, int64_t q_stride, const attn_paged_cache *cache,
                    const int32_t *seqlens, const int32_t *cu_seqlens, const int64_t *mask,
                    const int32_t *cu_groups, const int32_t *prefix_lens, void *o, float *lse, int B,
                    int total, int Hq, int max_new, int max_len, int groups, int max_group,
                    int max_prefix, float scale, int num_splits, void *workspace,
                    size_t workspace_bytes, attn_stream_t stream);

size_t attn_fwd_prefix_workspace(int B, int total, int Hq, int H, int d, int max_new, int max_len,
                                 int groups, int max_group, int max_prefix, int num_splits);

/*
 * attn_cache_fork: the page table of the next batch.  Its row i (of N) goes on
 * with row parents[i] of the present one (of B; -1: with none) to new_seqlens[i]
 * positions: a parent named once goes on, one named several times is forked, one
 * not named is given up; a row may grow, shrink, or end (0).  A row of length n
 * has ceil(n / page_size) pages; the rest of its table is -1.
 * refs[page] counts the rows whose tables name the page, 0: it is free.  A row
 * keeps its parent's pages as far as it needs them and gets free ones behind
 * them: the lowest-numbered, in the order of the rows and of their positions.
 * Where it grows into a page that its parent had filled in part, it writes there:
 * it keeps that page if nobody else has it (no other row before the call; of the
 * children that have it, all grow and it is the first), else it gets a free one,
 * and copy_src[i] and copy_dst[i] name the pages to copy (attn_cache_copy, for
 * each layer's cache); they are -1 elsewhere.  Pages given up may be handed out
 * by the next call, not by this one.
 * page_table [B, page_table_stride], page_table_out [N, page_table_stride] (not
 * the same memory: ATTN_ERR_SHAPE), refs and refs_out [num_pages] (the same, or
 * apart: ATTN_ERR_SHAPE), seqlens [B], parents, new_seqlens, copy_src and copy_dst [N], all int32
 * on the device.  page_size 16, 32, 64, 128 or 256.
 * workspace: attn_cache_fork_workspace(...) bytes of the caller's device memory,
 * 16-byte aligned, not initialised, in use until the call's work on stream has finished.
 * Errors in the error word: ATTN_ERR_SEQLENS (a length below 0 or beyond the
 * table), ATTN_ERR_INDEX (a parent outside the batch; a page outside the cache or
 * with a count below 1) and ATTN_ERR_PAGES (fewer free pages than asked for):
 * nothing changes hands then, refs_out is refs and the rest -1.  A page that a table
 * names more often than refs counts is reported (ATTN_ERR_INDEX) as its count falls
 * below 0.
 */
int attn_cache_fork(const int32_t *page_table, int page_table_stride, const int32_t *seqlens, int B,
                    const int32_t *parents, const int32_t *new_seqlens, int N, const int32_t *refs,
                    int32_t *refs_out, int num_pages, int page_size, int32_t *page_table_out,
                    int32_t *copy_src, int32_t *copy_dst, void *workspace, size_t workspace_bytes,
                    attn_stream_t stream);

size_t attn_cache_fork_workspace(int B, int N, int page_table_stride, int num_pages, int page_size);

/*
 * attn_cache_copy: page src[i] of the cache, all of it, into page dst[i], for the
 * n pairs in which src[i] is not -1 (int32[n] on the device).  A page may be the
 * source of many pairs; the target of one, and not a source as well.  The page table
 * is not read (it may be NULL).  ATTN_ERR_INDEX in the error word: a page outside
 * the cache; that pair is left out.
 */
int attn_cache_copy(const attn_paged_cache *cache, const int32_t *src, const int32_t *dst, int n,
                    attn_stream_t stream);

/*
 * attn_cache_compact: the accepted ones of the new tokens of every sequence moved
 * to the first of their places: new token path[cu_seqlens[b] + j] to place j, for j
 * below accepted[b] (as attn_verify_drafts returns them; they increase with j).
 * seqlens as for the attention that wrote them, all new tokens included; the
 * sequence goes on with seqlens[b] - n_b + accepted[b] positions, and what is behind
 * them is left as it was.  Two sequences whose new tokens share a page must not both
 * move in it.
 * Errors in the error word: ATTN_ERR_SEQLENS as for attn_cache_write; ATTN_ERR_INDEX
 * (accepted[b] below 0 or above n_b, a path that does not increase or leaves the new
 * tokens: nothing of that sequence is moved; a page outside the cache: that row is not).
 */
int attn_cache_compact(const attn_paged_cache *cache, const int32_t *seqlens, const int32_t *cu_seqlens,
                       const int32_t *path, const int32_t *accepted, int B, int total,
                       attn_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* IO_AWARE_EXACT_06_ATTN_CACHE_H */
