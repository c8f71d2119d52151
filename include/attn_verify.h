/*
 * C ABI of the verification of drafted tokens on GB300 (sm_103a): which of the
 * drafts that attn_fwd_tree attended to (attn_cache.h) the target model keeps, and
 * the token that follows them, drawn so that they are distributed as the target's
 * own.  Conventions as in attn_fwd.h.
 */
#ifndef IO_AWARE_EXACT_06_ATTN_VERIFY_H
#define IO_AWARE_EXACT_06_ATTN_VERIFY_H

#include <stddef.h>
#include <stdint.h>

#include "attn_fwd.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * attn_verify_drafts: new token 0 of a sequence (packed row cu_seqlens[b]) is
 * accepted already; the others are drafts, a chain (mask == NULL) or a tree (mask as
 * for attn_fwd_tree: a draft's parent is the highest new token before it whose bit it
 * has; one without is never reached).  Row i of probs is the target's distribution
 * behind new token i, row i of draft_probs the one that token i's children were drawn
 * from, [total, V] fp32 (bf16 == 0) or bf16, rows any stride apart.
 * From token 0 on, at each node, its children are tried in their order.  With p and q
 * the node's rows, s = 0, z = 1 and w = p at first, child x is accepted where
 *     u q(x) z < w(x),   u = u_accept of the child's row,
 * and the walk goes on from it; else s += z, w = max(p - s q, 0), z = sum w (the
 * residual of a rejection, not normed).  draft_probs == NULL: drafts count as certain;
 * a child is accepted where u z < w(x), else w(x) = 0 and z decreases by it.  Where no
 * child is left, the next token is the first x with w(0) + .. + w(x) > u_next[b] times
 * the sum of w; where that sum is 0, of p.
 * Probabilities are taken between 0 and 1 (NaN: 0).  Tests are made in fp64.  In sums, and
 * in the draw, each entry of w is taken to the nearest multiple of 2^-43 (one of 2^-44 or less
 * counts as 0, so it is never drawn), and these are added exactly: results do not depend on
 * the launch and repeat bit for bit.  The tokens are distributed as the target's, to that
 * rounding and to that of the random numbers, where rows add up to 1; rows are not normed: with
 * certain drafts z is 1 less what was rejected, whatever the row's sum.
 * tokens: int32[total]; u_accept: fp32[total], u_next: fp32[B], in [0, 1).
 * path: int32[total], from cu_seqlens[b] on the accepted new tokens, 0 and the accepted
 * drafts (indices within the sequence, increasing), then -1; accepted: int32[B], how
 * many; next_token: int32[B]; seqlens (NULL: none) with the new tokens and seqlens_out
 * (may be the same) with the accepted ones, int32[B].  A sequence without new tokens
 * has accepted 0 and next_token -1; next_token is also -1 where a row has no
 * entry above 2^-44.  At most 64 new tokens; V at most 262144.
 * Errors in the error word: ATTN_ERR_SEQLENS (offsets that decrease, for all sequences;
 * a sequence that begins below 0, the first anywhere but at 0, ends past total, has more
 * than 64 new tokens or is shorter than them: accepted 0, next_token -1, its length as
 * given, its path not written), ATTN_ERR_INDEX (a draft outside the vocabulary: it is
 * rejected).
 */
int attn_verify_drafts(const int32_t *tokens, const void *probs, int64_t probs_stride,
                       const void *draft_probs, int64_t draft_stride, int bf16,
                       const int32_t *cu_seqlens, const int64_t *mask, const float *u_accept,
                       const float *u_next, const int32_t *seqlens, int32_t *path, int32_t *accepted,
                       int32_t *next_token, int32_t *seqlens_out, int B, int total, int V,
                       attn_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* IO_AWARE_EXACT_06_ATTN_VERIFY_H */
