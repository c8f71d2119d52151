/*
 * C ABI of the step before attention on GB300 (sm_103a): the norm of every
 * query and key head with the rotary position rotation in the same pass, and
 * its gradient.
 *
 * For a row x (one token and head, d channels), w the weight of its kind
 * (queries or keys), r = (mean_c x_c^2 + eps)^(-1/2):
 *     y0_c = x_c r w_c
 *     y_a  = y0_a cos_j - y0_b sin_j,   y_b = y0_b cos_j + y0_a sin_j
 * for the pairs (a, b) of channels j < rot / 2: (j, j + rot/2), or
 * (2j, 2j + 1) when interleaved; channels from rot on are not rotated.
 * cos_j and sin_j are row pos of the caller's tables, pos the token's position
 * on the axis that pair j belongs to (one axis for text; time, height and width
 * for images and video).
 *
 * Numerics: bf16 in and out, everything between in fp32, rounded once.
 * Conventions (device pointers, asynchronous on stream, status codes, the
 * error word read by attn_last_device_error) as in attn_fwd.h.
 */
#ifndef IO_AWARE_EXACT_06_ATTN_NORM_H
#define IO_AWARE_EXACT_06_ATTN_NORM_H

#include <stddef.h>
#include <stdint.h>

#include "attn_fwd.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The rotation.  cos, sin: fp32 [table_len, rot / 2], 16-byte aligned.
 * positions: int32 [axes, T] on the device, each in [0, table_len).  Pair j
 * belongs to axis 0 for j < section[0], to axis 1 for the next section[1]
 * pairs, and so on; the sections of the axes add up to rot / 2 (with one axis
 * section is not read).  rot: a multiple of 16 from 0 to d; rot = 0 leaves
 * the norm alone and reads no table. */
typedef struct {
    const float *cos, *sin;
    const int32_t *positions;
    int table_len;
    int rot;
    int axes; /* 1, 2 or 3 */
    int section[3];
    int interleaved;
} attn_rotary;

/*
 * attn_qk_norm_rope: q [T, Hq, d] and k [T, Hk, d] bf16 to q_out and k_out of
 * the same shapes.  *_stride: elements from one token to the next (heads of a
 * token are contiguous, so at least H * d; slices of a fused projection have
 * more), multiples of 8.  wq, wk: bf16 [d].  eps: finite and >= 0.  d: 64 or
 * 128.  q_out may be q itself and k_out k itself (same stride); no other
 * overlap.  Hk = 0 (k, wk, k_out unused) or Hq = 0 is allowed.
 * Alignment: 16 bytes for the bf16 tensors and tables.
 * A token with a position outside its table is not written and sets
 * ATTN_ERR_INDEX in the error word.  T == 0 is a no-op.
 */
int attn_qk_norm_rope(const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                      const void *wq, const void *wk, void *q_out, int64_t q_out_stride,
                      void *k_out, int64_t k_out_stride, int T, int Hq, int Hk, int d, float eps,
                      const attn_rotary *rotary, attn_stream_t stream);

/*
 * attn_qk_norm_rope_bwd: the gradient.  q, k: the forward's inputs (not its
 * outputs); dq_out, dk_out: the gradients of its outputs; writes dq, dk (bf16)
 * and dwq, dwk (fp32 [d], summed over all tokens and heads in an order that
 * depends on the shape alone, so that results repeat bit for bit).  dq may be
 * dq_out itself and dk dk_out itself (same stride); no other overlap.  A token
 * with a position outside its table adds nothing to dwq and dwk and its dq and
 * dk are not written (ATTN_ERR_INDEX).  T == 0 writes dwq = dwk = 0; Hq = 0
 * writes dwq = 0 and Hk = 0 dwk = 0, unless they are NULL.
 * workspace: attn_qk_norm_rope_bwd_workspace(T, Hq, Hk, d) bytes of the
 * caller's device memory, 16-byte aligned, not initialised, in use until the
 * call's work on stream has finished (calls that may run at the same time
 * need one each).  Missing or too small: ATTN_ERR_SCRATCH.
 */
int attn_qk_norm_rope_bwd(const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                          const void *wq, const void *wk, const void *dq_out, int64_t dq_out_stride,
                          const void *dk_out, int64_t dk_out_stride, void *dq, int64_t dq_stride,
                          void *dk, int64_t dk_stride, float *dwq, float *dwk, int T, int Hq, int Hk,
                          int d, float eps, const attn_rotary *rotary, void *workspace,
                          size_t workspace_bytes, attn_stream_t stream);

size_t attn_qk_norm_rope_bwd_workspace(int T, int Hq, int Hk, int d);

#ifdef __cplusplus
}
#endif

#endif /* IO_AWARE_EXACT_06_ATTN_NORM_H */
