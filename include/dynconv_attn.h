/*
 * dynconv_attn.h -- C ABI of the operators that follow the Q/K/V convolution: rotary
 * positions, causal attention over packed prompts (forward and backward) and attention of
 * new or drafted tokens over a key/value cache.
 *
 * They take what dynconv_fwd / dynconv_fwd_varlen leave: token-major rows whose heads are
 * runs of head_dim channels, so that Q, K and V may be column slices of one [N, C] buffer
 * (row strides in the descriptors) and their gradients may be written into one [N, C]
 * buffer that dynconv_bwd reads.
 *
 * Conventions are those of dynconv.h: storage dtype fp32 or bf16; every sum, softmax
 * statistic and norm in fp32; the caller owns every buffer (device pointers, 16-byte
 * aligned; a host pointer is DYNCONV_ERR_INVALID); nothing is allocated; work is enqueued
 * on `stream` of the current device and nothing synchronises; arguments are validated
 * before any launch; a row stride of 0 means dense rows.  The workspace is zeroed once
 * before its first use, must not serve two calls that overlap on the device (two captured
 * graphs may share one where they replay one after the other), and holds the device error word that dynconv_device_status(ws, ...) reports and clears.
 * A call may be captured into a CUDA graph.  But for dynconv_rope in place, no output may
 * overlap an input.
 */
#ifndef DYNCONV_ATTN_H
#define DYNCONV_ATTN_H

#include "dynconv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------ rotary positions
 * Pair layouts of the rotated channels [0, rot_dim) of a head (RoFormer, section 3.4.2,
 * rotates consecutive channels; the half layout pairs channel i with i + rot_dim / 2). */
typedef enum { DYNCONV_ROPE_INTERLEAVED = 0, DYNCONV_ROPE_HALF = 1 } dynconv_rope_layout;

typedef struct {
    int32_t dtype;          /* dynconv_dtype of x and y */
    int32_t layout;         /* dynconv_rope_layout */
    int64_t batch;          /* sequences of seqlen tokens (packed documents: 1) */
    int64_t seqlen;         /* tokens per sequence (packed documents: all N, up to 2^31 - 256) */
    int64_t heads;          /* heads per row */
    int64_t head_dim;       /* channels per head */
    int64_t rot_dim;        /* rotated channels of each head: even, 2..head_dim */
    int64_t x_row_stride;   /* elements between tokens of x; 0 = heads * head_dim */
    int64_t y_row_stride;   /* elements between tokens of y; 0 = heads * head_dim */
    int64_t max_pos;        /* rows of cos_sin; every position must be below it */
    const float *cos_sin;   /* DEVICE fp32 [max_pos, rot_dim]: entries 2i, 2i+1 of row p are the
                               factors of pair i at position p (cosine and sine of its angle,
                               times a gain where the context scaling has one) */
    int32_t inverse;        /* 1: the transposed rotation (the backward of the forward one) */
} dynconv_rope_desc;

/* Rotary positions: y[n, head, :] = R(p(n)) x[n, head, :].  Pair (a, b) of channels becomes
 *   (a cos - b sin, a sin + b cos)      (inverse: (a cos + b sin, b cos - a sin)),
 * channels from rot_dim on are copied.  p(n) = positions[n] (DEVICE int32 [N]) or, with
 * positions NULL, n's place in its sequence or packed document (cu_seqlens as in
 * dynconv_fwd_varlen, batch 1).  y may be x (same row stride); other overlaps are undefined.
 *   ws  256 bytes or more, zeroed once (the device error word)
 * Errors: DYNCONV_ERR_INVALID; a position outside [0, max_pos) or a malformed cu_seqlens
 * raises the device check, and that token's row of the table is clamped into range. */
DYNCONV_API dynconv_status dynconv_rope(const dynconv_rope_desc *desc, const int32_t *cu_seqlens, int64_t n_docs,
                                        const int32_t *positions, const void *x, void *y, void *ws,
                                        size_t ws_bytes, void *stream);

/* ------------------------------------------------------------------ causal attention */
typedef struct {
    int32_t dtype;          /* dynconv_dtype of every tensor but lse */
    int32_t algo;           /* dynconv_algo: AUTO, SIMT (CUDA cores) or TC (tensor cores) */
    int64_t batch;          /* sequences of seqlen tokens (packed documents: 1) */
    int64_t seqlen;         /* tokens per sequence (packed documents: all N, up to 2^31 - 256) */
    int64_t heads;          /* query heads; query head i reads key/value head i / (heads / kv_heads) */
    int64_t kv_heads;       /* divides heads */
    int64_t head_dim;       /* 1..128 */
    int64_t q_row_stride, k_row_stride, v_row_stride, o_row_stride;        /* elements between tokens; 0 = dense */
    int64_t do_row_stride, dq_row_stride, dk_row_stride, dv_row_stride;    /* backward; 0 = dense */
    float scale;            /* positive and finite; 0 = 1 / sqrt(head_dim) */
} dynconv_attn_desc;

/* Workspace of both passes (0 for an invalid descriptor). */
DYNCONV_API size_t dynconv_attn_workspace_bytes(const dynconv_attn_desc *desc);

/* Kernel families of a descriptor, as dynconv_query_family: bf16 with head_dim and every row
 * stride a multiple of 8 runs the tcgen05 kernels, the rest the CUDA-core kernels (the
 * reason in dynconv_last_error()).  Host-only. */
DYNCONV_API dynconv_status dynconv_attn_query_family(const dynconv_attn_desc *desc, int32_t *fwd_family,
                                                     int32_t *bwd_family);

/* Causal attention, every head of every sequence or packed document:
 *   o[n] = sum_j p[n,j] v[j],  p[n,:] = softmax over s(n) <= j <= n of scale q[n].k[j]
 * with s(n) the first token of n's sequence (dense batch, cu_seqlens NULL) or document
 * (cu_seqlens: DEVICE int32 [n_docs + 1], batch 1; 0 ... N, non-decreasing; documents of no
 * tokens are allowed).  A token outside that range has no influence on o[n], whatever it holds
 * (infinities and NaN among it).  A row without a finite score has no softmax: its o is NaN.
 *   q [N, heads * head_dim], k and v [N, kv_heads * head_dim], o [N, heads * head_dim]
 *   lse  nullable fp32 [heads, N]: log of the sum of exp(scale q.k), for the backward
 * Errors: DYNCONV_ERR_INVALID, _UNSUPPORTED (head_dim above 128, N * heads beyond the grid, more than
 * 2^30 documents), _WORKSPACE, _CUDA; a malformed cu_seqlens raises the device check (the call's
 * results are then undefined, every access stays inside the tensors). */
DYNCONV_API dynconv_status dynconv_attn_fwd(const dynconv_attn_desc *desc, const int32_t *cu_seqlens, int64_t n_docs,
                                            const void *q, const void *k, const void *v, void *o, float *lse,
                                            void *ws, size_t ws_bytes, void *stream);

/* Backward of dynconv_attn_fwd from its o and lse and the gradient d_o = dL/do:
 *   dp[n,j] = d_o[n].v[j],  D[n] = d_o[n].o[n],  ds[n,j] = p[n,j] (dp[n,j] - D[n])
 *   dq[n] = scale sum_j ds[n,j] k[j],  dk[j] = scale sum ds[n,j] q[n],  dv[j] = sum p[n,j] d_o[n]
 * the sums of dk and dv over every token n of the document and every head of the group.
 * All outputs are overwritten.  Every sum is in a fixed order: the results repeat bitwise.
 * dq, dk, dv may be column slices of one buffer. */
DYNCONV_API dynconv_status dynconv_attn_bwd(const dynconv_attn_desc *desc, const int32_t *cu_seqlens, int64_t n_docs,
                                            const void *d_o, const void *q, const void *k, const void *v,
                                            const void *o, const float *lse, void *dq, void *dk, void *dv,
                                            void *ws, size_t ws_bytes, void *stream);

/* ------------------------------------------------------------------ attention over a cache */
typedef struct {
    int32_t dtype;          /* dynconv_dtype of every tensor and of the caches */
    int32_t rope_layout;    /* dynconv_rope_layout (rope_dim > 0) */
    int64_t batch;          /* sequences */
    int64_t tokens;         /* new or drafted tokens per sequence: 1..64 */
    int64_t heads, kv_heads, head_dim;   /* as dynconv_attn_desc; head_dim a multiple of 16 bytes */
    int64_t max_len;        /* tokens each sequence's cache holds */
    int64_t q_row_stride, k_row_stride, v_row_stride, o_row_stride;   /* multiples of 16 bytes; 0 = dense */
    int64_t rope_dim;       /* rotated channels of each q and k head: 0 (none) or even, up to head_dim */
    int64_t rope_max_pos;   /* rows of rope_cos_sin */
    const float *rope_cos_sin;   /* as dynconv_rope_desc.cos_sin, [rope_max_pos, rope_dim] */
    float scale;            /* positive and finite; 0 = 1 / sqrt(head_dim) */
} dynconv_attn_decode_desc;

DYNCONV_API size_t dynconv_attn_decode_workspace_bytes(const dynconv_attn_decode_desc *desc);

/* One serving step: the `tokens` new tokens of each sequence are rotated, appended to the
 * caches and attend to them.  With L = lens[b] tokens already cached,
 *   - token m stands at position L + depth(m), depth(m) = the number of its ancestors; q and k
 *     are rotated there (rope_dim > 0);
 *   - k (rotated, rounded to the storage dtype) and v go to rows L + m of the caches;
 *   - o[b, m] = softmax attention of q[b, m] over rows 0 .. L - 1 and the rows L + j of its
 *     ancestors j and of itself.
 * lens is read, not advanced: the caller adds the tokens it keeps.
 *   q [batch * tokens, heads * head_dim], k and v [batch * tokens, kv_heads * head_dim],
 *   o like q; rows ordered by sequence, then token
 *   k_cache, v_cache [batch, kv_heads, max_len, head_dim], updated in place
 *   lens       DEVICE int32 [batch].  A negative entry marks an idle slot: its o rows are
 *              zero and its caches are left as they are.
 *   ancestors  nullable DEVICE uint64 [batch, tokens]: bit j of entry m set where token m sees
 *              drafted token j (its own bit included; an entry may be 0: it then sees the cached
 *              rows only, and its o is zero where there are none).  depth(m) counts the bits
 *              other than m.  NULL: token m sees tokens 0 .. m (a chain).
 * Rows of the cache at L + tokens and beyond are not written.  They may be read, whole tiles at a
 * time, up to max_len, so nothing may write to them meanwhile; what they and masked rows hold
 * (infinities and NaN among it) does not reach o.
 * Errors: DYNCONV_ERR_INVALID, _UNSUPPORTED, _WORKSPACE, _CUDA; L + tokens above max_len, or a
 * position at or beyond rope_max_pos, raises the device check and the sequence is treated as idle. */
DYNCONV_API dynconv_status dynconv_attn_decode(const dynconv_attn_decode_desc *desc, const void *q, const void *k,
                                               const void *v, void *k_cache, void *v_cache, const int32_t *lens,
                                               const uint64_t *ancestors, void *o, void *ws, size_t ws_bytes,
                                               void *stream);

#ifdef __cplusplus
}
#endif

#endif /* DYNCONV_ATTN_H */
