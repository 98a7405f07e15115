/*
 * kda_qk.h -- C ABI of the per-head norm of queries and keys with the position
 * rotation in the same pass, and its gradients, on B200 (sm_100a), library
 * libkda_layer.so.  It produces the q and k that kda_decode, kda_prefill and
 * kda_scan take.
 *
 * Per row and head, on the D components x:
 *
 *     y = x                                         KDA_QK_NORM_NONE
 *     y = x / sqrt(sum(x^2) + eps) * weight         KDA_QK_NORM_L2
 *     y = x / sqrt(mean(x^2) + eps) * weight        KDA_QK_NORM_RMS
 *
 * (weight [D] shared by the heads, NULL: ones; not with KDA_QK_NORM_NONE), then
 * the first `rot` components are turned in pairs (a, b) by the row's angles:
 *
 *     a' = rope_scale (a cos - b sin),  b' = rope_scale (a sin + b cos),
 *     angle of pair i = position * inv_freq[i],
 *
 * pair i being components i and i + rot/2 (halves) or 2i and 2i + 1
 * (interleaved).  The remaining D - rot components keep y.  Frequencies scaled
 * for long contexts are the caller's inv_freq and rope_scale.
 *
 * Layouts.  x, y, dy, dx bf16 [rows, heads, D], a row stride in elements
 * (>= heads * D), heads dense inside a row: q and k may be slices of one packed
 * row buffer.  weight bf16 [D], dweight fp32 [D]; positions int32 or int64
 * [rows], any sign; inv_freq fp64 [rot/2].  k may be absent (heads 0).  An
 * output may be exactly its own input (y = x forward, dx = dy backward, equal
 * strides); any other overlap is refused.
 *
 * Supported sizes: D a multiple of 8 from 8 to 256, rot a multiple of 16 from 0
 * to D, rows >= 0, heads from 0 to 4096.  Alignment: x, y, dy, dx, weight, workspace 16
 * bytes and strides multiples of 8 elements; inv_freq, int64 positions 8, the
 * rest 4.
 *
 * Accuracy.  Sums and products in fp32, angles in fp64 (reduced to one turn
 * before cos and sin, so far positions keep their angle), outputs rounded once
 * to bf16; dweight is summed in fp32 per thread and fp64 across blocks, in a
 * fixed order.  A head's sum of squares has to stay in fp32's range: components
 * below 2^60 (a sum beyond it makes the head zero), and one above 2^-60 or an eps
 * above 2^-120.  An infinity or NaN stays in its row and head (and in dweight).
 *
 * Execution: forward 1 kernel; backward 1, or 2 with a dweight.  Enqueued on
 * `stream`, no allocation, no host synchronisation, capturable.  The workspace
 * (kda_qk_workspace_bytes, only with a dweight) is the caller's; calls that
 * share one must be ordered.
 *
 * Errors: as in kda_decode.h, nothing is enqueued unless KDA_OK is returned.
 */
#ifndef KDA_QK_H
#define KDA_QK_H

#include "../kda_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

#define KDA_QK_NORM_NONE 0
#define KDA_QK_NORM_L2 1
#define KDA_QK_NORM_RMS 2

typedef struct {
    const void *x;   int64_t x_row_stride;
    void *y;         int64_t y_row_stride;    /* forward: the output */
    const void *dy;  int64_t dy_row_stride;   /* backward */
    void *dx;        int64_t dx_row_stride;   /* backward */
    const void *weight;
    float *dweight;                           /* backward; NULL: not wanted */
    int64_t heads;
} kda_qk_tensor;

typedef struct {
    kda_qk_tensor q, k;
    int64_t rows, D, rot;
    const void *positions;       /* NULL with rot = 0 */
    const double *inv_freq;      /* NULL with rot = 0 */
    int32_t positions_64;        /* positions are int64 (else int32) */
    int32_t norm, interleaved;
    float eps, rope_scale;
    void *workspace; int64_t workspace_bytes;
} kda_qk_args;

/* Bytes of workspace of the backward pass with a dweight (-1: unsupported D). */
KDA_API int64_t kda_qk_workspace_bytes(int64_t D);

KDA_API kda_status kda_qk_norm_rope(const kda_qk_args *args, kda_stream_t stream);
KDA_API kda_status kda_qk_norm_rope_backward(const kda_qk_args *args, kda_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_QK_H */
