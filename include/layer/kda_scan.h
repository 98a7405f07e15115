/*
 * kda_scan.h -- C ABI of the gated linear recurrence over long packed
 * sequences and its backward pass on B200 (sm_100a), library libkda_layer.so.
 *
 * The operation is the recurrence of kda_decode.h over whole sequences: per
 * sequence n and value head h, over its tokens t in order, on the fp32 state
 * S[K][V]:
 *
 *     S   <- Diag(exp(g[t,h,:])) S
 *     r   <- v[t,h,:] - S^T k[t,h,:]
 *     S   <- S + beta[t,h] k[t,h,:] r^T
 *     out[t,h,:] <- bf16(scale * S^T q[t,h,:])
 *
 * from an initial state to a final state.  kda_scan computes it for serving
 * (packed prompts, states in slots) and training; kda_scan_backward the
 * gradients of a loss with respect to q, k, v, g, beta and the initial states,
 * given those with respect to out and the final states.  Single tokens are
 * kda_decode's.
 *
 * Sequences.  Dense: cu_seqlens NULL, N sequences of T tokens, token t of
 * sequence n in row n*T + t.  Packed: cu_seqlens (device int32 [N+1],
 * non-decreasing from >= 0 to <= T), T the number of rows, sequence n in rows
 * [cu_seqlens[n], cu_seqlens[n+1]); lengths may be 0.  Rows outside every
 * sequence are neither read nor written.  Offsets outside [0, T] or decreasing
 * are clamped: they never make an access out of range, but results of the
 * sequences concerned are then undefined.
 *
 * Layouts.  q, k bf16 [rows, HV, K]; v, out bf16 [rows, HV, V]; g fp32
 * [rows, HV, K] (log-decay, normally <= 0; growing ones: see Accuracy); beta
 * fp32 [rows, HV].  Every one has a row stride in elements (>= the row's width),
 * heads dense inside a row: q, k and v may be slices of one packed row buffer,
 * and so may the gradients.
 * States fp32 [N, HV, K, V], dense.  With slot_idx (device int32 [N],
 * kda_scan only) sequence n's state is block slot_idx[n] of [num_slots, HV, K,
 * V] pools instead; a slot < 0 or >= num_slots makes the sequence inactive
 * (zero outputs, no state touched), active slots are distinct.
 * initial_state NULL starts from zeros, final_state NULL drops the result;
 * the two may be the same buffer (a pool updated in place).
 *
 * Supported sizes: K = V = 128, HV >= 1, N, T >= 0.  Alignment: q, k, v, out,
 * d_out, dq, dk, dv 16 bytes with strides that are multiples of 8 elements;
 * workspace and states 16 bytes; g, beta, dg, dbeta, cu_seqlens, slot_idx 4.
 *
 * Accuracy.  Operands are pairs of fp16 or tf32 numbers (22 bits) with one
 * power-of-two scale for a chunk (64 tokens) and head, accumulated in fp32, with
 * decays accumulated in pairs of fp32; bf16 results are rounded once.  A value
 * keeps 2^-22 of itself or 2^-39 of the largest one under its scale, whichever
 * is more, so fp32 results are as exact as fp32 relative to the largest of their
 * chunk and head.  Apart from it:
 *   - tokens, or value columns of the same 32, more than 2^17 below that
 *     largest lose bits;
 *   - in dq, dk, dg and dbeta, which sum over the value columns, so does what
 *     columns of initial states or values more than 2^9 below the largest add;
 *   - growth (g > 0) is a spread of magnitudes within its chunk: up to 2^16 over
 *     64 tokens keeps every token's own accuracy, more takes it from those that
 *     are left behind.
 * Range: values, states, gradients and what decays make of them, chunk by chunk,
 * with largest magnitudes of 0 or 2^-80 to 2^100, and products of two (a state
 * and its gradient) inside fp32's.  Below, bits and then values are lost; above
 * lie infinities and NaN.
 * An infinity or NaN in a sequence's inputs makes that sequence's and head's
 * outputs and final state undefined from its chunk on, and all gradients of that
 * sequence and head, nothing else; but a log-decay of -inf, like any below -1e4,
 * is a decay of zero.
 *
 * Workspace.  Caller-owned device memory of kda_scan_workspace_bytes bytes; the
 * library allocates nothing.  With save = 1 (and a workspace sized for
 * training) kda_scan leaves in it what kda_scan_backward reads: the same
 * inputs, the untouched workspace and saved = 1 then run the backward pass
 * alone; with saved = 0 kda_scan_backward recomputes the forward pass into the
 * workspace first (any contents).  Calls that share a workspace must be
 * ordered.  Its first int32 is an error word: the kernels' waits for their
 * copies are bounded, and one that ever gives up stores 1 there and leaves
 * results undefined; the library never clears it.
 *
 * Execution: kda_scan enqueues 2 kernels (4 where long sequences of few heads
 * are walked in segments), kda_scan_backward 2 (4), and those of the forward pass
 * before them with saved = 0, on `stream`; no host synchronisation; can be
 * captured in a CUDA graph.
 * Results do not depend on the launch's timing (no atomics on data).
 *
 * Errors: as in kda_decode.h, nothing is enqueued unless KDA_OK is returned.
 * KDA_ERR_ALIAS: an output overlaps an input, another output or the workspace
 * (rows of one packed buffer with equal strides and disjoint columns do not).
 */
#ifndef KDA_SCAN_H
#define KDA_SCAN_H

#include "../kda_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
    const void *q;      int64_t q_row_stride;
    const void *k;      int64_t k_row_stride;
    const void *v;      int64_t v_row_stride;
    const float *g;     int64_t g_row_stride;
    const float *beta;  int64_t beta_row_stride;
    const int32_t *cu_seqlens;
    const float *initial_state;
    float *final_state;          /* kda_scan_backward ignores it */
    const int32_t *slot_idx;     /* kda_scan_backward: must be NULL */
    int64_t num_slots;
    void *out;          int64_t out_row_stride;   /* kda_scan_backward ignores it */
    void *workspace;    int64_t workspace_bytes;
    int64_t N, T, HV, K, V;
    float scale;
    int32_t save;                /* kda_scan: keep what the backward pass reads */
} kda_scan_args;

typedef struct {
    const void *d_out;  int64_t d_out_row_stride;
    const float *d_final_state;  /* NULL: zeros */
    void *dq;           int64_t dq_row_stride;
    void *dk;           int64_t dk_row_stride;
    void *dv;           int64_t dv_row_stride;
    float *dg;          int64_t dg_row_stride;
    float *dbeta;       int64_t dbeta_row_stride;
    float *d_initial_state;      /* NULL: not wanted */
    int32_t saved;               /* the workspace holds this call's forward pass */
} kda_scan_grads;

/* Bytes of workspace (0 when there is nothing to do, -1 for unsupported or
 * negative sizes).  packed: cu_seqlens will be set; training: for save = 1 and
 * for kda_scan_backward. */
KDA_API int64_t kda_scan_workspace_bytes(int64_t N, int64_t T, int32_t packed, int64_t HV, int64_t K, int64_t V,
                                         int32_t training);

KDA_API kda_status kda_scan(const kda_scan_args *args, kda_stream_t stream);

/* args: the forward call's. */
KDA_API kda_status kda_scan_backward(const kda_scan_args *args, const kda_scan_grads *grads, kda_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_SCAN_H */
