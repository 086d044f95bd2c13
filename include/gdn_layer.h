/*
 * gdn_layer.h -- C ABI of the operators that serve a Gated DeltaNet layer around the chunked prefill
 * of kkt.h: what produces the delta rule's q, k, v, g and beta from a layer's projections, the delta
 * rule token by token over a pool of states, the norms before and behind it, and the copying and
 * clearing of pool slots.  Same library (libkkt.so), status codes and conventions as kkt.h.
 *
 * Conventions: every pointer is a device pointer owned by the caller; the library allocates nothing;
 * calls are asynchronous on `stream` and never synchronise the host; tensors are row-major and
 * contiguous (but for those with a stride of their own) and 16-byte aligned, fp32 vectors and index
 * arrays 4-byte aligned.  Invalid arguments
 * return a nonzero kkt_status without launching.  What only the device can see (a malformed
 * cu_seqlens: KKT_ERR_SEQLENS; a slot at or past num_slots: KKT_ERR_INDEX) is recorded in the status
 * word that kkt_device_status() reads; the kernels leave the sequences concerned alone.
 *
 * Sequences: cu_seqlens == NULL: N sequences of T tokens, tensors [N, T, ...]; else int32[N + 1]
 * offsets into a packed token axis of T tokens, tensors [1, T, ...].
 *
 * Slots: a pool holds one state per slot, [num_slots, ...].  slots[n] (int32) is the slot of sequence
 * n; NULL is the identity (N <= num_slots).  A negative slot is no slot: reading it gives a zero
 * state, and nothing is written to it (the padding rows of a captured batch).  No two sequences of a
 * call may write one slot, and none may write a slot that another one reads: the sequences run in no
 * particular order.
 */
#ifndef GDN_LAYER_H_
#define GDN_LAYER_H_

#include "kkt.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Type of a norm's output. */
enum {
    GDN_OUT_BF16 = 0,
    GDN_OUT_F32 = 1,
    GDN_OUT_E4M3 = 2 /* 8 bits (4 exponent, 3 mantissa, largest value 448) with fp32 scales */
};

/*
 * gdn_recurrent_fwd -- the gated delta rule, one token after the other: the form of
 * gdn_chunk_state_fwd's recurrence for decode steps, drafted tokens and other short runs.  For every
 * sequence and value head, from the state S (dk x dv) of the sequence's slot,
 *
 *   S <- e^{g_t} S;   d = beta_t (v_t - S^T k_t);   S <- S + k_t d^T;   o_t = scale S^T q_t,
 *
 * and the state after the last token goes back to the pool.
 *
 *   q, k    [.., Hk, dk]   io_dtype (KKT_IO_BF16 or KKT_IO_F32); Hv a multiple of Hk: value head h
 *                          uses key head h / (Hv / Hk)
 *   v, o    [.., Hv, dv]   io_dtype (o: output)
 *   beta, g [.., Hv]       fp32; g NULL: no gate
 *   state   [num_slots, Hv, dk, dv]  fp32 (state_dtype KKT_IO_F32) or bf16 (KKT_IO_BF16), updated in
 *                          place.  Kept in fp32 within a call; a bf16 pool is rounded once, when the
 *                          call writes it back
 *   slots, slots_out       where each sequence's state is read and written; slots_out NULL: where it
 *                          was read
 *   dk, dv  64 or 128
 * A sequence without tokens keeps its state (copied, where slots_out differs from slots).
 */
int gdn_recurrent_fwd(const void *q, const void *k, const void *v, const float *beta, const float *g,
                      const int32_t *cu_seqlens, int N, int T, int Hk, int Hv, int dk, int dv, float scale,
                      int io_dtype, void *state, int state_dtype, int num_slots, const int32_t *slots,
                      const int32_t *slots_out, void *o, struct CUstream_st *stream);

/*
 * gdn_prep_fwd -- from a layer's projections to the delta rule's inputs.  With the channels of a
 * token packed as [Hk dk | Hk dk | Hv dv] = [q | k | v], D of them:
 *
 *   y_t = silu(bias + sum_{j < taps} weight[:, j] x_{t - taps + 1 + j}),   x before the sequence's
 *         first token taken from its convolution state (the last taps - 1 inputs, oldest first);
 *   q, k = y / sqrt(sum over the head of y^2 + eps);   v = y;
 *   beta = 1 / (1 + e^-b);   g = -e^{A_log} softplus(a + dt_bias).
 *
 *   x       [.., D]     io_dtype          weight [D, taps], bias [D] (or NULL)   io_dtype
 *   a, b    [.., Hv]    io_dtype          A_log, dt_bias [Hv]   fp32
 *   x_stride, a_stride, b_stride          values from a token's to the next one's: D, Hv and Hv, or
 *           more for slices of a larger tensor, as one product for all projections gives them (below
 *           2^31; x_stride a multiple of 16 bytes; a, b and the weights aligned to their type only)
 *   conv_state [num_slots, taps - 1, D]   io_dtype, updated in place to the last taps - 1 inputs
 *   q, k    [.., Hk, dk] or, with expand, [.., Hv, dk] (each key head written once for every value
 *           head that uses it, as kkt_solve_fwd takes them);   v [.., Hv, dv];   io_dtype, outputs
 *   g, beta [.., Hv]    fp32, outputs
 *   dk = dv = 64 or 128;   taps 2, 3 or 4
 */
int gdn_prep_fwd(const void *x, int64_t x_stride, const void *weight, const void *bias, const void *a,
                 int64_t a_stride, const void *b, int64_t b_stride, const float *A_log, const float *dt_bias,
                 const int32_t *cu_seqlens, int N, int T, int Hk, int Hv, int dk, int dv, int taps, float eps,
                 int expand, int io_dtype, void *conv_state, int num_slots, const int32_t *slots, void *q, void *k, void *v, float *g, float *beta, struct CUstream_st *stream);

/*
 * add_rms_norm_fwd -- h = x + residual (h = x where residual is NULL), residual_out = h, and
 *   y = h / sqrt(mean(h^2) + eps) * weight    over rows of `dim`.
 * The sum is normalised as it is in fp32; residual_out is its rounding to io_dtype, and may be
 * `residual` (or x) itself.  x, residual, residual_out [rows, dim], weight [dim]: io_dtype.
 * y [rows, dim]: out_dtype.  With GDN_OUT_E4M3, scales [rows, ceil(dim / group)] fp32 holds for each
 * `group` consecutive values of a row s = max|y| / 448 (at least 2^-126; 1 where they are all zero),
 * and y holds y / s.  group: 128, or 0 for one scale a row (scales [rows]).  dim 1 .. 16384.
 */
int add_rms_norm_fwd(const void *x, const void *residual, const void *weight, int64_t rows, int dim, float eps,
                     int io_dtype, int out_dtype, int group, void *y, float *scales, void *residual_out,
                     struct CUstream_st *stream);

/*
 * gated_rms_norm_fwd -- y = x / sqrt(mean(x^2) + eps) * weight * silu(z) over rows of `dim` (one head
 * of one token: dim 64 or 128).  x, z [rows, dim], weight [dim]: io_dtype; y [rows, dim]: out_dtype;
 * with GDN_OUT_E4M3, scales [rows] fp32: one for each row, as in add_rms_norm_fwd.  z_rows: 0, or z
 * is a slice of a larger tensor, z_rows rows (a token's heads) behind one another and z_stride values
 * from the first of them to the next token's (a multiple of 16 bytes, at most 2^31).
 */
int gated_rms_norm_fwd(const void *x, const void *z, int z_rows, int64_t z_stride, const void *weight,
                       int64_t rows, int dim, float eps, int io_dtype, int out_dtype, void *y, float *scales, struct CUstream_st *stream);

/* Tensors of one gdn_state_copy call. */
#define GDN_COPY_MAX_TENSORS 64

/*
 * gdn_state_copy -- copies pool slots: for every tensor i < ntensors and every m < nmoves,
 *   dst[i] slot dst_slots[m]  <-  src[i] slot src_slots[m],
 * or zeros where src_slots[m] is negative or src is NULL.  A negative dst_slots[m] is skipped.
 * Forking is a source named more than once; freeing is clearing.  A slot is slot_bytes[i] consecutive
 * bytes, and slots are dst_stride[i] (src_stride[i]) bytes apart.
 *   dst, src, slot_bytes, dst_stride, src_stride   HOST arrays of ntensors (at most
 *                         GDN_COPY_MAX_TENSORS) device pointers and byte counts
 *   dst_slots, src_slots  device int32[nmoves], below dst_num_slots / src_num_slots
 * No two moves may have the same destination, and none may write a slot that another one reads: the
 * moves run in no particular order.
 */
int gdn_state_copy(void *const *dst, const void *const *src, const size_t *slot_bytes, const size_t *dst_stride,
                   const size_t *src_stride, int ntensors, const int32_t *dst_slots, const int32_t *src_slots,
                   int nmoves, int dst_num_slots, int src_num_slots, struct CUstream_st *stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_LAYER_H_ */
