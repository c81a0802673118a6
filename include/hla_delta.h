/*
 * hla_delta.h - C ABI of the gated delta rule and of the group norm that stands around it.
 *
 * Part of libhla.so; status codes, element types, streams, memory ownership and error
 * behaviour are those of hla.h.  The rule's workspaces begin with a device status word as those do (a
 * call clears it, and none of these kernels has a wait that could run out); the norm's holds sums only.
 *
 * Gated delta rule.  Every value head keeps a matrix S [d][dv] (fp32).  Token t with query q_t,
 * key k_t, value v_t, log decay g_t and write strength beta_t does
 *     S <- exp(g_t) S
 *     S <- S + beta_t k_t (v_t - S^T k_t)^T
 *     o_t = scale * S^T q_t
 *
 * Layout.  With HLA_BHTD: q, k [B][Hk][T][d]; v, o [B][H][T][dv]; g, beta [B][H][T].  With
 * HLA_BTHD the head and time axes change places: q, k [B][T][Hk][d]; v, o [B][T][H][dv]; g, beta
 * [B][T][H].  All contiguous.  q, k, v, o (and dout, dq, dk, dv) share one type, HLA_F32 or
 * HLA_BF16; g, beta, states and their gradients are fp32.  H is a multiple of Hk: value head h
 * uses query/key head h / (H / Hk).  States are [B][H][d][dv].  Base addresses are 16-byte
 * aligned (g, beta, lengths: 4-byte).
 *
 * Supported shapes.  d and dv each in {32, 64, 128}; 1 <= T <= 2^31 - 64; B, Hk, H >= 1; B*H <= 2^24,
 * B*H*T < 2^31.  Anything else returns HLA_ERR_UNSUPPORTED or HLA_ERR_SHAPE before any launch.
 * Outputs must not overlap inputs or one another, except where a call says so.
 *
 * Padded batches.  lengths: NULL, or device int [B]; sequence b then has min(max(lengths[b], 0), T)
 * tokens.  What stands in the rows behind a sequence's end is not used (it may be NaN); the
 * outputs and gradients of those rows are written as zero, and the state is the one after the
 * last token (state_in itself where there is none).
 *
 * Values.  g below -120 (-inf too) counts as -120, whose exp is zero in fp32, and so starts the head
 * anew at that token.  Positive g are allowed while their sums over 64 neighbouring tokens stay below
 * 88 (exp of it is the largest fp32); decays (g <= 0) always do.
 * A NaN or an infinity in a live token, or one that the recurrence comes to there, leaves the outputs of the
 * tokens before it as they are without it, and one in v the outputs and the state of the other columns;
 * from there on everything is NaN (one in q: that token's output only).  fp32 values are to stay below bf16's
 * largest, 3.39e38.  Gradients: everything of that value head, and of its key head, may be NaN then.
 */
#ifndef HLA_DELTA_H_
#define HLA_DELTA_H_

#include "hla.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { HLA_BHTD = 0, HLA_BTHD = 1 } hla_layout_t;

/* Version of this header's ABI (bumped on any signature change or addition). */
int hla_delta_abi_version(void);

/* Bytes of device workspace a forward call needs, or 0 when the request is invalid or
 * unsupported.  The size does not depend on the layout, on lengths or on the states. */
size_t hla_delta_workspace_bytes(hla_dtype_t dtype, int B, int Hk, int H, int T, int d, int dv);

/* Kernels one forward call enqueues, or 0.  Same arguments. */
int hla_delta_kernel_launches(hla_dtype_t dtype, int B, int Hk, int H, int T, int d, int dv);

/*
 * Forward over a whole sequence (training, prefill).
 *   state_in:  [B][H][d][dv], the state before the first token, or NULL for zeros.
 *   state_out: the state after the last token, or NULL when it is not wanted.  May be state_in.
 *   o:         written for every row (see "Padded batches").
 */
hla_status_t hla_delta_forward(const void* q, const void* k, const void* v, const float* g, const float* beta,
                               const float* state_in, const int* lengths, void* o, float* state_out, int B,
                               int Hk, int H, int T, int d, int dv, hla_dtype_t dtype, hla_layout_t layout,
                               float scale, void* workspace, size_t workspace_bytes, void* stream);

/* Decode: one token of every sequence.  q, k [B][Hk][d], v, o [B][H][dv], g, beta [B][H];
 * advances state [B][H][d][dv] in place.  One kernel, no workspace. */
hla_status_t hla_delta_step(float* state, const void* q, const void* k, const void* v, const float* g,
                            const float* beta, void* o, int B, int Hk, int H, int d, int dv, hla_dtype_t dtype,
                            float scale, void* stream);

/*
 * Gradients of sum(o * dout) + sum(state_out * dstate_out) for the forward call of the same q, k,
 * v, g, beta, state_in, lengths and scale (recomputed: nothing of the forward call is kept).
 *   dout, dq, dk, dv_out: typed and laid out like o, q, k, v; dq and dk of a shared key head are the
 *     sums over its value heads.  dg, dbeta: like g.  Rows behind a sequence's end get zeros.
 *   dstate_out: [B][H][d][dv], or NULL for zeros.  dstate_in: the gradient at state_in, or NULL when
 *     it is not wanted.
 * The workspace holds about 1.6 kB a token and head at d = dv = 64 (bf16).  A fixed order of sums:
 * the same inputs give the same bits.
 */
size_t hla_delta_backward_workspace_bytes(hla_dtype_t dtype, int B, int Hk, int H, int T, int d, int dv);
int hla_delta_backward_kernel_launches(hla_dtype_t dtype, int B, int Hk, int H, int T, int d, int dv);
hla_status_t hla_delta_backward(const void* q, const void* k, const void* v, const float* g, const float* beta,
                                const float* state_in, const int* lengths, const void* dout,
                                const float* dstate_out, void* dq, void* dk, void* dv_out, float* dg, float* dbeta,
                                float* dstate_in, int B, int Hk, int H, int T, int d, int dv, hla_dtype_t dtype,
                                hla_layout_t layout, float scale, void* workspace, size_t workspace_bytes,
                                void* stream);

/*
 * Group norm with an activation over channels-last rows, each position by itself (the norm of a
 * linear-attention layer's heads: groups = heads).  x is [rows][C]; a group is C / groups
 * neighbouring channels of one row:
 *     n = (x - m) / sqrt(mean((x - m)^2) + eps),  m = mean(x) with HLA_NORM_CENTER, else 0
 *     z = n * weight + bias        (weight, bias: fp32 [C]; NULL: 1 and 0)
 *     y = act(z), or z * act(gate) when gate [rows][C] is given
 * act is x / (1 + exp(-x)) with HLA_NORM_SILU, else the identity.  x, gate, y, dy, dx, dgate share
 * one type (HLA_F32 or HLA_BF16); statistics and sums are fp32.  C / groups <= 512; rows * C < 2^40,
 * rows * groups < 2^33, rows < 2^31.  16-byte aligned (weight, bias and their gradients: 4-byte).  y may be x or gate.
 */
#define HLA_NORM_CENTER 1
#define HLA_NORM_SILU 2

hla_status_t hla_group_norm_forward(const void* x, const void* gate, const float* weight, const float* bias,
                                    void* y, long long rows, int C, int groups, hla_dtype_t dtype, float eps,
                                    int flags, void* stream);

/* Gradients of sum(y * dy).  dgate: required with a gate (NULL without); dweight, dbias: fp32 [C],
 * each may be NULL when it is not wanted.  Workspace: hla_group_norm_backward_workspace_bytes()
 * (partial column sums; needed when dweight or dbias is wanted).  Sums are taken in a fixed order. */
size_t hla_group_norm_backward_workspace_bytes(hla_dtype_t dtype, long long rows, int C, int groups);
hla_status_t hla_group_norm_backward(const void* x, const void* gate, const float* weight, const float* bias,
                                     const void* dy, void* dx, void* dgate, float* dweight, float* dbias,
                                     long long rows, int C, int groups, hla_dtype_t dtype, float eps, int flags,
                                     void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* HLA_DELTA_H_ */
