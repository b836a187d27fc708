/*
 * kda_layer.h -- C ABI of the operators around the recurrence of kda.h (same library, same
 * descriptors, statuses, kda_last_error() and kda_profile_* records):
 *
 *   kda_conv, kda_conv_decode        the short causal convolution in front of the recurrence
 *   kda_qk_norm                      the per-head norm of queries and keys, and the rotation of
 *                                    positions, in one pass
 *   kda_ssm_prefill, kda_ssm_decode  the selective state space scan
 *
 * What kda.h says of tensors holds here too: device pointers owned by the caller, strides in
 * elements, unit last stride, every check on the host before anything is enqueued, no
 * synchronisation, KDA_CHECK=1 for the checks of device data.  Dense and packed layouts, zero
 * length sequences and int32 cu_seqlens [N + 1] are those of kda_prefill.  No function here
 * allocates device memory except kda_ssm_prefill's cached workspace.
 */
#ifndef KDA_LAYER_H
#define KDA_LAYER_H

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { KDA_ACT_NONE = 0, KDA_ACT_SILU = 1 };

/*
 * kda_conv -- depthwise causal convolution over each sequence's tokens:
 *     out[t, c] = act(sum_{w < W} weight[c, w] x[t - (W - 1) + w, c] + bias[c])
 * where inputs before the sequence's first token are the rows of its initial state (the W - 1
 * inputs before it, oldest first; zeros when NULL).  act: KDA_ACT_NONE or KDA_ACT_SILU,
 * silu(y) = y / (1 + e^-y).  final_state receives the last W - 1 inputs of every sequence
 * (rows of the initial state among them when the sequence is shorter than that).
 * x, out: dense [B, T, C] or packed [T, C] / [1, T, C] with cu_seqlens; bf16 or fp32 alike.
 * weight [C, W], W in 2..4, and bias [C] (or NULL): each bf16 or fp32; weight is contiguous.
 * States [N, W - 1, C], each bf16 or fp32 (x is kept exactly in x's dtype).
 * out may not overlap any input; final_state may be exactly initial_state (same view; one more small
 * launch), or must not overlap any input.  Sums in fp32, one rounding to out's dtype.  Rows behind
 * cu[N] are not read and left as they were.
 */
kda_status_t kda_conv(const kda_tensor_t *x, const kda_tensor_t *weight, const kda_tensor_t *bias,
                      const kda_tensor_t *initial_state, const kda_tensor_t *cu_seqlens, kda_tensor_t *out,
                      kda_tensor_t *final_state, int32_t activation, void *stream);

/*
 * kda_conv_decode -- the same convolution over 1..8 tokens per request against a pool of states,
 * with kda_decode's semantics: request r runs its first n_r = num_tokens[r] tokens (clamped to
 * [0, T]; NULL: T) from pool[state_indices[r]]; a slot outside [0, P) skips the request; rows of
 * out past n_r are left as they were; update_state != 0 writes the last W - 1 inputs back.
 * x, out: [R, T, C] (out may be NULL: commit only); state_pool: [P, W - 1, C], bf16 or fp32.
 * Two requests that name one slot with update_state race (KDA_CHECK=1 refuses them).
 */
kda_status_t kda_conv_decode(const kda_tensor_t *x, const kda_tensor_t *weight, const kda_tensor_t *bias,
                             kda_tensor_t *state_pool, const kda_tensor_t *state_indices,
                             const kda_tensor_t *num_tokens, kda_tensor_t *out, int32_t update_state,
                             int32_t activation, void *stream);

enum { KDA_NORM_NONE = 0, KDA_NORM_RMS = 1, KDA_NORM_L2 = 2 };
enum { KDA_ROTARY_HALF = 0, KDA_ROTARY_INTERLEAVED = 1 };

typedef struct {
    int32_t norm;           /* KDA_NORM_*                                                        */
    float norm_eps;         /* >= 0, finite                                                      */
    int32_t rotary_layout;  /* KDA_ROTARY_*                                                      */
    int32_t rotary_offset;  /* first rotated channel, 0 .. D - rot                               */
    float rotary_scale;     /* multiplies cos and sin (long-context attention scaling)           */
} kda_qk_norm_options_t;

/*
 * kda_qk_norm -- norm and rotation of queries and keys, one read and one write of each.  For every
 * (token, head) row x of q (weight q_weight) and k (weight k_weight):
 *     KDA_NORM_RMS:  y = x / sqrt(mean(x^2) + eps) * weight
 *     KDA_NORM_L2:   y = x / sqrt(sum(x^2) + eps) * weight     (unit rows for the recurrence)
 *     KDA_NORM_NONE: y = x                                     (weights must be NULL)
 * weights fp32 [D], NULL for ones.  Then, with inv_freq (fp32 [rot / 2]) and positions (int32, one
 * per token), channels [offset, offset + rot) rotate in pairs (a, b):
 *     (a, b) -> scale * (a cos - b sin, b cos + a sin),   angle = position * inv_freq[i]
 * pair i being channels (i, i + rot / 2) of the part (KDA_ROTARY_HALF) or (2 i, 2 i + 1)
 * (KDA_ROTARY_INTERLEAVED).  Angles are formed and reduced in 64 bits, so far positions keep their
 * phase.  inv_freq NULL or empty: no rotation (positions may then be NULL).  With KDA_NORM_NONE
 * and no rotation the call is refused.
 * q, q_out: [T, Hq, D] or [B, T, Hq, D]; k, k_out: [.., Hk, D] alike, both NULL to leave k out;
 * positions: [T] or [B, T].  All of q, k and outputs bf16, or all fp32.  D a multiple of 4, at most
 * 256; base addresses and strides aligned to 4 elements.  An output may be exactly its input (in
 * place) and may overlap nothing else.
 */
kda_status_t kda_qk_norm(const kda_tensor_t *q, const kda_tensor_t *k, const kda_tensor_t *q_weight,
                         const kda_tensor_t *k_weight, const kda_tensor_t *positions, const kda_tensor_t *inv_freq,
                         kda_tensor_t *q_out, kda_tensor_t *k_out, const kda_qk_norm_options_t *opts, void *stream);

/* Optional inputs of the scan, all fp32 except z; a zero-filled struct (or NULL) means none. */
typedef struct {
    const kda_tensor_t *D;        /* [H]: adds D x to the output                                  */
    const kda_tensor_t *dt_bias;  /* [H]: added to dt                                             */
    const kda_tensor_t *z;        /* out's shape and dtype: out = y silu(z)                       */
    int32_t dt_softplus;          /* 1: the step is softplus(dt + dt_bias)                        */
    int32_t segment;              /* prefill: tokens per segment, a multiple of 32; 0 = planner's, -1 = whole sequences */
                                  /* choice, -1 = whole sequences                                 */
} kda_ssm_options_t;

/*
 * kda_ssm_prefill -- the selective state space scan: per sequence and head, over tokens in order,
 *     step_t = softplus(dt_t + dt_bias)     (or dt_t + dt_bias)
 *     S_t = e^{A step_t} S_{t-1} + step_t B_t x_t^T        S: N x P (row = state channel)
 *     y_t = S_t^T C_t + D x_t,   out = y_t silu(z_t)
 * x, z, out: dense [B, T, H, P] or packed [T, H, P] / [1, T, H, P]; dt: [.., H], x's dtype or fp32;
 * A: fp32 [H]; B, C: [.., G, N], head h reading group h / (H / G).  P and N each 64 or 128; G
 * divides H.  x, B, C, z, out all bf16, or all fp32.  States [n, H, N, P], fp32 or bf16 each; the
 * state is carried in fp32 or better in between.  A and steps finite, A step <= 0 (a growing head,
 * A step > 0, follows the same formula while a chunk grows by less than 2^96).
 * Chunks of 32 tokens run on the matrix cores.  On bf16 data products of inputs are exact, the
 * state's additive term keeps 24 bits, and the state and the products of B and C are rounded to bf16
 * where they only feed out (to 16 bits where no two workgroups share a CU).  Terms are weighted by up to 2^96 against each other, so |x B C| (and
 * their sums) may reach 2^31.  A NaN or infinity in x or dt at a token can reach the outputs of up to
 * 31 tokens before it in its sequence, never another sequence, and only its own head.
 * Rows behind cu[N] are not read and left as they were.  Token strides below 2^24 - 256 elements and
 * head strides of x and z within 2^28.
 * Uses the library's cached workspace like kda_prefill; kda_ssm_prefill_ws takes the caller's
 * (256-byte aligned, kda_ssm_workspace_size() bytes, NULL when 0), allocates nothing and can be
 * captured.  out may not overlap any input; final_state may be exactly initial_state.
 */
kda_status_t kda_ssm_prefill(const kda_tensor_t *x, const kda_tensor_t *dt, const kda_tensor_t *A,
                             const kda_tensor_t *B, const kda_tensor_t *C, const kda_tensor_t *initial_state,
                             const kda_tensor_t *cu_seqlens, kda_tensor_t *out, kda_tensor_t *final_state,
                             const kda_ssm_options_t *opts, void *stream);
kda_status_t kda_ssm_workspace_size(const kda_tensor_t *x, const kda_tensor_t *dt, const kda_tensor_t *A,
                                    const kda_tensor_t *B, const kda_tensor_t *C, const kda_tensor_t *initial_state,
                                    const kda_tensor_t *cu_seqlens, const kda_tensor_t *out,
                                    const kda_tensor_t *final_state, const kda_ssm_options_t *opts, size_t *bytes);
kda_status_t kda_ssm_prefill_ws(const kda_tensor_t *x, const kda_tensor_t *dt, const kda_tensor_t *A,
                                const kda_tensor_t *B, const kda_tensor_t *C, const kda_tensor_t *initial_state,
                                const kda_tensor_t *cu_seqlens, kda_tensor_t *out, kda_tensor_t *final_state,
                                const kda_ssm_options_t *opts, void *workspace, size_t workspace_bytes, void *stream);

/*
 * kda_ssm_decode -- the scan token by token, 1..8 tokens per request, against a pool of states
 * [P, H, N, P], fp32 or bf16, with kda_decode's semantics (state_indices, num_tokens, rows past
 * n_r, verify with update_state == 0, commit with out == NULL).  x, z, out: [R, T, H, P]; dt:
 * [R, T, H]; B, C: [R, T, G, N].  opts->segment is ignored.
 */
kda_status_t kda_ssm_decode(const kda_tensor_t *x, const kda_tensor_t *dt, const kda_tensor_t *A,
                            const kda_tensor_t *B, const kda_tensor_t *C, kda_tensor_t *state_pool,
                            const kda_tensor_t *state_indices, const kda_tensor_t *num_tokens, kda_tensor_t *out,
                            int32_t update_state, const kda_ssm_options_t *opts, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* KDA_LAYER_H */
