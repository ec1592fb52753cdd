/*
 * losses.h — C ABI of the losses over a vocabulary on one GB300 GPU (sm_103a).
 *
 * Operation.  The logits x[batch, seq, vocab] of a language model are reduced
 * to a loss, and the gradient of the loss with respect to the logits is
 * written in the same call (over the logits themselves, if the caller wants).
 * The optimizer steps of this library take the gradients that follow from it.
 * With z = x / temperature, q = softmax(z) and y a token's target:
 *     logp = z[y] - ln sum_j exp(z[j])
 *
 *   token_logprobs   logp of every token, and the backward pass
 *                    dx[j] = g (1[j = y] - q[j]) / temperature
 *   policy           r = exp(logp - old);  d = ref - logp
 *                    l = -min(r A, clip(r, 1 - clip_low, 1 + clip_high) A)
 *                        + kl_coef (exp(d) - d - 1)
 *                    loss = sum over tokens of w l;  w = 1 / (number of tokens
 *                    whose target is not ignored), or the caller's weights.
 *                    r A counts for the gradient where r A <= clip(r) A.
 *   preference       D = sum (or mean) over a sequence of logp - ref;
 *                    h = D(chosen) - D(rejected), and per pair
 *       SIGMOID      -(1 - e) ln s(beta h - margin) - e ln s(margin - beta h),
 *                    s the logistic function, e = label_smoothing
 *       HINGE        max(0, 1 + margin - beta h)
 *       SQUARED      (h - 1 / (2 beta) - margin)^2
 *                    loss = mean over the pairs.
 *   distill          p[k] the teacher's probabilities of top_k entries:
 *                    softmax over the entries of t[k] / temperature, or, with
 *                    the teacher's ln sum exp(t / temperature) over its whole
 *                    vocabulary, p[k] = exp(t[k] / temperature - lse) and a
 *                    rest u = max(0, 1 - sum p) that stands for all other words
 *                    (0 where every word is listed):
 *                    l = T^2 [ sum p[k] (ln p[k] - ln q[k])
 *                              + u (ln u - ln sum_{j not listed} q[j]) ]
 *                    loss = sum over tokens of w l, w as above with `mask`.
 *
 * Tokens.  A token is a pair (b, s), b < batch, s < seq; every per-token
 * argument has element strides of its own over b and s (0 repeats a value),
 * and the innermost stride of logits and gradient is 1.  Any alignment of the
 * element's own size is accepted.  2D logits are batch = 1.
 *
 * Tokens that do not count.  Where the target is ignore_index (or mask is 0)
 * the logits may hold anything (rows of up to 1024 vectors of 16 bytes are read
 * all the same, by policy and distill, longer ones are not), the token's loss
 * and logp are 0 and its gradient row is written as 0.  With no token left the loss is 0.  A token whose
 * teacher lists nothing (every id -1) counts, with loss and gradient 0.
 *
 * Values.  Logits of -inf have probability 0; a term whose factor is 0 counts
 * as 0 beside the infinite logarithm of one.  A row with NaN or +inf, or
 * with nothing but -inf, answers NaN in its own values, and so does a row
 * whose target (or a listed teacher id) lies outside the vocabulary, and one
 * whose teacher lists an id twice: bad data shows in the loss and reads or
 * writes nothing out of range.  A teacher's rest for which the student leaves
 * nothing (no unlisted logit above -inf) is a loss of inf.  Of the 16 bytes that hold a row's first or last
 * value all are read where they lie within the logits' extent.
 *
 * Logits are fp32 or bf16 and the gradient has their type; everything between
 * is fp32 (sums over tokens with compensation), and gradients are rounded
 * once.  The sums run in a fixed order: equal inputs give equal bits.
 *
 * Every call only launches kernels on the caller's stream: it allocates
 * nothing on the device, waits for nothing and may be captured in a graph.
 * Every wait inside a kernel is bounded; if one runs out, which no input
 * brings about, the call ends with a loss of NaN.  The workspace
 * needs no initialisation.  Calls on different streams may run at the same
 * time if each has its own workspace.  Status codes, dtypes and the message
 * slot are shared with adafactor.h; every argument check runs before the
 * first CUDA call, so a failing call changes nothing.
 */
#ifndef MEO_LOSSES_H
#define MEO_LOSSES_H

#include <stddef.h>
#include <stdint.h>

#include "adafactor.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Index types of targets, teacher ids and sequence offsets. */
#define LOSS_INT32 0
#define LOSS_INT64 1

#define LOSS_MAX_TOP_K 1024

typedef struct loss_logits {
    const void* p;
    int32_t dtype;               /* ADAF_FLOAT32 or ADAF_BFLOAT16            */
    int64_t batch, seq, vocab;   /* batch * seq <= 2^30, 1 <= vocab <= 2^21  */
    int64_t stride_b, stride_s;  /* elements, >= 0                           */
    double temperature;          /* > 0                                      */
} loss_logits;

/* One value a token: p[b * stride_b + s * stride_s]; p == NULL where optional. */
typedef struct loss_rows {
    const void* p;
    int64_t stride_b, stride_s;
} loss_rows;

typedef struct loss_targets {
    loss_rows rows;
    int32_t dtype;               /* LOSS_INT32 or LOSS_INT64                 */
    int64_t ignore_index;
} loss_targets;

/* Gradient of the logits, in their dtype.  p == NULL: the loss alone.  p may
 * be the logits' own p with the same strides (the gradient takes their
 * place); any other overlap is an error, and so are rows that overlap. */
typedef struct loss_grad {
    void* p;
    int64_t stride_b, stride_s;
    double scale;                /* multiplies the gradient, not the loss    */
} loss_grad;

typedef struct loss_policy_args {
    loss_rows advantages;        /* fp32                                     */
    loss_rows old_logp;          /* fp32; NULL: r = 1 (first step on policy) */
    loss_rows ref_logp;          /* fp32; NULL only with kl_coef = 0         */
    loss_rows weights;           /* fp32; NULL: the mean over counted tokens */
    double clip_low, clip_high;  /* 0 <= clip_low <= 1, clip_high >= 0       */
    double kl_coef;              /* >= 0                                     */
} loss_policy_args;

#define LOSS_PREFERENCE_SIGMOID 0
#define LOSS_PREFERENCE_HINGE 1
#define LOSS_PREFERENCE_SQUARED 2

typedef struct loss_preference_args {
    loss_rows ref_logp;          /* fp32 per token; NULL: 0                  */
    int64_t pairs;               /* sequence i < pairs was preferred to
                                    sequence pairs + i                       */
    const void* seq_offsets;     /* device [2 pairs + 1], non-decreasing from
                                    0 to seq, with batch = 1: sequence n has
                                    the tokens offsets[n] .. offsets[n + 1];
                                    a pair with a bad offset answers NaN (its
                                    loss and both rewards; a bad sequence has
                                    no tokens to give a gradient to).
                                    NULL: batch = 2 pairs, one per sequence  */
    int32_t offsets_dtype;       /* LOSS_INT32 or LOSS_INT64                 */
    int32_t kind;                /* LOSS_PREFERENCE_*                        */
    int32_t average;             /* non-zero: D is a mean over the counted
                                    tokens (0 for a sequence without any)    */
    double beta;                 /* > 0                                      */
    double label_smoothing;      /* 0 <= e < 0.5; SIGMOID only               */
    double margin;               /* finite                                   */
} loss_preference_args;

typedef struct loss_distill_args {
    const void* ids;             /* [batch, seq, top_k], innermost stride 1  */
    int32_t ids_dtype;           /* -1 marks an entry that is not there      */
    int64_t ids_stride_b, ids_stride_s;
    const void* values;          /* teacher logits of the ids, same layout   */
    int32_t values_dtype;        /* ADAF_FLOAT32 or ADAF_BFLOAT16            */
    int64_t values_stride_b, values_stride_s;
    int32_t top_k;               /* 1 .. LOSS_MAX_TOP_K                      */
    loss_rows lse;               /* fp32; NULL: renormalise over the entries */
    loss_rows mask;              /* uint8; NULL: every token counts          */
    loss_rows weights;           /* fp32; NULL: the mean over counted tokens */
} loss_distill_args;

/* Bytes of workspace of loss_policy, loss_distill (pairs = 0) and
 * loss_preference for batch * seq tokens. */
adaf_status loss_workspace_size(int64_t tokens, int64_t pairs, size_t* bytes);

/* logp [batch * seq] fp32 and, if not NULL, stats [batch * seq][2] fp32: the
 * row's largest logit and sum exp((x - largest) / temperature) as the backward
 * pass takes them (the sum is relative to a rounded exponent, so no value to
 * compute with).  Stats of ignored tokens are 0. */
adaf_status loss_token_logprobs(const loss_logits* x, const loss_targets* y, float* logp, float* stats, void* stream);

/* grad from the stats of the forward pass on the same logits, and grad_logp
 * (fp32 per token). */
adaf_status loss_token_logprobs_backward(const loss_logits* x, const loss_targets* y, const float* stats,
                                         const loss_rows* grad_logp, const loss_grad* grad, void* stream);

/* loss [1]; logp, token_loss [batch * seq] fp32 (each may be NULL). */
adaf_status loss_policy(const loss_logits* x, const loss_targets* y, const loss_policy_args* args,
                        const loss_grad* grad, float* loss, float* logp, float* token_loss, void* workspace,
                        size_t workspace_bytes, void* stream);

/* loss [1], pair_loss [pairs], rewards [2 pairs] (beta D), logp [batch * seq];
 * the last three may be NULL. */
adaf_status loss_preference(const loss_logits* x, const loss_targets* y, const loss_preference_args* args,
                            const loss_grad* grad, float* loss, float* pair_loss, float* rewards, float* logp,
                            void* workspace, size_t workspace_bytes, void* stream);

/* loss [1], token_loss [batch * seq] (may be NULL). */
adaf_status loss_distill(const loss_logits* x, const loss_distill_args* args, const loss_grad* grad, float* loss,
                         float* token_loss, void* workspace, size_t workspace_bytes, void* stream);

/* Testing hook: while on, the bulk copies of loss_policy and loss_distill calls
 * of the calling thread are expected but not made, so that the kernel's waits
 * for them run out (after about a second each); the loss of such a call is NaN.
 * Other threads' calls are as ever. */
void loss_debug_stall_copies(int32_t on);

/* Per-kernel CUDA-event timing, as in adafactor.h. */
adaf_status loss_profile_enable(int32_t on);
adaf_status loss_profile_read(double* ms, int64_t* launches, int32_t n);
int32_t loss_num_kernels(void);
const char* loss_kernel_name(int32_t k);

#ifdef __cplusplus
}
#endif

#endif /* MEO_LOSSES_H */
