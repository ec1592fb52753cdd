/*
 * linear_ce.h — C ABI of the cross entropy of a linear output layer on one
 * GB300 GPU (sm_103a): the loss from the hidden states and the layer's weight,
 * and the gradients of both, without the logits.
 *
 * Operation.  With x = hidden weight^T (fp32 sums), z = x / temperature and y a
 * token's target:
 *     lse  = ln sum_j exp(z[j]),   logp = z[y] - lse
 *     loss = sum over tokens of w (z_loss lse^2 - logp)
 *     dx[j] = w (q[j] (1 + 2 z_loss lse) - 1[j = y]) / temperature,  q = softmax(z)
 *     grad_hidden = grad_scale dx weight,   grad_weight = grad_scale dx^T hidden
 * w = 1 / (number of tokens whose target is not ignore_index), or the caller's
 * weights.  Ignored tokens cost nothing but a look at their targets: the others
 * are put side by side first.  Without tokens that count the loss and the
 * gradients are 0.
 *
 * Pieces.  Tokens are worked on in pieces of so many that 16 bits for each of
 * their words take 2 GB (8192 tokens of 128256 words), 65536 tokens at most: exp(z[j] - m) relative to
 * a power of two of 128 words' own, which the second pass over it turns into dx
 * in bf16.  The weight's gradient over several pieces is summed in fp32.
 *
 * Types.  Hidden states and weight are bf16, or fp32, which are rounded to bf16
 * first (as under autocast); gradients have the type asked for.  exp and sums
 * are fp32; dx is rounded to bf16 once before the gradients' products, whose
 * sums are fp32 and are rounded once.  The tensor cores cut a sum off at each
 * of its steps, so a gradient that one token or word makes most of comes out up
 * to 3e-4 of itself smaller in fp32, however many tokens and words there are.
 *
 * Values.  A token with a target outside the vocabulary answers NaN (logp, the
 * loss, its hidden gradient and the weight's), and so does one with a logit of
 * NaN or +inf, or with nothing but -inf.  A word of logit -inf has probability 0
 * (the hidden gradient, a sum with 0 times its weight, is NaN where that is
 * infinite; the loss of such a target is +inf).  Equal inputs give equal bits.  Every call only launches
 * kernels on the caller's stream: nothing is allocated on the device or waited
 * for, and it may be captured in a graph.  Every wait inside a kernel is
 * bounded; if one runs out, which no input brings about, the loss is NaN.
 * Calls on different streams may run at the same time if each has its own
 * workspace.  Status codes, dtypes and the message slot are shared with
 * adafactor.h; every argument check runs before the first CUDA call.
 */
#ifndef MEO_LINEAR_CE_H
#define MEO_LINEAR_CE_H

#include <stddef.h>
#include <stdint.h>

#include "adafactor.h"
#include "losses.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Hidden states, and their gradient (p == NULL: none): value (b, s, i) at
 * p[b * stride_b + s * stride_s + i].  The gradient may take the hidden states'
 * own place (same p, dtype and strides); no other overlap. */
typedef struct linear_ce_hidden {
    void* p;
    int32_t dtype;               /* ADAF_FLOAT32 or ADAF_BFLOAT16            */
    int64_t batch, seq, dim;     /* batch * seq <= 2^26, 1 <= dim <= 2^16    */
    int64_t stride_b, stride_s;  /* elements, >= 0                           */
} linear_ce_hidden;

/* The weight [vocab, dim], and its gradient: value (v, i) at p[v * stride_v + i]. */
typedef struct linear_ce_weight {
    void* p;
    int32_t dtype;
    int64_t vocab;               /* 1 .. 2^21                                */
    int64_t stride_v;            /* elements, >= dim                         */
    int32_t accumulate;          /* gradient: add to what is there           */
} linear_ce_weight;

typedef struct linear_ce_args {
    loss_rows weights;           /* fp32; p == NULL: the mean                */
    double temperature;          /* > 0                                      */
    double z_loss;               /* >= 0                                     */
    double grad_scale;           /* multiplies the gradients, not the loss   */
} linear_ce_args;

/* Bytes of workspace.  grad_hidden and grad_weight: both NULL for the loss
 * alone.  Depends on sizes, types and the weight's alignment only. */
adaf_status linear_ce_workspace_size(const linear_ce_hidden* hidden, const linear_ce_weight* weight,
                                     const linear_ce_hidden* grad_hidden, const linear_ce_weight* grad_weight,
                                     size_t* bytes);

/* loss [1]; logp, lse [batch * seq] fp32 (0 where ignored; each may be NULL).
 * Either gradient may be NULL.  workspace: 256-byte aligned. */
adaf_status linear_ce(const linear_ce_hidden* hidden, const linear_ce_weight* weight, const loss_targets* targets,
                      const linear_ce_args* args, const linear_ce_hidden* grad_hidden,
                      const linear_ce_weight* grad_weight, float* loss, float* logp, float* lse, void* workspace,
                      size_t workspace_bytes, void* stream);

/* Testing hook: while on, the copies of the calling thread's calls are expected
 * but not made, so that the kernels' waits run out (after about a second each). */
void linear_ce_debug_stall_copies(int32_t on);

/* Per-kernel CUDA-event timing, as in adafactor.h. */
adaf_status linear_ce_profile_enable(int32_t on);
adaf_status linear_ce_profile_read(double* ms, int64_t* launches, int32_t nk);
int32_t linear_ce_num_kernels(void);
const char* linear_ce_kernel_name(int32_t k);

#ifdef __cplusplus
}
#endif

#endif /* MEO_LINEAR_CE_H */
