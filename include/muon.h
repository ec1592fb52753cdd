/*
 * muon.h — C ABI of the multi-tensor Muon step and of its orthogonalisation on
 * one GB300 GPU (sm_103a).
 *
 * Operation.  Per matrix p [rows, cols] with gradient g, step by step:
 *     m = momentum m + g
 *     u = g + momentum m   (nesterov; else u = m)
 *     o = orthogonalise(u)
 *     p = p - lr weight_decay p - lr s o
 *     s = sqrt(max(1, rows / cols))        (MUON_ADJUST_ORIGINAL)
 *         0.2 sqrt(max(rows, cols))        (MUON_ADJUST_MATCH_RMS: the update's
 *                                           root mean square is about 0.2 lr)
 * orthogonalise(u) brings the singular values of u near 1 and keeps its
 * singular vectors, by Newton-Schulz steps on x = u / max(||u||_F, eps):
 *     x = a x + (b A + c A A) x,   A = x x^T    (of x^T where rows > cols)
 * with (a, b, c) given per step; the default is five times
 * (3.4445, -4.7750, 2.0315), which leaves singular values between 0.68 and 1.21
 * from any above 0.01 of the largest sum.
 *
 * Precision.  Products run on the tensor cores with fp16 factors and fp32 sums.
 * x is carried in fp32, and the diagonals of A and of b A + c A A, where
 * most of their size is, are kept in fp32 and multiplied apart, so a rounding
 * is relative to what a step changes and small singular values are not lost in
 * the large ones' roundings.  Against the formula (2-norm of the difference over
 * 2-norm) the result is
 *     within 1.5e-3 where no side is below 128 and the singular values are those
 *         of noise or fall as 1 / sqrt(k) to 1 / k^2 (2e-4 to 1.1e-3 measured);
 *     within 6e-3 there whatever they are (4e-3 measured for exact low rank: the
 *         steps enlarge an error by up to ten, alike for like singular values);
 *     within 1.5e-2 for smaller matrices (1e-3 as a rule; 8e-3 measured), if
 *         they do not fall faster than 1 / k^2.  Where they do, as 1 / k^6, most
 *         directions come out far below 1, and 3e-2 was measured.
 *
 * Values.  A matrix with NaN or infinities, or whose sum of squares overflows
 * fp32, answers NaN; a matrix of zeros stays zero.  Equal inputs give equal
 * bits.  Status codes, dtypes and the message slot are shared with
 * adafactor.h; every argument check runs before the first CUDA call.  Calls
 * only launch kernels: nothing is allocated on the device or waited for, and
 * they may be captured in a graph.  Every wait inside a kernel is bounded; if
 * one runs out, which no input brings about, bit 0 of the status word is set,
 * the step leaves the parameters of the matrices it had not finished as they
 * were, and muon_orthogonalize answers NaN in the parts it could not compute.
 */
#ifndef MEO_MUON_H
#define MEO_MUON_H

#include <stddef.h>
#include <stdint.h>

#include "adafactor.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MUON_ADJUST_ORIGINAL 0
#define MUON_ADJUST_MATCH_RMS 1
#define MUON_MAX_STEPS 16

/* One parameter: `batch` matrices one after another, contiguous, row-major. */
typedef struct muon_tensor {
    float* p;                    /* fp32, updated in place                   */
    const void* g;               /* gradient, grad_dtype                     */
    int32_t grad_dtype;          /* ADAF_FLOAT32 or ADAF_BFLOAT16            */
    int64_t batch, rows, cols;   /* >= 0; a size of 0: nothing to do         */
    float* momentum;             /* fp32, zero before the first step         */
} muon_tensor;

/* The orthogonalisation's steps. */
typedef struct muon_iteration {
    int32_t steps;                       /* 1 .. MUON_MAX_STEPS              */
    double coef[MUON_MAX_STEPS][3];      /* a, b, c of each                  */
    double eps;                          /* > 0                              */
} muon_iteration;

typedef struct muon_hparams {
    double lr;                   /* >= 0                                     */
    double momentum;             /* in [0, 1)                                */
    double weight_decay;         /* >= 0                                     */
    int32_t nesterov;
    int32_t adjust_lr;           /* MUON_ADJUST_*                            */
    muon_iteration iteration;
} muon_hparams;

/* Matrices to orthogonalise: value (b, i, j) at x[b * stride_b + i * stride_r + j]. */
typedef struct muon_matrices {
    const void* x;
    int32_t dtype;               /* ADAF_FLOAT32 or ADAF_BFLOAT16            */
    int64_t batch, rows, cols;
    int64_t stride_b, stride_r;  /* elements, >= 0                           */
} muon_matrices;

void muon_default_iteration(muon_iteration* it);

/* Checks the values; ADAF_ERR_INVALID_ARGUMENT on a bad one.  Coefficients are
 * refused if, from some singular value in [0, 1], a step would pass what the
 * scaled fp16 factors hold (a singular value of 1.9, or |b s^2 + c s^4| of 3.9). */
adaf_status muon_validate(const muon_hparams* hp);
adaf_status muon_validate_iteration(const muon_iteration* it);

/* Bytes of workspace (host only).  Matrices are worked on together, up to 48 of
 * them or 2^28 values at a time.  ADAF_ERR_UNSUPPORTED for a matrix with a side
 * above 2^20 or more than 2^31 - 1 values, or more than 2^20 matrices. */
adaf_status muon_workspace_size(const muon_tensor* tensors, int32_t n, size_t* bytes);
adaf_status muon_orthogonalize_workspace_size(int64_t batch, int64_t rows, int64_t cols, size_t* bytes);

/* One step over the list, enqueued on `stream`.  All of it is stepped at once:
 * parameters and momenta share no memory with anything else in the list (nor
 * one tensor listed twice); gradients may with one another.  workspace: 256-byte aligned
 * device memory, not used by another call in flight. */
adaf_status muon_step(const muon_tensor* tensors, int32_t n, const muon_hparams* hp, void* workspace,
                      size_t workspace_bytes, void* stream);

/* out [batch, rows, cols] contiguous, out_dtype ADAF_FLOAT32 or ADAF_BFLOAT16;
 * it may be x itself where that is contiguous and of the same dtype. */
adaf_status muon_orthogonalize(const muon_matrices* x, const muon_iteration* it, void* out, int32_t out_dtype,
                               void* workspace, size_t workspace_bytes, void* stream);

/* The status word of the last call on this workspace (synchronises `stream`). */
adaf_status muon_device_status(const void* workspace, void* stream, int32_t* status);

/* Testing hook: while on, the copies of the calling thread's calls are expected
 * but not made, so that the kernels' waits run out (after about a second each). */
void muon_debug_stall_copies(int32_t on);

/* Per-kernel CUDA-event timing, as in adafactor.h. */
adaf_status muon_profile_enable(int32_t on);
adaf_status muon_profile_read(double* ms, int64_t* launches, int32_t nk);
int32_t muon_num_kernels(void);
const char* muon_kernel_name(int32_t k);

#ifdef __cplusplus
}
#endif

#endif /* MEO_MUON_H */
