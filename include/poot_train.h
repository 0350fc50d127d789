/*
 * poot_train.h -- C ABI of the two ends of a training step on the GB300
 * (sm_103a) linear library: the softmax cross entropy of a vocabulary head with
 * its gradients, and the AdamW step over a list of tensors.
 *
 * Conventions are those of poot_ffn.h: device pointers of the current device,
 * sizes in elements, status codes, work queued on `stream` without
 * synchronising; argument errors are found before any CUDA call and leave
 * everything untouched.
 */
#ifndef POOT_TRAIN_H
#define POOT_TRAIN_H

#include "poot_ffn.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Softmax cross entropy on a linear head, without the logits in memory:
 *   z = x W^T + b                      [M, V], FP32, kept in registers
 *   lse[i]  = log sum_v exp z[i, v]
 *   loss[i] = lse[i] - z[i, target[i]]
 * for x [M, K] (rows ldx apart), W [V, K] contiguous, b [V] or NULL, target
 * [M].  A row whose target is ignore_index has loss 0 (its lse is computed all the same); one whose
 * target is outside [0, V) otherwise has loss NaN.  lse may be NULL; it is what
 * poot_linear_cross_entropy_backward reads.  Logits are FP32 sums, rounded to
 * nearest over chunks of 1024 elements of K; loss and lse are FP32.  Infinite
 * logits follow the formula: -inf takes no part in the sum, rows of nothing
 * else have lse -inf, +inf gives lse +inf.
 * The library's workspace holds 32 bytes for every row and 256 columns, and
 * copies of operands that TMA cannot read in place (see poot_gated_linear).
 * M == 0 does nothing; K == 0 gives z = b.
 * Errors: POOT_ERR_INVALID_ARG (sizes outside [0, POOT_FFN_MAX_SIZE], V == 0
 * with M > 0, NULL, ldx < K, a matrix that spans more than 2^50 elements, an
 * unknown dtype, an output overlapping an input or another output);
 * POOT_ERR_MISALIGNED (a pointer below its element's alignment); POOT_ERR_CUDA
 * where there is no memory for the workspace (nothing is queued then);
 * otherwise as poot_linear_f16.
 */
typedef struct poot_linear_cross_entropy_args {
    const void* x;
    const void* w;
    const void* b;
    const int64_t* target;
    float* loss;
    float* lse;
    int64_t M, V, K, ldx;
    int64_t ignore_index;
    int dtype;       /* POOT_DTYPE_F16 or POOT_DTYPE_BF16: x, W, b */
} poot_linear_cross_entropy_args;
POOT_API int poot_linear_cross_entropy(const poot_linear_cross_entropy_args* args, poot_stream_t stream);

/*
 * Gradients of sum_i dloss[i] loss[i]:
 *   q[i, v] = dloss[i] (exp(z[i, v] - lse[i]) - [v == target[i]])   0 in ignored rows
 *   dx = q W [M, K],   dw = q^T x [V, K],   db = column sums of q [V]
 * dloss: FP32, elements dloss_stride apart (0: one value for all rows; it is
 * not read in ignored rows).  The logits are computed again, over pieces of the vocabulary:
 * q of a piece is held in the workspace in the head dtype (at most 256 MB, or
 * 512 columns), scaled by a power of two that brings the largest |dloss| to
 * [2^14, 2^15), so that in binary16 probabilities down to 2^-29 keep their precision;
 * dx is added up over the pieces in FP32.  Results are rounded once, after the
 * scale is taken out.  Ignored rows contribute nothing to any result, whatever
 * their x, lse and dloss hold; their dx is 0.  A row whose target is outside [0, V)
 * otherwise gives NaN.
 * Optional outputs as in poot_linear_backward; x, W, target, lse and dloss are
 * needed for each of them.  M == 0 writes zeros to dw and db; K == 0 leaves dx
 * and dw without elements.  Equal calls give equal bits.
 * Errors as above.
 */
typedef struct poot_linear_cross_entropy_backward_args {
    const float* dloss;
    const void* x;
    const void* w;
    const void* b;
    const int64_t* target;
    const float* lse;
    void* dx;
    void* dw;
    void* db;
    int64_t M, V, K, ldx;
    int64_t dloss_stride;
    int64_t ignore_index;
    int dtype;
} poot_linear_cross_entropy_backward_args;
POOT_API int poot_linear_cross_entropy_backward(const poot_linear_cross_entropy_backward_args* args,
                                                poot_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* POOT_TRAIN_H */
