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
 * The library's workspace holds 32 bytes for every row and tile of 64 to 256
 * columns, and copies of operands that TMA cannot read in place (see
 * poot_gated_linear).
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
 *   dx = q W [M, K],   dw = q^T x [V, K],   db = column sums of q [V] (FP32, before q is rounded)
 * dloss: FP32, elements dloss_stride apart (0: one value for all rows; it is
 * not used in ignored rows).  The logits are computed again, over pieces of the vocabulary:
 * q of a piece is held in the workspace in the head dtype (at most 256 MB, or
 * 512 columns), scaled by a power of two that brings the largest |dloss| to
 * [2^14, 2^15), so that in binary16 probabilities down to 2^-28 keep their precision in the rows
 * of that |dloss|, and lose a step of 2^-39 of it at most in any;
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

/*
 * One AdamW step (Loshchilov and Hutter, decoupled weight decay) over a list of tensors:
 *   g = grad * grad_scale
 *   m = beta1 m + (1 - beta1) g           v = beta2 v + (1 - beta2) g^2
 *   param = param (1 - lr weight_decay)
 *           - lr / (1 - beta1^step) * m / (sqrt(v) / sqrt(1 - beta2^step) + eps)
 *   copy  = param                          where copy is given
 * in FP32, each operation rounded on its own in this order; the factors that depend on lr,
 * weight_decay, step and the betas alone are computed in FP64 and rounded once.  param is rounded
 * once to its dtype.  Equal calls give equal bits, whatever else is in the list.
 * param, grad: binary16, bfloat16 or FP32 (POOT_GRAD_*), any alignment of their elements; copy:
 * binary16 or bfloat16, for an FP32 param (master weights).
 * bits 32: m and v are FP32 [n].  bits 8: m is int8 [n], v uint8 [n], and each has an FP32
 * scale for every POOT_ADAMW_BLOCK elements in order ([ceil(n / 256)]):
 *   m = m_scale c |c|       (-127 <= c <= 127, m_scale = max |m| / 127^2)
 *   v = (v_scale c^2)^2     (0 <= c <= 255, v_scale = max sqrt(v) / 255^2)
 * The step itself uses the new m and v before they are rounded to codes; codes are
 * nearest in c, a nonzero v has a code of at least 1, and a block whose |m| are all below 2^-110
 * counts as zero.  An average moves only when a step changes it by half the distance of two codes:
 * 0.8% of m and of v at the top of a block, more below.  A block with an m or v that is not finite
 * reads as NaN.  All zeros are a valid first state in either form.
 * step counts from 1.  lr, step and grad_scale are read from device memory
 * when the step runs where lr_device, step_device or grad_scale_device is given
 * (a captured graph follows them); with lr_device, 1 - lr weight_decay is one FP32 operation.
 * Tensors may be empty.  What a call writes may overlap nothing else of it.
 * Errors: POOT_ERR_INVALID_ARG (count < 0, NULL, n < 0 or n > 2^40, an unknown dtype or
 * bits, a copy of a 16-bit param, beta outside [0, 1), eps, lr or weight_decay negative or not
 * finite, a grad_scale that is not finite, step < 1, overlap), POOT_ERR_MISALIGNED (a pointer
 * below its element's alignment), POOT_ERR_CUDA.
 */
#define POOT_ADAMW_BLOCK 256

typedef struct poot_adamw_tensor {
    void* param;
    const void* grad;
    void* m;
    void* v;
    float* m_scale;
    float* v_scale;
    void* copy;
    int64_t n;
    double weight_decay;
    int param_dtype, grad_dtype, copy_dtype;
} poot_adamw_tensor;

typedef struct poot_adamw_args {
    const poot_adamw_tensor* tensors;
    int64_t count;
    const float* lr_device;
    const int64_t* step_device;
    const float* grad_scale_device;
    int64_t step;
    double lr, beta1, beta2, eps, grad_scale;
    int bits;
} poot_adamw_args;
POOT_API int poot_adamw_step(const poot_adamw_args* args, poot_stream_t stream);

/*
 * The FP32 values that 8-bit states stand for (for a checkpoint, or to look at
 * them): m_out and v_out, [n] each.  Errors as above.
 */
typedef struct poot_adamw_codes {
    const void* m;
    const void* v;
    const float* m_scale;
    const float* v_scale;
    float* m_out;
    float* v_out;
    int64_t n;
} poot_adamw_codes;
POOT_API int poot_adamw_values(const poot_adamw_codes* states, int64_t count, poot_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* POOT_TRAIN_H */
