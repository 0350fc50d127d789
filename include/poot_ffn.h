/*
 * poot_ffn.h -- C ABI of the feed-forward operators of the GB300 (sm_103a)
 * linear library: the gated block, its gradients, the linear's gradients,
 * and clipping by the global gradient norm.
 *
 * Conventions are those of poot_linear.h: device pointers of the current
 * device, sizes in elements, status codes, work queued on `stream` without
 * synchronising; argument errors are found before any CUDA call and leave
 * everything untouched.  Matrices are row-major; a leading dimension (`ld*`,
 * elements between rows) of 0 means contiguous rows.  Where ld is larger, the
 * memory between two rows of an input may be read (never used).  The ld of a
 * single row is not used.  Weights are [out_features, in_features] and
 * contiguous, read in place.
 *
 * Numerics: unlike poot_contract, whose steps round one by one, these
 * operators keep every value in FP32 from the sums to the result and round
 * once to the head dtype (binary16 or bfloat16).  The one exception: the
 * gradients of gate and up (dg, du below) are rounded to the head dtype
 * before they are multiplied with the weights and x, as operands of 16-bit
 * products.  Sums are FP32 in a fixed order: equal calls give equal bits.  The
 * tensor core truncates towards zero where it adds products to a sum, so sums of
 * many terms of one sign come out low: whatever their length by about an eighth
 * of binary16's rounding and a twentieth of bfloat16's (5e-5 and 2e-4); in the
 * GEMV kernels (M <= 16) by 8e-10 per element of K, 5e-5 at 65536.
 */
#ifndef POOT_FFN_H
#define POOT_FFN_H

#include "poot_linear.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Largest M, N and K of these operators (2^31 - 4096: tiles and vectors that
 * start inside a matrix end below 2^31). */
#define POOT_FFN_MAX_SIZE 2147479552

/* Activation of the gate. */
enum poot_ffn_act {
    POOT_ACT_SILU = 0,       /* t / (1 + exp(-t)) */
    POOT_ACT_GELU_TANH = 1,  /* 0.5 t (1 + tanh(sqrt(2/pi) (t + 0.044715 t^3))) */
    POOT_ACT_GELU_ERF = 2    /* 0.5 t (1 + erf(t / sqrt 2)) */
};

/*
 * The gated block:
 *   g = x Wg^T + bg,   u = x Wu^T + bu,   h = act(g) * u
 * for x [M, K] (rows ldx apart), Wg and Wu [N, K], bg and bu [N] (either may
 * be NULL), h [M, N] contiguous.  With g and u non-NULL (both or neither;
 * [M, N] contiguous) they are stored too, each rounded once: the state that
 * poot_gated_linear_backward reads.  h is computed from the FP32 values.
 * M <= 16 streams the weights once (GEMV kernels, HBM-bound; 16-byte loads
 * with 16-byte aligned x and weights, K % 8 == 0 and ldx % 8 == 0); larger M
 * runs on the tcgen05 GEMM, whose operands, where TMA cannot read them in
 * place (base not 16-byte aligned, row pitch not a multiple of 8), are first
 * copied to 16-byte-pitched rows in the library's workspace.
 * M == 0 or N == 0 does nothing; K == 0 gives g = bg, u = bu.
 * Errors: POOT_ERR_INVALID_ARG (sizes outside [0, POOT_FFN_MAX_SIZE], NULL,
 * ldx < K, a matrix that spans more than 2^50 elements, an unknown dtype or
 * activation, only one of g and u, an output overlapping an input or another
 * output); POOT_ERR_MISALIGNED (a pointer not 2-byte aligned); POOT_ERR_CUDA
 * where there is no memory for copies (nothing is queued then; sums that were to
 * be split over K, for which there is none, go unsplit); otherwise as
 * poot_linear_f16.
 */
typedef struct poot_gated_linear_args {
    const void* x;
    const void* wg;
    const void* wu;
    const void* bg;
    const void* bu;
    void* h;
    void* g;
    void* u;
    int64_t M, N, K, ldx;
    int dtype;       /* POOT_DTYPE_F16 or POOT_DTYPE_BF16: every tensor */
    int activation;  /* POOT_ACT_* */
} poot_gated_linear_args;
POOT_API int poot_gated_linear(const poot_gated_linear_args* args, poot_stream_t stream);

/*
 * Gradients of the gated block for the output gradient dh [M, N] and the
 * saved g, u [M, N]:
 *   dg = dh * u * act'(g)       du = dh * act(g)
 *   dx = dg Wg + du Wu          [M, K]
 *   dwg = dg^T x, dwu = du^T x  [N, K]
 *   dbg = sum over rows of dg, dbu likewise   [N]
 * Any output pointer may be NULL (not wanted); the inputs it alone needs may
 * then be NULL too (x only for dwg / dwu, wg and wu only for dx).  Outputs are
 * contiguous.  M == 0 writes zeros to dwg, dwu, dbg and dbu; N == 0 zeros to
 * dx; K == 0 leaves dx, dwg and dwu without elements.  dg and du live in the
 * library's workspace (4 * M * ceil8(N) bytes).
 * Errors as poot_gated_linear; POOT_ERR_CUDA when no workspace can be had.
 */
typedef struct poot_gated_linear_backward_args {
    const void* dh;
    const void* x;
    const void* wg;
    const void* wu;
    const void* g;
    const void* u;
    void* dx;
    void* dwg;
    void* dwu;
    void* dbg;
    void* dbu;
    int64_t M, N, K, ld_dh, ldx, ld_g, ld_u;
    int dtype;
    int activation;
} poot_gated_linear_backward_args;
POOT_API int poot_gated_linear_backward(const poot_gated_linear_backward_args* args, poot_stream_t stream);

/*
 * Gradients of y = x W^T + b (poot_linear_f16, poot_contract without steps)
 * for the output gradient dy [M, N]:
 *   dx = dy W [M, K],   dw = dy^T x [N, K],   db = sum over rows of dy [N]
 * Optional outputs, inputs, empty sizes and errors as above.
 */
typedef struct poot_linear_backward_args {
    const void* dy;
    const void* x;
    const void* w;
    void* dx;
    void* dw;
    void* db;
    int64_t M, N, K, ld_dy, ldx;
    int dtype;
} poot_linear_backward_args;
POOT_API int poot_linear_backward(const poot_linear_backward_args* args, poot_stream_t stream);

/* Element types of a gradient tensor (the first two are POOT_DTYPE_*). */
enum poot_grad_dtype { POOT_GRAD_F16 = 0, POOT_GRAD_BF16 = 1, POOT_GRAD_F32 = 2 };

typedef struct poot_grad_tensor {
    const void* src;
    void* dst;      /* src itself: clipped in place */
    int64_t n;      /* elements, contiguous */
    int dtype;      /* POOT_GRAD_* */
} poot_grad_tensor;

/*
 * Clipping by the global norm over `count` tensors:
 *   norm  = sqrt(sum over all tensors of sum src^2)
 *   scale = min(1, max_norm / (norm + 1e-6))
 *   dst   = RN(src * scale), in the tensor's dtype
 * norm: device pointer to one float, written on `stream` (the call does not
 * synchronise).  Squares are summed in FP32 over at most 33 elements and in
 * FP64 beyond (scaled first where FP32 squares would overflow or vanish).  A
 * norm that is NaN makes every result NaN; an infinite norm gives scale 0 under
 * a finite max_norm, and NaN under an infinite one, as the formula does.
 * Tensors may be empty, of mixed dtypes and at any alignment of their elements;
 * count == 0 writes norm = 0.
 * A dst must be its own src or overlap no src and no other dst.
 * Errors: POOT_ERR_INVALID_ARG (count < 0, NULL, n < 0 or n > 2^40, an
 * unknown dtype, max_norm negative or NaN, overlap), POOT_ERR_MISALIGNED (a
 * pointer below its element's alignment), POOT_ERR_CUDA.
 */
POOT_API int poot_clip_grad_norm(const poot_grad_tensor* tensors, int64_t count, float max_norm, float* norm,
                                 poot_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* POOT_FFN_H */
