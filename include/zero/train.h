/*
 * zero/train.h -- C ABI of the training operators that sit next to the ZeRO
 * shard step: AdamW over a list of tensors with 32-bit or 8-bit states, the
 * conversion between the two states, and the softmax cross entropy of a
 * large vocabulary with its gradient.
 *
 * libzero_train_mi355x.so holds them; it uses libzero_mi355x.so (errors,
 * the step's constants).  The conventions are those of zero.h: ZERO_OK or a
 * negative ZERO_E* code with the text in zero_last_error(); arguments are
 * checked before any work is queued; the caller owns every buffer and no
 * call allocates device memory; work is queued on `stream` and not waited
 * for unless a call says so; every call can be captured in a HIP graph
 * (kernels only) unless it waits.
 */
#ifndef ZERO_TRAIN_H
#define ZERO_TRAIN_H

#include "zero.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------
 * 8-bit optimizer state.  A tensor's moments are held in blocks of
 * ZERO_STATE8_BLOCK elements; block b of a tensor takes bytes
 * [512 b, 512 b + 256) of state8 for the first moment, the next 256 for the
 * second, and bytes 2b and 2b + 1 of scale8 for their exponents E.  The last
 * block of a tensor is padded with zero codes.
 *
 * E is the biased fp32 exponent of the block's largest magnitude, one more
 * where its mantissa is above 1.875, clamped to [1, 254].
 *   first moment:  sign, 4 exponent bits e, 3 mantissa bits f
 *   second moment: 5 exponent bits e, 3 mantissa bits f, no sign
 * With B = 15 (first) or 31 (second) a code stands for
 *   e > 0:  (1 + f/8) * 2^(e - B + E - 127)
 *   e = 0:  (f/8)     * 2^(1 - B + E - 127)      (gradual underflow)
 * A second moment above zero never takes code 0, so that no update divides
 * by eps alone because of the rounding.  A magnitude past the top code
 * (an infinite second moment) takes the top code: the format has no infinity
 * and no NaN.  Either moves its block to E = 254, under which a first moment
 * below 2^109 becomes 0 and a second moment below 2^94 becomes 2^94.
 */
#define ZERO_STATE8_BLOCK 256

/* m[0, n) and v[0, n) (fp32, device, 16-byte aligned; v >= 0) into n8 =
 * ceil(n / 256) blocks: state8 (512 n8 bytes, 16-byte aligned) and scale8
 * (2 n8 bytes, 2-byte aligned), rounded to nearest even.  Moments that hold
 * NaN are not detected: a NaN in m, or one without its sign bit in v, is
 * held as an infinity is, one with it in v as 0.  zero_tensors_step writes
 * none (a gradient that is not finite skips the step).
 * Errors: n < 0, a NULL pointer when n > 0 -> ZERO_EINVAL; misalignment ->
 * ZERO_EALIGN; launch -> ZERO_EDEVICE. */
int zero_state8_encode(const float* m, const float* v, int64_t n, void* state8, void* scale8,
                       void* stream);

/* The reverse, into m[0, n) and v[0, n) of dtype ZERO_FP32, ZERO_BF16 or
 * ZERO_FP16 (rounded to nearest even; every value of the format that bf16
 * can reach is a bf16 value).  m and v 16-byte aligned.  Errors as above, a
 * bad dtype -> ZERO_EINVAL. */
int zero_state8_decode(const void* state8, const void* scale8, int64_t n, void* m, void* v,
                       int32_t dtype, void* stream);

/* ------------------------------------------------------------------------
 * AdamW over a list of tensors.
 *
 * The tensors lie anywhere: each pointer needs only its element's alignment
 * (state8: 16 bytes, scale8: 2 bytes), so parameters packed end to end are
 * fine.  Ranges of different fields and tensors must not overlap.
 */
#define ZERO_MAX_GROUPS 8

typedef struct {
    const void* grad;         /* device, numel values of the list's grad_dtype  */
    float* master;            /* device fp32[numel], updated in place           */
    /* 32-bit states: fp32[numel] each.  8-bit: state8 and scale8.             */
    void* exp_avg;            /* exp_avg, or state8                             */
    void* exp_avg_sq;         /* exp_avg_sq, or scale8                          */
    void* param;              /* param_dtype values out; NULL if the list has none */
    int64_t numel;            /* >= 0; 0: the tensor is skipped, NULLs allowed  */
    int32_t group;            /* index into zero_tensors_args.groups            */
    int32_t reserved;         /* 0                                              */
} zero_tensor_t;

/* What a list of tensors needs; filled by zero_tensors_plan. */
typedef struct {
    int64_t numel;            /* elements of all tensors                        */
    int64_t n_chunks;         /* blocks of work                                 */
    int32_t n_tensors;
    int32_t n_groups;         /* 1 + the largest group used                     */
    int32_t state_bits;       /* 32 or 8                                        */
    int32_t grad_dtype;       /* ZERO_FP16, ZERO_BF16 or ZERO_FP32              */
    int32_t param_dtype;      /* ZERO_FP16, ZERO_BF16, or 0: no parameters out  */
    int32_t reserved;
    uint64_t table_bytes;     /* device table the kernels read                  */
    uint64_t workspace_bytes;
} zero_tensors_plan_t;

/* Host only.  Checks the list and fills *plan; with `table` not NULL also
 * writes the list's table (plan->table_bytes long; table_cap is the room
 * there) for the caller to copy to the device, 16-byte aligned.  Plan and
 * table serve every step until a pointer or size changes.
 * Errors: NULL or out-of-range arguments, param set in some tensors and not
 * in others or not matching param_dtype, more than 2^31 - 1 chunks of 1024
 * elements -> ZERO_EINVAL; a pointer off its element's alignment -> ZERO_EALIGN; table_cap too
 * small -> ZERO_ESIZE. */
int zero_tensors_plan(const zero_tensor_t* tensors, int32_t n_tensors, int32_t state_bits,
                      int32_t grad_dtype, int32_t param_dtype, void* table, size_t table_cap,
                      zero_tensors_plan_t* plan);

typedef struct {
    double lr, beta1, beta2, eps, weight_decay;
} zero_adam_group_t;

/* Per-step constants of a list, as the kernels take them: launch arguments,
 * or read from device memory when zero_tensors_args.scalars is set. */
typedef struct zero_tensors_scalars_s {
    float    inv_scale;       /* fp32(1 / (loss_scale * grad_predivide))        */
    int32_t  peer_overflow;
    uint32_t key;             /* of the stochastic rounding, from the seed      */
    uint32_t reserved;
    double   max_grad_norm;
    double   peer_sumsq;
    struct {                  /* as zero_step_scalars_t                         */
        float decay, beta1, one_minus_beta1, beta2, one_minus_beta2, step_size, inv_sqrt_bc2, eps;
    } group[ZERO_MAX_GROUPS];
} zero_tensors_scalars_t;

typedef struct {
    zero_tensors_plan_t plan;
    const void* table;        /* device copy of the table, 16-byte aligned      */
    void* workspace;          /* device, plan.workspace_bytes, 16-byte aligned  */
    size_t workspace_bytes;
    const zero_adam_group_t* groups;   /* host, n_groups entries                */
    int32_t n_groups;         /* plan.n_groups .. ZERO_MAX_GROUPS               */
    int32_t peer_overflow;    /* the other ranks' OR'd flag                     */
    int64_t step;             /* t >= 1                                         */
    double loss_scale;        /* > 0                                            */
    double grad_predivide;    /* > 0                                            */
    double max_grad_norm;     /* <= 0: no clipping                              */
    double peer_sumsq;        /* the other ranks' sum of squares, >= 0          */
    uint64_t seed;            /* 8-bit states: stochastic rounding of this step */
    zero_global_t* result;    /* device, 32 bytes, 16-byte aligned              */
    const zero_tensors_scalars_t* scalars;  /* device or NULL, 16-byte aligned  */
} zero_tensors_args;

/* One step over the list, the arithmetic of zero_shard_step with one
 * replica: g = grad * fp32(1 / (loss_scale * grad_predivide)); the fp64 sum
 * of squares, the norm, clip factor and overflow flag over the whole list go
 * to *result; unless the overflow flag is set (then no tensor is written),
 *   g' = g * coef;  m' = b1 m + (1 - b1) g';  v' = b2 v + (1 - b2) g'^2
 *   p' = p (1 - lr wd) - lr/(1 - b1^t) * m' / (sqrt(v')/sqrt(1 - b2^t) + eps)
 * in fp32 with each tensor's group's constants, then param = p' rounded to
 * nearest even.  8-bit states: m and v are decoded, p' uses m' and v'
 * unrounded, and the new codes round stochastically: an element at block
 * ordinal B of the list (tensors in order, blocks of 256) and place j in it
 * takes two 16-bit noises from the 32-bit finalizer of MurmurHash3 over
 * (256 B + j) * 0x9E3779B1 + key, the low half for the first moment.  The
 * result depends on the inputs and the seed only, never on timing.
 * info not NULL: waits for the stream and copies *result there (not under
 * graph capture).  Errors as zero_shard_step; a plan that zero_tensors_plan
 * cannot have made -> ZERO_EINVAL. */
int zero_tensors_step(const zero_tensors_args* a, zero_step_info* info, void* stream);

/* The step in two parts, for a world of ranks that each own some tensors:
 * zero_tensors_norm leaves the list's partial sums in slot `slot` of a
 * zero_partials_bytes table (as zero_shard_reduce does), zero_shard_combine
 * joins the slots of the ranks into a zero_global_t, and zero_tensors_apply
 * updates the list by it.  peer_sumsq, peer_overflow and result of *a are
 * not used by these two. */
int zero_tensors_norm(const zero_tensors_args* a, int32_t slot, void* partials_dev, void* stream);
int zero_tensors_apply(const zero_tensors_args* a, const void* global_dev, void* stream);

/* Fills *out as the kernels' launch arguments are filled (see
 * zero_step_scalars): a caller that captures the step once copies it to
 * a->scalars before each replay.  Host only. */
int zero_tensors_scalars(const zero_tensors_args* a, zero_tensors_scalars_t* out);

/* ------------------------------------------------------------------------
 * Softmax cross entropy of a large vocabulary.
 *
 *   logits = x w^T           x: tokens x dim, w: vocab x dim, 16 bits
 *   lse_i  = log sum_j exp(logits_ij)
 *   loss_i = lse_i - logits_{i, target_i}
 *   mean   = sum_i loss_i / max(1, count)
 * over the count tokens whose target lies in [0, vocab); any other target
 * gives loss 0 and no gradient (out_of_range counts those >= vocab).  The
 * gradient of grad_scale * mean is
 *   P_ij = grad_scale / max(1, count) * (exp(logits_ij - lse_i) - [j = target_i])
 *   dx = P w,  dw = P^T x.
 * The logits are formed piece by piece of the vocabulary and never kept:
 * the backward forms them again, of the tokens that have a target only.  A
 * token without one has an lse like any other, but its row of x reaches no
 * other token's loss and neither the mean nor dw, whatever it holds (NaN and
 * infinities too), and its row of dx is zero.  Products are of the 16-bit inputs with
 * fp32 sums; loss and lse are fp32; the sum over tokens is fp64 in a fixed
 * order.  P is rounded to 16 bits for the two products of the gradient
 * (a relative half step of the dtype, what dx and dw are rounded by too).
 * Results do not depend on timing.  A row whose logits are all -inf has
 * lse = -inf; +inf or NaN logits give an infinite or NaN lse; any finite
 * logits, the type's lowest value among them, a finite lse.
 */
typedef struct {
    double  loss_sum;
    int64_t count;            /* tokens with a target in [0, vocab)             */
    int32_t out_of_range;     /* targets >= vocab                               */
    int32_t reserved;
    float   mean;
    float   inv_count;        /* fp32(1 / max(1, count))                        */
} zero_xent_result_t;

typedef struct {
    int64_t tokens, dim, vocab;   /* each >= 0; vocab and dim >= 1 if tokens > 0 */
    int64_t x_stride, w_stride;   /* elements from row to row, >= dim            */
    int64_t dx_stride, dw_stride;
    int32_t dtype;            /* ZERO_FP16 or ZERO_BF16: x, w, dx, dw           */
    int32_t reserved;         /* 0                                              */
    const void* x;            /* device, 2-byte aligned                         */
    const void* w;
    const int64_t* target;    /* device, 8-byte aligned                         */
    float* loss;              /* device fp32[tokens], out                       */
    float* lse;               /* device fp32[tokens], out of the forward, in of
                                 the backward                                   */
    zero_xent_result_t* result;   /* device, 16-byte aligned, likewise          */
    void* dx;                 /* device, out of the backward                    */
    void* dw;
    double grad_scale;        /* finite; the loss scale                         */
    void* workspace;          /* device, 256-byte aligned                       */
    size_t workspace_bytes;
} zero_xent_args;

/* Bytes of workspace forward and backward need (one buffer serves both; no
 * call reads what another left there).  0 for out-of-range sizes.  Host only. */
size_t zero_xent_workspace_bytes(int64_t tokens, int64_t dim, int64_t vocab);

/* Writes loss, lse and *result; dx and dw are not used.
 * Errors: NULL or out-of-range arguments -> ZERO_EINVAL; misalignment ->
 * ZERO_EALIGN; workspace_bytes too small -> ZERO_ESIZE; launch ->
 * ZERO_EDEVICE. */
int zero_xent_forward(const zero_xent_args* a, void* stream);

/* Writes dx and dw from x, w, target and the forward's lse and *result;
 * loss is not used.  Errors as above. */
int zero_xent_backward(const zero_xent_args* a, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* ZERO_TRAIN_H */
