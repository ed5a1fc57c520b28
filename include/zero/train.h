/*
 * zero/train.h -- C ABI of the training operators that sit next to the ZeRO
 * shard step: AdamW over a list of tensors with 32-bit or 8-bit states, the
 * conversion between the two states, the softmax cross entropy of a large
 * vocabulary with its gradient, and activations held in 8 bits with what
 * reads them: a gated activation and a product, each with its gradient.
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

/* Bytes of workspace that forwards and backwards of up to `tokens` tokens need
 * (one buffer serves them all; no call reads what another left there).  It
 * never falls as tokens rise.  0 for out-of-range sizes.  Host only; a search
 * over the numbers of tokens, 20 us to 1 ms. */
size_t zero_xent_workspace_bytes(int64_t tokens, int64_t dim, int64_t vocab);

/* Writes loss, lse and *result; dx and dw are not used.
 * Errors: NULL or out-of-range arguments -> ZERO_EINVAL; misalignment ->
 * ZERO_EALIGN; workspace_bytes too small -> ZERO_ESIZE; launch ->
 * ZERO_EDEVICE. */
int zero_xent_forward(const zero_xent_args* a, void* stream);

/* Writes dx and dw from x, w, target and the forward's lse and *result;
 * loss is not used.  Errors as above. */
int zero_xent_backward(const zero_xent_args* a, void* stream);

/* ------------------------------------------------------------------------
 * Rows of 8-bit codes: an activation kept for the backward (a row is a
 * token), or a weight (a row is an output channel).
 *
 * A row is held as whole numbers q of [-127, 127] and one fp32 scale s, and
 * stands for q s.  The encoder takes s = 2^e with the smallest e under which
 * the row's largest magnitude rounds to 127 or less, e clamped to [-24, 9]
 * for fp16 and [-126, 121] for bf16 and fp32, and q = row / s to nearest
 * even, clamped.  A power of two makes every q s a value of the row's own
 * 16-bit type: nothing that reads the row in 16 bits rounds it again, and
 * the codes depend on the row alone.  A row that holds an infinity or a NaN
 * has a NaN scale (and codes 0): all of it reads as NaN, so that the
 * overflow reaches the gradients and the step's flag.
 *
 * A row of codes takes ZERO_ROWS8_BYTES(dim) bytes, dim rounded up to a
 * multiple of 16, and holds zeros from dim on; the encoder writes them.
 * Whoever makes codes by other means writes them too, and rows cut out of
 * wider ones have them only where dim is a multiple of 16.  Rows start at
 * multiples of 16 bytes: 16-byte aligned, strides multiples of 16.  What
 * lies between a row's ZERO_ROWS8_BYTES and the next row is neither read nor
 * written.  The readers below take codes of [-128, 127] and any fp32 scale
 * as they are.
 */
#define ZERO_ROWS8_MAX_DIM 131071
#define ZERO_ROWS8_BYTES(dim) (((dim) + 15) / 16 * 16)

/* x: rows x dim values of dtype ZERO_FP16, ZERO_BF16 or ZERO_FP32, aligned to
 * its element, x_stride (elements, >= dim, <= 2^31) from row to row.
 * rows in [0, 2^31), dim in [0, ZERO_ROWS8_MAX_DIM]; a row of no elements or
 * of zeros has the least scale.
 * The codes and scales must not overlap x.
 * Errors: a size, stride or dtype out of range, a NULL pointer where there is
 * something to read or write -> ZERO_EINVAL; misalignment -> ZERO_EALIGN;
 * launch -> ZERO_EDEVICE. */
int zero_rows8_encode(const void* x, int64_t x_stride, int32_t dtype, int64_t rows, int64_t dim,
                      void* codes, int64_t codes_stride, float* scale, void* stream);

/* The reverse: y = q s in fp32, rounded to nearest even to dtype.  y must not
 * overlap the codes and scales.  Errors as above. */
int zero_rows8_decode(const void* codes, int64_t codes_stride, const float* scale, int64_t rows,
                      int64_t dim, void* y, int64_t y_stride, int32_t dtype, void* stream);

/* ------------------------------------------------------------------------
 * The gated activation with its input kept in 8 bits.
 *
 *   forward    h = act(gate) up,  or act(gate) where up is NULL,
 *              in fp32, rounded to dtype; gate and up into gate8 and up8 as
 *              zero_rows8_encode does, and h into h8 (the rounded h, as
 *              zero_rows8_encode would find it), in one pass
 *   backward   dgate = dh up^ act'(gate^),  dup = dh act(gate^)
 *              of the values gate^ and up^ that the codes stand for
 *
 *   ZERO_GLU_SILU  act(x) = x p, p = 1 / (1 + exp(-x))
 *   ZERO_GLU_GELU  act(x) = x p, p = 1 / (1 + exp(-2 sqrt(2/pi) (x + 0.044715 x^3)))
 *                  (the tanh form of gelu: p = (1 + tanh(..)) / 2)
 *   p is held in fp32, below 2^-126 to the nearest multiple of 2^-149.
 *
 * Results depend on the inputs alone.  A token whose gate or up holds an
 * infinity or a NaN has NaN in all of the gradients that read that row of
 * codes; so has, in h8, one whose h overflowed.  Other tokens are not
 * touched by it.
 */
#define ZERO_GLU_SILU 0
#define ZERO_GLU_GELU 1

typedef struct {
    int64_t tokens, width;    /* [0, 2^31), [0, ZERO_ROWS8_MAX_DIM]             */
    /* elements from row to row, >= width, <= 2^31; of codes bytes, multiples of
     * 16, >= ZERO_ROWS8_BYTES(width), <= 2^31; of a buffer that is NULL unused */
    int64_t gate_stride, up_stride, h_stride, dh_stride, dgate_stride, dup_stride;
    int64_t gate8_stride, up8_stride, h8_stride;
    int32_t dtype;            /* ZERO_FP16 or ZERO_BF16: gate, up, h, dh, dgate, dup */
    int32_t kind;             /* ZERO_GLU_SILU or ZERO_GLU_GELU                 */
    const void* gate;         /* device, 2-byte aligned                         */
    const void* up;           /* or NULL                                        */
    void* gate8;              /* out of the forward, in of the backward; NULL in
                                 a forward that no backward follows             */
    float* gate_scale;
    void* up8;                /* as gate8; NULL where there is no up            */
    float* up_scale;
    void* h;                  /* out; NULL: not wanted in 16 bits               */
    void* h8;                 /* out; NULL: not wanted in 8 bits                */
    float* h_scale;
    const void* dh;           /* in of the backward                             */
    void* dgate;              /* out of the backward                            */
    void* dup;                /* as dgate; NULL where there is no up8           */
} zero_glu8_args;

/* Writes h or h8 or both, and gate8 and up8 where they are given; dh, dgate
 * and dup are not used.  No output may overlap an input or another output.
 * No token, or a width of 0: nothing is written.
 * Errors: NULL or out-of-range arguments -> ZERO_EINVAL; misalignment (2
 * bytes for the 16-bit buffers, 16 for codes, 4 for scales) -> ZERO_EALIGN;
 * launch -> ZERO_EDEVICE. */
int zero_glu8_forward(const zero_glu8_args* a, void* stream);

/* Writes dgate and dup from dh, gate8 and up8 with their scales; gate, up, h
 * and h8 are not used.  dgate or dup may be dh itself, with its stride; no other output
 * may overlap an input or another output.
 * Errors as above. */
int zero_glu8_backward(const zero_glu8_args* a, void* stream);

/* ------------------------------------------------------------------------
 * The product of 8-bit rows with 8-bit weights, and its gradient.
 *
 *   forward    y_tn = x_scale_t w_scale_n sum_k x8_tk w8_nk + bias_n
 *   backward   dx = dy w^,  dw = dy^T x^,  db_n = sum_t dy_tn
 *              of the values x^ = x8 x_scale and w^ = w8 w_scale
 *
 * x8: tokens rows of dim codes, w8: out rows of dim codes, each with its
 * rows' scales.  The forward's sums are whole numbers in 32 bits, exact; one
 * is multiplied in fp32 by x_scale, then by w_scale with the bias added, and
 * rounded once (where its product with x_scale is past fp32's range, y is an
 * infinity, however small w_scale).  The backward takes
 * x^ and w^ in dtype (exact where the scales are the encoder's for rows of
 * that dtype, else rounded to nearest even) times dy, with fp32 sums, and
 * rounds once.  Results do not depend on timing.
 */
typedef struct {
    int64_t tokens, dim, out; /* [0, 2^20], [0, ZERO_ROWS8_MAX_DIM], [0, 2^20]  */
    int64_t x8_stride, w8_stride;     /* bytes, multiples of 16, >= ZERO_ROWS8_BYTES(dim),
                                         <= 2^22                                */
    int64_t y_stride, dy_stride;      /* elements, >= out, <= 2^31              */
    int64_t dx_stride, dw_stride;     /* >= dim, <= 2^31                        */
    int32_t dtype;            /* ZERO_FP16 or ZERO_BF16: y, bias, dy, dx, dw, db */
    int32_t reserved;         /* 0                                              */
    const void* x8;           /* device, 16-byte aligned                        */
    const float* x_scale;     /* device fp32[tokens]                            */
    const void* w8;
    const float* w_scale;     /* device fp32[out]                               */
    const void* bias;         /* device, out values, 2-byte aligned, or NULL    */
    void* y;                  /* out of the forward, 2-byte aligned             */
    const void* dy;           /* in of the backward, 2-byte aligned             */
    void* dx;                 /* out of the backward; NULL: not wanted          */
    void* dw;                 /* likewise                                       */
    void* db;                 /* likewise                                       */
    void* workspace;          /* device, 256-byte aligned                       */
    size_t workspace_bytes;
} zero_linear8_args;

/* Bytes of workspace that calls of up to `tokens` tokens need: of the forward
 * (ZERO_LINEAR8_FORWARD), of a backward whose dy is read where it lies
 * (ZERO_LINEAR8_BACKWARD: dy 16-byte aligned, out and dy_stride multiples of
 * 8, dy_stride at most 2^21) and of one whose dy may lie anyhow
 * (ZERO_LINEAR8_BACKWARD_ANY_DY); the largest of the uses named.  One buffer
 * serves them all and all calls that follow each other; no call reads what
 * another left there; calls that overlap, on two streams or in two graphs,
 * need one each.  It never falls as tokens rise.
 * The forward uses it for the whole sums of slices of dim, where few tiles and
 * a long dim are cut so (34 MB at most, mostly nothing: 256 bytes).  The
 * backward has in it at most 512 MB of x^ and w^ in 16 bits (of 256 columns,
 * if that is more), fp32 parts of dx and dw where their sums are cut (34 MB
 * each), shares of db's sum, and a copy of dy, 2 tokens out bytes, where its
 * rows are not read as they lie; a call that wants fewer of dx, dw and db has
 * their parts alone.  Of few tokens it has parts of dx's sums, or nothing.
 * 0 for out-of-range sizes or uses.  Host only; a search over the numbers of
 * tokens, 10 us to 1 ms. */
#define ZERO_LINEAR8_FORWARD 1
#define ZERO_LINEAR8_BACKWARD 2
#define ZERO_LINEAR8_BACKWARD_ANY_DY 4
size_t zero_linear8_workspace_bytes_for(int64_t tokens, int64_t dim, int64_t out, int32_t uses);

/* That of the forward and any backward. */
size_t zero_linear8_workspace_bytes(int64_t tokens, int64_t dim, int64_t out);

/* Writes y; dy, dx, dw and db are not used.  No output may overlap an input.
 * Errors: NULL or out-of-range arguments -> ZERO_EINVAL; misalignment ->
 * ZERO_EALIGN; workspace_bytes less than this call uses -> ZERO_ESIZE; launch
 * -> ZERO_EDEVICE. */
int zero_linear8_forward(const zero_linear8_args* a, void* stream);

/* Writes those of dx, dw and db that are given from dy, w8 (dx) and x8 (dw)
 * with their scales; bias and y are not used.  No output may overlap an input
 * or another output.  No token: dw and db are zero; no output channel: dx is
 * zero.  Errors as above. */
int zero_linear8_backward(const zero_linear8_args* a, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* ZERO_TRAIN_H */
