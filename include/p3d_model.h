/*
 * p3d_model.h -- the operators of the model around the transformer block
 * (libp3d, gfx950): group norm with an activation over channels-last maps,
 * with its gradient; linear layers in 8-bit integers; and the AdamW step over
 * many tensors, with the gradient norm that it is clipped by.
 *
 * The maps that p3d_proj_cond samples and the structure grids that the flow
 * models make pass convolutional decoders, whose group norms run over
 * channels-last data (pixal3d_mrp_mlx README: ss_dec, channels last). The
 * block's gradients (p3d_block.h) end in a weight update, and its finished
 * weights may be served in 8-bit integers.
 *
 * The conventions of p3d.h and p3d_block.h hold: DEVICE pointers owned by the
 * caller, HOST tables and descriptors read during the call only, work enqueued
 * on `stream` without allocating or synchronising, nothing enqueued on any
 * status other than P3D_OK, the same bytes from the same call, workspaces of
 * the size their *_workspace_size function returns (256-byte aligned, not
 * shared by calls that may overlap). Arithmetic is binary32 or wider.
 */
#ifndef P3D_MODEL_H
#define P3D_MODEL_H

#include "p3d_block.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Activations: SILU u / (1 + e^-u); GELU in its tanh form,
 * u (1 + tanh(sqrt(2 / pi) (u + 0.044715 u^3))) / 2. */
typedef enum p3d_act {
    P3D_ACT_NONE = 0,
    P3D_ACT_SILU = 1,
    P3D_ACT_GELU = 2
} p3d_act;

/* ------------------------------------------------------------------------
 * p3d_group_norm -- for item b (its rows: the pixels, cells or sparse tokens
 * of one map) and group g of channels / groups neighbouring channels:
 *   mean, var = over the item's rows and the group's channels
 *   rstd = 1 / sqrt(var + eps)
 *   out = act((x - mean) rstd weight[c] + bias[c])
 * var is the mean squared deviation. weight and bias may be NULL (1, 0).
 *
 *   channels     C: a multiple of 8 (BF16) or 4 (F32), up to 4096
 *   groups       a divisor of C
 *   x, out       [n, C] of dtype, rows x_stride / out_stride elements apart
 *                (>= C, a multiple of 8 / 4: a channel range of a wider map
 *                needs no copy); out may be x with equal strides and must not
 *                overlap it otherwise
 *   mean, rstd   float [batch, groups], or NULL; 0 and 1 / sqrt(eps) for an
 *                item without rows. The gradient needs both, of every item.
 *   Alignment: 16 bytes (mean, rstd: 4).
 *   workspace    p3d_group_norm_workspace_size(desc) bytes, for the forward
 *                call and the gradient alike
 * No result overlaps another tensor of the call (out in place apart).
 * A value that is not finite makes its item's group NaN. (Squared deviations
 * are binary32: values beyond 2^40 may end as one that is not finite would.)
 * --------------------------------------------------------------------- */
typedef struct p3d_group_desc {
    int64_t n;                  /* rows */
    const int64_t* offsets;     /* HOST [batch + 1] */
    int32_t batch;
    int32_t channels;
    int32_t groups;
    p3d_dtype dtype;            /* of x, out, weight, bias and their like */
    p3d_act act;
    float eps;                  /* finite, > 0 */
    const void* weight;         /* device [C] or NULL */
    const void* bias;           /* device [C] or NULL */
} p3d_group_desc;

size_t p3d_group_norm_workspace_size(const p3d_group_desc* desc);
p3d_status p3d_group_norm(const p3d_group_desc* desc, const void* x, int64_t x_stride, void* out,
                          int64_t out_stride, float* mean, float* rstd, void* workspace,
                          size_t workspace_bytes, void* stream);

/* p3d_group_norm_backward -- the gradients of p3d_group_norm from dout, the
 * forward call's x, and its mean and rstd. With x^ = (x - mean) rstd,
 * u = x^ weight + bias and du = dout act'(u):
 *   dbias = sum du,  dweight = sum du x^               (over all rows)
 *   dx = rstd (du weight - avg(du weight) - x^ avg(du weight x^))
 * avg: over the item's rows and the group's channels.
 *   dx             [n, C] of dtype; may be dout or x (with that tensor's
 *                  stride) and must not overlap them otherwise
 *   dweight, dbias float [C], each NULL where it is not wanted; overwritten,
 *                  0 where there are no rows
 * mean is a binary32 number here, and a more exact one within the forward call:
 * of a mean that is t deviations from 0, x^ is off by t 2^-25 in the gradient
 * alone.
 * No result overlaps another tensor of the call (dx in place apart). */
p3d_status p3d_group_norm_backward(const p3d_group_desc* desc, const void* dout,
                                   int64_t dout_stride, const void* x, int64_t x_stride,
                                   const float* mean, const float* rstd, void* dx,
                                   int64_t dx_stride, float* dweight, float* dbias,
                                   void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------
 * p3d_quantize_rows -- rows in 8-bit integers, a scale for each:
 *   scale[i] = max_k |x[i, k]| * c    (binary32; c: the number nearest to 1 / 127)
 *   q[i, k]  = x[i, k] / scale[i] to the nearest integer, ties to even
 * exactly (no rounding on the way). Tokens before a linear layer, or a weight
 * [out, in], whose scales are then its output channels'.
 * A row whose scale rounds to 0 gets q = 0, one with an entry that is not
 * finite scale = NaN and q = 0. (Scales below 2^-126 are held to few bits;
 * q is limited to +-127.)
 *
 *   dtype        F32 or BF16, of x
 *   width        K: a multiple of 16, 16..65536
 *   x            [n, K], rows x_stride (>= K, a multiple of 8 / 4) apart
 *   q            int8 [n, K], rows q_stride (>= K, a multiple of 16) apart
 *   scale        float [n]
 *   Alignment: 16 bytes (scale: 4). q and scale must not overlap each other
 *   or x.
 * --------------------------------------------------------------------- */
p3d_status p3d_quantize_rows(const void* x, p3d_dtype dtype, int64_t n, int32_t width,
                             int64_t x_stride, int8_t* q, int64_t q_stride, float* scale,
                             void* stream);

/* ------------------------------------------------------------------------
 * p3d_linear_i8 -- a linear layer on 8-bit integers:
 *   y[i, d] = (sum_k q[i, k] weight[d, k]) scale[i] weight_scale[d] + bias[d]
 *   out[i, d] = act(y[i, d]) + residual[i, d]
 * The sum is exact (32-bit integers on the matrix cores); what follows is
 * binary32, rounded once into out. -128 is allowed.
 *
 *   dtype        F32 or BF16, of out, bias and residual
 *   in_dim       K: a multiple of 16, 16..65536
 *   out_dim      D: a multiple of 8
 *   q            int8 [n, K], rows q_stride (>= K, a multiple of 16, at most
 *                2^22) apart
 *   weight       int8 [D, K] contiguous
 *   scale        float [n];  weight_scale: float [D]
 *   bias         [D] or NULL (0)
 *   residual     [n, D], rows residual_stride apart, or NULL (0); may be out
 *                with equal strides
 *   out          [n, D], rows out_stride (>= D, a multiple of 8 / 4) apart;
 *                must not overlap another tensor of the call
 *   Alignment: 16 bytes (scale, weight_scale: 4). n, D < 2^30, and their
 *   product, each rounded up to a multiple of 64, below 2^36.
 * --------------------------------------------------------------------- */
typedef struct p3d_linear_i8_desc {
    int64_t n;                  /* tokens */
    int32_t in_dim;
    int32_t out_dim;
    p3d_dtype dtype;
    p3d_act act;
    const int8_t* weight;
    const float* weight_scale;
    const void* bias;
} p3d_linear_i8_desc;

p3d_status p3d_linear_i8(const p3d_linear_i8_desc* desc, const int8_t* q, int64_t q_stride,
                         const float* scale, const void* residual, int64_t residual_stride,
                         void* out, int64_t out_stride, void* stream);

/* ------------------------------------------------------------------------
 * p3d_adamw -- one AdamW step over many tensors. For every element of every
 * tensor, with t = step and g = grad * grad_scale:
 *   m = beta1 m + (1 - beta1) g,   v = beta2 v + (1 - beta2) g^2
 *   w = w (1 - lr weight_decay)
 *       - lr / (1 - beta1^t) * m / (sqrt(v) / sqrt(1 - beta2^t) + eps)
 * in binary32 (the factors in binary64, rounded once). States in 8 bits are
 * reproducible bit for bit: m = (b1 m) + (c1 g), v = (b2 v) + ((c2 g) g) and
 * sqrt(v) take one rounding an operation, c = 1 - b.
 *
 * weights      param, of param_dtype. With a master (binary32, same size; for
 *              BF16 params), the step updates the master and param is the
 *              master rounded. Without one, param is updated and rounded.
 * state_bits   32: m and v are float [size]. 8: m holds m, and v holds
 *              sqrt(v), as e4m3 numbers [size] (1 sign, 4 exponent bits of
 *              bias 7, 3 mantissa bits) of which each block of 256 elements
 *              shares a scale, m_scale and v_scale, float [(size + 255) / 256]:
 *              the state is number * scale (v: its square). After a step a
 *              block's scale is its largest state times the number nearest to
 *              1 / 448, its states are multiplied by (1 / largest) 448, and one
 *              between two numbers goes to the upper one where 16 random bits
 *              say so (the one below otherwise): on average the state is kept,
 *              which rounding to nearest would not do for changes smaller than
 *              half a step. A
 *              sqrt(v) that is not 0 never becomes 0. A block whose largest
 *              state is below 2^-100 holds zeros; one with an element that is
 *              not finite holds none that is. The step itself uses m and v
 *              before they are rounded.
 * random bits  of the element with index i of tensor number j under `seed`,
 *              all in 32-bit arithmetic, with
 *                mix(x): x ^= x >> 15;  x *= 0xB504F335;  x ^= x >> 13;
 *                        x *= 0xDDB3D743;  x ^= x >> 16
 *                key = mix(j * 0x9E3779B1 ^ mix(low(seed)) ^ high(seed))
 *                x = mix(low(i) * 0x9E3779B1 ^ high(i) * 0xDDB3D743 ^ key)
 *              are x's low half for m and its high half for v: a number with
 *              20 mantissa bits to drop gets the 16 bits added into the upper
 *              ones of those. A step needs a seed of its own: with a
 *              device_step, the step's number is added to `seed` first, so that
 *              a captured graph's replays have theirs.
 * grad_scale   DEVICE float or NULL (1). Where it is not finite the whole
 *              step is left out: nothing is written.
 * device_lr, device_step: DEVICE float / int32, or NULL; read by the kernels
 *              instead of lr / step, so that a captured graph replays with
 *              their values of the time. A device step below 1 counts as 1.
 *
 *   count        tensors, 0..65536; their table is a HOST array and travels in
 *                kernel arguments, 64 tensors a launch
 *   tensors      size >= 0 elements each, below 2^34; no two tensors of the
 *                table, nor two parts of one, may overlap in what a step
 *                writes, nor overlap a gradient or a device scalar
 *   lr           finite, >= 0; beta1, beta2 in [0, 1); eps finite, > 0;
 *   step         >= 1 (its value is used without device_step)
 *   weight_decay finite, per tensor
 * eps is what binary32 makes of it: the smallest is 2^-149, below the normal
 * numbers.
 *   Alignment: 16 bytes (the scales and device scalars: 4).
 * --------------------------------------------------------------------- */
typedef struct p3d_adamw_tensor {
    void* param;                /* [size] of param_dtype */
    float* master;              /* [size], or NULL in every tensor */
    const void* grad;           /* [size] of grad_dtype */
    void* m;                    /* [size]: float, or e4m3 */
    void* v;                    /* [size]: float, or e4m3 (of sqrt(v)) */
    float* m_scale;             /* 8 bits: [(size + 255) / 256]; 32: NULL */
    float* v_scale;
    int64_t size;
    float weight_decay;
} p3d_adamw_tensor;

typedef struct p3d_adamw_desc {
    int32_t count;
    const p3d_adamw_tensor* tensors;    /* HOST [count] */
    p3d_dtype param_dtype;
    p3d_dtype grad_dtype;
    int32_t state_bits;                 /* 32 or 8 */
    double lr, beta1, beta2, eps;
    int64_t step;
    uint64_t seed;                      /* 8 bits: of the random bits */
    const float* grad_scale;
    const float* device_lr;
    const int32_t* device_step;
} p3d_adamw_desc;

p3d_status p3d_adamw(const p3d_adamw_desc* desc, void* stream);

/* p3d_grad_norm -- the norm over every tensor's gradient, and the factor that
 * clips it, for p3d_adamw's grad_scale:
 *   out[0] = norm = sqrt(sum of squares)   (summed in binary64)
 *   out[1] = norm > max_norm ? max_norm / norm : 1;  NaN where out[0] is not
 *            finite (a norm beyond binary32 among them), so that the step is
 *            left out
 * out: DEVICE float [2], no part of a gradient. Of desc, count, grad_dtype and the tensors' grad and
 * size are read. max_norm > 0 (infinity: no clipping).
 * workspace: p3d_grad_norm_workspace_size(desc) bytes. */
size_t p3d_grad_norm_workspace_size(const p3d_adamw_desc* desc);
p3d_status p3d_grad_norm(const p3d_adamw_desc* desc, float max_norm, float* out, void* workspace,
                         size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* P3D_MODEL_H */
