/*
 * p3d_block.h -- the operators of the transformer block that the
 * conditioning goes into (libp3d, gfx950): the gated norm between a block's
 * branches, rotary positions, and attention, each with its gradient.
 *
 * The flow transformers that p3d_proj_cond feeds add proj_linear's output
 * into a block's residual (trellis.cpp PR #38, commit adding proj mode to the
 * DiT). Around that addition every block normalises its residual stream under
 * a per-item modulation, rotates rms-normed queries and keys by the tokens'
 * grid coordinates, and attends over the sparse tokens of each batch item and
 * over a few global tokens (pixal3d_mrp_mlx README: rope_phases_from_coords,
 * qk_rms_norm before RoPE, AdaLN modulation).
 *
 * The conventions of p3d.h hold: DEVICE pointers owned by the caller, no
 * allocation, work enqueued on `stream` without synchronising, nothing
 * enqueued on any status other than P3D_OK, p3d_last_error() names the
 * argument. In addition:
 *   - Item tables (offsets) are HOST arrays, read during the call only; they
 *     travel in the kernel arguments, so a captured graph replays the table
 *     it was captured with. offsets[b] .. offsets[b + 1] are item b's rows;
 *     offsets[0] must be 0, entries must not decrease (items may be empty),
 *     and the last entry is the number of rows. 1 <= batch <= P3D_MAX_BATCH.
 *   - Descriptors are HOST structs, read during the call only.
 *   - Sums, norms, softmax statistics and all arithmetic are binary32 or
 *     wider; BF16 results are rounded once, to nearest even, except where a
 *     call says that a factor of a matrix product is rounded first.
 *   - Results do not depend on the order in which the device runs the work:
 *     the same call on the same data writes the same bytes.
 *   - Workspaces are DEVICE buffers of the size the call's
 *     *_workspace_size function returns for the same arguments (0 there:
 *     invalid arguments, p3d_last_error() says which), 256-byte aligned,
 *     contents undefined on entry and on return, not shared by calls that
 *     may overlap.
 */
#ifndef P3D_BLOCK_H
#define P3D_BLOCK_H

#include "p3d.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------
 * p3d_gated_norm -- the step between two branches of a block: the finished
 * branch's output y is normalised (sandwich norm, optional), gated and added
 * to the residual stream x, and the sum is normalised and modulated for the
 * next branch. For row i of item b and every column c, with s = res_scale:
 *   t = post(y) * post_weight            (post NONE: t = y)
 *   r = x + s * gate[b] * t              (y NULL: r = x)
 *   h = (pre(r) * weight + bias) * (1 + scale[b]) + shift[b]
 * where LAYER is (v - mean v) / sqrt(var v + eps), var the mean squared
 * deviation, and RMS is v / sqrt(mean v^2 + eps), over the row's columns.
 * pre takes r before it is rounded. Any of gate, scale, shift, weight, bias
 * and post_weight may be NULL (1, 0, 0, 1, 0, 1).
 *
 *   dim          columns D: a multiple of 8 (BF16) or 4 (F32), 1..8192
 *   mod_stride   elements between the items' rows of gate, scale and shift
 *                (D for separate [batch, D] tensors, 6 D inside a packed
 *                [batch, 6, D]); >= D, a multiple of 8 / 4 where batch > 1
 *   x, y         [n, D] contiguous, of `dtype`; y may be NULL (post and gate
 *                are then not used)
 *   r            [n, D] or NULL (not written); may be x or y
 *   h            [n, D]; may be x or y
 *   Alignment: 16 bytes for every tensor.
 * --------------------------------------------------------------------- */
typedef enum p3d_norm_kind {
    P3D_NORM_NONE = 0,
    P3D_NORM_LAYER = 1,
    P3D_NORM_RMS = 2
} p3d_norm_kind;

typedef struct p3d_norm_desc {
    int64_t n;                  /* rows */
    const int64_t* offsets;     /* HOST [batch + 1] */
    int32_t batch;
    int32_t dim;
    p3d_dtype dtype;            /* of every tensor but the parameter gradients */
    p3d_norm_kind pre;          /* LAYER or RMS */
    p3d_norm_kind post;         /* NONE, LAYER or RMS */
    float res_scale;            /* finite */
    float eps;                  /* finite, > 0 */
    int64_t mod_stride;
    const void* gate;           /* device [batch, D] by mod_stride, or NULL */
    const void* scale;          /* device [batch, D] by mod_stride, or NULL */
    const void* shift;          /* device [batch, D] by mod_stride, or NULL */
    const void* weight;         /* device [D] or NULL */
    const void* bias;           /* device [D] or NULL */
    const void* post_weight;    /* device [D] or NULL; NULL when post is NONE */
} p3d_norm_desc;

p3d_status p3d_gated_norm(const p3d_norm_desc* desc, const void* x, const void* y, void* r,
                          void* h, void* stream);

/* p3d_gated_norm_backward -- the gradients of p3d_gated_norm. dh is the
 * gradient of h, dr the gradient that reaches r by its other uses (the
 * residual path; NULL: none). r, the norms and their statistics are
 * recomputed from x and y, so nothing else need be kept from the forward
 * call. desc is the forward call's (shift is not read).
 *   dx          [n, D] of dtype: the gradient of x, which is r's whole
 *               gradient; may be dh, dr or x
 *   dy          [n, D] of dtype, or NULL; may be y (needs y)
 * and binary32 parameter gradients, each NULL where it is not wanted:
 *   dgate, dscale, dshift        [batch, D] contiguous (dgate needs y)
 *   dweight, dbias, dpost_weight [D] (dpost_weight needs y)
 * Parameter gradients are overwritten; those of an item without rows are 0.
 * workspace: p3d_gated_norm_workspace_size(desc) bytes. */
size_t p3d_gated_norm_workspace_size(const p3d_norm_desc* desc);
p3d_status p3d_gated_norm_backward(const p3d_norm_desc* desc, const void* dh, const void* dr,
                                   const void* x, const void* y, void* dx, void* dy,
                                   float* dgate, float* dscale, float* dshift, float* dweight,
                                   float* dbias, float* dpost_weight, void* workspace,
                                   size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------
 * p3d_rotary -- rotary positions of query and key heads, with the rms norm
 * that stands before them. For token t, head j and m = magnitude:
 *   x^ = x / sqrt(mean x^2 + eps) * gamma[j]     (gamma NULL: x^ = x)
 * then pair p = a * pairs + i (axis a, frequency i) turns by the angle
 * positions[t, a] * freqs[i]:
 *   (u, w) -> m (u cos - w sin, u sin + w cos)
 * with (u, w) = elements (2p, 2p + 1) of the head (INTERLEAVED) or
 * (p, p + axes * pairs) (HALF). Elements from 2 * axes * pairs on keep x^.
 * The angle is reduced in binary64, so long contexts lose nothing.
 *
 *   x, out       [n, heads, head_dim] of dtype; head_dim elements of a head
 *                and the heads of a token are contiguous, tokens are
 *                x_stride / out_stride elements apart (a multiple of 8 BF16 /
 *                4 F32), so the query and key heads of a packed qkv are one
 *                call; out may be x (with equal strides)
 *   head_dim     a multiple of 8, 8..256; heads 1..1024
 *   positions    DEVICE int32 [n, axes], rows pos_stride (>= axes) apart:
 *                coords + 1 with pos_stride 4 takes the grid cell (x, y, z) of
 *                [n, 4] coords; 1 <= axes <= 3
 *   freqs        DEVICE float [pairs], radians per position, one table for
 *                every axis; pairs >= 1, 2 * axes * pairs <= head_dim
 *   gamma        DEVICE [heads, head_dim] of dtype, or NULL
 *   Alignment: 16 bytes (positions, freqs: 4).
 * --------------------------------------------------------------------- */
typedef enum p3d_rotary_layout {
    P3D_ROTARY_INTERLEAVED = 0,
    P3D_ROTARY_HALF = 1
} p3d_rotary_layout;

typedef struct p3d_rotary_desc {
    int64_t n;                  /* tokens */
    int32_t heads;
    int32_t head_dim;
    p3d_dtype dtype;
    p3d_rotary_layout layout;
    int32_t axes;
    int32_t pairs;              /* per axis */
    int32_t pos_stride;
    float magnitude;            /* finite */
    float eps;                  /* finite, > 0 */
    const int32_t* positions;
    const float* freqs;
    const void* gamma;
} p3d_rotary_desc;

p3d_status p3d_rotary(const p3d_rotary_desc* desc, const void* x, int64_t x_stride, void* out,
                      int64_t out_stride, void* stream);

/* p3d_rotary_backward -- the gradients of p3d_rotary from dout, the gradient
 * of out. dx may be dout or x (with that tensor's stride). With gamma, x is
 * the forward call's input and dgamma (binary32 [heads, head_dim], NULL: not
 * wanted) is overwritten; without gamma, x is not read (NULL) and dgamma must
 * be NULL. workspace: p3d_rotary_workspace_size(desc) bytes, needed (not
 * NULL) only with dgamma. */
size_t p3d_rotary_workspace_size(const p3d_rotary_desc* desc);
p3d_status p3d_rotary_backward(const p3d_rotary_desc* desc, const void* dout,
                               int64_t dout_stride, const void* x, int64_t x_stride, void* dx,
                               int64_t dx_stride, float* dgamma, void* workspace,
                               size_t workspace_bytes, void* stream);

/* p3d_rotary_frequencies -- a frequency table, on the HOST, computed in
 * binary64 and rounded once. With f_i = base^(-i / pairs), i in [0, pairs):
 *   P3D_ROTARY_PLAIN      f_i
 *   P3D_ROTARY_LINEAR     f_i / factor (positions interpolated)
 *   P3D_ROTARY_BASE       f_i with base * factor^(pairs / (pairs - 1)): the
 *                         fastest pair keeps its frequency, the slowest is
 *                         divided by factor; pairs >= 2
 *   P3D_ROTARY_BY_PARTS   f_i k + (f_i / factor) (1 - k), where a pair that
 *                         makes w = trained f_i / (2 pi) turns over the
 *                         trained length keeps k = clamp((w - 1) / 31, 0, 1)
 *                         of its frequency
 *   base > 1 and factor >= 1, finite; trained >= 1 positions (BY_PARTS only);
 *   1 <= pairs <= 128; freqs: HOST [pairs]. */
typedef enum p3d_rotary_scaling {
    P3D_ROTARY_PLAIN = 0,
    P3D_ROTARY_LINEAR = 1,
    P3D_ROTARY_BASE = 2,
    P3D_ROTARY_BY_PARTS = 3
} p3d_rotary_scaling;

p3d_status p3d_rotary_frequencies(double base, int32_t pairs, p3d_rotary_scaling scaling,
                                  double factor, double trained, float* freqs);

/* ------------------------------------------------------------------------
 * p3d_attention -- softmax attention over the items' own rows, query heads
 * sharing key heads in groups of heads / kv_heads. For query i and key j of
 * one item (numbered within it), query head a and key head a / group:
 *   s_ij = scale * q_i . k_j      for the keys that query i sees
 *   out_i = sum_j exp(s_ij - lse_i) v_j,   lse_i = log sum_j exp(s_ij)
 * Every key is seen; with `causal`, key j is seen when j <= i + nk - nq (the
 * last query sees every key; a single query over a filled cache sees it
 * all). A query that sees no key gets out = 0 and lse = -inf. Keys and values
 * of other items and past the last row are not read. Under `causal` a value
 * that is not finite reaches the item's queries that do not see it, too (its
 * weight 0 still multiplies it).
 *
 * The products run on the matrix cores with binary32 accumulation; the
 * probabilities are rounded to bf16 as factors of the second product, their
 * sum is not.
 *
 *   dtype        BF16 only (P3D_ERR_UNSUPPORTED otherwise)
 *   q, out       [nq, heads, head_dim]; k, v [nk, kv_heads, head_dim], nq and
 *                nk the last entries of q_offsets and k_offsets; a token's
 *                heads are contiguous, tokens are *_stride elements apart (a
 *                multiple of 8), so views of a packed qkv need no copy;
 *                out may be q with equal strides, and must not overlap q
 *                otherwise, nor k or v (checked as the gradients' tensors are)
 *   head_dim     a multiple of 8, 8..128; heads a multiple of kv_heads,
 *                heads <= 1024
 *   scale        finite, > 0, at most 2^127 (the gradient: at least 2^-100)
 *   lse          float [nq, heads] (natural logarithm) or NULL
 *   Alignment: 16 bytes (lse: 4). nq * heads and nk * kv_heads < 2^30.
 *   workspace    p3d_attention_workspace_size(desc) bytes (few queries over
 *                many keys are split along the keys and joined through it)
 * --------------------------------------------------------------------- */
typedef struct p3d_attn_desc {
    const int64_t* q_offsets;   /* HOST [batch + 1] */
    const int64_t* k_offsets;   /* HOST [batch + 1] */
    int32_t batch;
    int32_t heads;
    int32_t kv_heads;
    int32_t head_dim;
    p3d_dtype dtype;
    float scale;
    int32_t causal;             /* 0 or 1 */
} p3d_attn_desc;

size_t p3d_attention_workspace_size(const p3d_attn_desc* desc);
p3d_status p3d_attention(const p3d_attn_desc* desc, const void* q, int64_t q_stride,
                         const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                         void* out, int64_t out_stride, float* lse, void* workspace,
                         size_t workspace_bytes, void* stream);

/* p3d_attention_backward -- the gradients of p3d_attention from dout, out and
 * lse as the forward call wrote it. The probabilities P are recomputed:
 *   D_i = dout_i . out_i,  dS_ij = P_ij (dout_i . v_j - D_i)
 *   dq_i = scale sum_j dS_ij k_j,  dk_j = scale sum_i dS_ij q_i,
 *   dv_j = sum_i P_ij dout_i       (dk, dv: summed over the group's heads)
 * P and dS are rounded to bf16 as factors of the last three products (dS of
 * queries that see at most 256 keys, and of those that share one of the
 * launch's 128-row tiles with such a query, for dq, as the sum of two bf16
 * numbers). dk, and dq of items of at most 64 keys, take D_i as sum_j P_ij
 * dout_i . v_j, the same number without out's rounding. Rows that nothing
 * reaches get 0, and so does dq of a query that sees one key (its probability is
 * 1). Entries that are not finite reach, as in the forward call, every result of
 * their item that takes them with weight 0.
 * dq, dk and dv are strided like q, k and v, are overwritten and must not
 * overlap another tensor of the call (P3D_ERR_INVALID_ARG where the two have
 * equal strides, one has a single row or both start at one place; not looked for
 * otherwise). */
size_t p3d_attention_backward_workspace_size(const p3d_attn_desc* desc);
p3d_status p3d_attention_backward(const p3d_attn_desc* desc, const void* dout,
                                  int64_t dout_stride, const void* q, int64_t q_stride,
                                  const void* k, int64_t k_stride, const void* v,
                                  int64_t v_stride, const void* out, int64_t out_stride,
                                  const float* lse, void* dq, int64_t dq_stride, void* dk,
                                  int64_t dk_stride, void* dv, int64_t dv_stride,
                                  void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* P3D_BLOCK_H */
