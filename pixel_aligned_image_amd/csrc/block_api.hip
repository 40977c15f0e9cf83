// block_api.hip -- the extern "C" entry points of include/p3d_block.h:
// validation of every argument before anything is enqueued, workspace sizes,
// the frequency tables, and dispatch to the kernels.
#include <math.h>
#include <stdio.h>

#include "block_internal.h"

using namespace p3d;

namespace {

constexpr int64_t kMaxRows = int64_t(1) << 30;     // rows and offsets are int32 in the kernels

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

p3d_status hip_fail(const char* fn, hipError_t e) {
    return set_error(P3D_ERR_HIP, "%s: HIP launch failed: %s", fn, hipGetErrorString(e));
}

p3d_status check_dtype(const char* fn, p3d_dtype dt) {
    if (dt != P3D_F32 && dt != P3D_BF16)
        return set_error(P3D_ERR_DTYPE, "%s: dtype must be F32 or BF16, got %d", fn, (int)dt);
    return P3D_OK;
}

// A required (or, `needed` false, optional) device tensor.
p3d_status check_tensor(const char* fn, const char* name, const void* p, bool needed,
                        size_t align = 16) {
    if (needed && !p) return set_error(P3D_ERR_INVALID_ARG, "%s: %s is NULL", fn, name);
    if (!aligned(p, align))
        return set_error(P3D_ERR_UNSUPPORTED, "%s: %s must be %zu-byte aligned, got %p", fn, name,
                         align, p);
    return P3D_OK;
}

p3d_status check_items(const char* fn, const char* name, const int64_t* offsets, int32_t batch,
                       ItemTable* t) {
    if (batch < 1 || batch > P3D_MAX_BATCH)
        return set_error(P3D_ERR_INVALID_ARG, "%s: batch must be in [1, %d], got %d", fn,
                         P3D_MAX_BATCH, batch);
    if (!offsets)
        return set_error(P3D_ERR_INVALID_ARG, "%s: %s is NULL (host array [batch + 1])", fn, name);
    if (offsets[0] != 0)
        return set_error(P3D_ERR_INVALID_ARG, "%s: %s[0] must be 0, got %lld", fn, name,
                         (long long)offsets[0]);
    for (int32_t b = 0; b < batch; ++b) {
        if (offsets[b + 1] < offsets[b])
            return set_error(P3D_ERR_INVALID_ARG,
                             "%s: %s must not decrease, got %s[%d] = %lld after %lld", fn, name,
                             name, b + 1, (long long)offsets[b + 1], (long long)offsets[b]);
        if (offsets[b + 1] > kMaxRows)
            return set_error(P3D_ERR_UNSUPPORTED, "%s: %s[%d] must be <= %lld, got %lld", fn, name,
                             b + 1, (long long)kMaxRows, (long long)offsets[b + 1]);
        t->start[b] = (int32_t)offsets[b];
    }
    for (int32_t b = batch; b <= P3D_MAX_BATCH; ++b) t->start[b] = (int32_t)offsets[batch];
    return P3D_OK;
}

p3d_status check_workspace(const char* fn, const char* size_fn, const void* ws, size_t got,
                           size_t need) {
    if (!ws || got < need)
        return set_error(P3D_ERR_INVALID_ARG,
                         "%s: workspace must be a device buffer of at least %zu bytes (%s), got "
                         "%zu bytes at %p", fn, need, size_fn, got, ws);
    if (!aligned(ws, 256))
        return set_error(P3D_ERR_UNSUPPORTED, "%s: workspace must be 256-byte aligned", fn);
    return P3D_OK;
}

#define P3D_TRY(call)                     \
    do {                                  \
        const p3d_status st_ = (call);    \
        if (st_ != P3D_OK) return st_;    \
    } while (0)

// ------------------------------------------------------------- gated norm ---
p3d_status check_norm(const char* fn, const p3d_norm_desc* d, NormArgs* a, ItemTable* items) {
    if (!d) return set_error(P3D_ERR_INVALID_ARG, "%s: desc is NULL", fn);
    P3D_TRY(check_dtype(fn, d->dtype));
    const int epv = d->dtype == P3D_BF16 ? 8 : 4;
    if (d->n < 0 || d->n > kMaxRows)
        return set_error(P3D_ERR_INVALID_ARG, "%s: n must be in [0, %lld], got %lld", fn,
                         (long long)kMaxRows, (long long)d->n);
    P3D_TRY(check_items(fn, "offsets", d->offsets, d->batch, items));
    if (d->offsets[d->batch] != d->n)
        return set_error(P3D_ERR_SHAPE, "%s: offsets[%d] must be n = %lld, got %lld", fn,
                         d->batch, (long long)d->n, (long long)d->offsets[d->batch]);
    if (d->dim < 1)
        return set_error(P3D_ERR_INVALID_ARG, "%s: dim must be >= 1, got %d", fn, d->dim);
    if (d->dim % epv || d->dim > 8192)
        return set_error(P3D_ERR_UNSUPPORTED,
                         "%s: dim must be a multiple of %d up to 8192, got %d", fn, epv, d->dim);
    if (d->pre != P3D_NORM_LAYER && d->pre != P3D_NORM_RMS)
        return set_error(P3D_ERR_INVALID_ARG, "%s: pre must be LAYER or RMS, got %d", fn,
                         (int)d->pre);
    if (d->post != P3D_NORM_NONE && d->post != P3D_NORM_LAYER && d->post != P3D_NORM_RMS)
        return set_error(P3D_ERR_INVALID_ARG, "%s: post must be NONE, LAYER or RMS, got %d", fn,
                         (int)d->post);
    if (!isfinite(d->res_scale))
        return set_error(P3D_ERR_INVALID_ARG, "%s: res_scale must be finite, got %g", fn,
                         (double)d->res_scale);
    if (!(isfinite(d->eps) && d->eps > 0.f))
        return set_error(P3D_ERR_INVALID_ARG, "%s: eps must be finite and > 0, got %g", fn,
                         (double)d->eps);
    if (d->post == P3D_NORM_NONE && d->post_weight)
        return set_error(P3D_ERR_INVALID_ARG,
                         "%s: post_weight must be NULL when post is NONE", fn);
    if ((d->gate || d->scale || d->shift) && d->batch > 1) {
        if (d->mod_stride < d->dim)
            return set_error(P3D_ERR_SHAPE, "%s: mod_stride must be >= dim = %d, got %lld", fn,
                             d->dim, (long long)d->mod_stride);
        if (d->mod_stride % epv || d->mod_stride > (int64_t(1) << 40))
            return set_error(P3D_ERR_UNSUPPORTED,
                             "%s: mod_stride must be a multiple of %d up to 2^40, got %lld", fn,
                             epv, (long long)d->mod_stride);
    }
    P3D_TRY(check_tensor(fn, "gate", d->gate, false));
    P3D_TRY(check_tensor(fn, "scale", d->scale, false));
    P3D_TRY(check_tensor(fn, "shift", d->shift, false));
    P3D_TRY(check_tensor(fn, "weight", d->weight, false));
    P3D_TRY(check_tensor(fn, "bias", d->bias, false));
    P3D_TRY(check_tensor(fn, "post_weight", d->post_weight, false));
    *a = NormArgs{};
    a->gate = d->gate;
    a->scale = d->scale;
    a->shift = d->shift;
    a->weight = d->weight;
    a->bias = d->bias;
    a->post_weight = d->post_weight;
    a->n = d->n;
    a->mod_stride = d->batch > 1 ? d->mod_stride : 0;
    a->batch = d->batch;
    a->dim = d->dim;
    a->pre = d->pre;
    a->post = d->post;
    a->res_scale = d->res_scale;
    a->eps = d->eps;
    return P3D_OK;
}

size_t norm_workspace(const NormArgs& a, const ItemTable& items) {
    ItemTable chunks;
    norm_chunks(a.n, a.batch, items, &chunks);
    const size_t rows = (size_t)chunks.start[a.batch] + (size_t)a.batch;
    return (rows * 3 * (size_t)a.dim * sizeof(float) + 255) / 256 * 256;
}

// ----------------------------------------------------------------- rotary ---
p3d_status check_rotary(const char* fn, const p3d_rotary_desc* d, RotaryArgs* a) {
    if (!d) return set_error(P3D_ERR_INVALID_ARG, "%s: desc is NULL", fn);
    P3D_TRY(check_dtype(fn, d->dtype));
    if (d->n < 0 || d->n > kMaxRows)
        return set_error(P3D_ERR_INVALID_ARG, "%s: n must be in [0, %lld], got %lld", fn,
                         (long long)kMaxRows, (long long)d->n);
    if (d->heads < 1 || d->heads > 1024)
        return set_error(P3D_ERR_INVALID_ARG, "%s: heads must be in [1, 1024], got %d", fn,
                         d->heads);
    if (d->head_dim < 8 || d->head_dim % 8 || d->head_dim > 256)
        return set_error(P3D_ERR_UNSUPPORTED,
                         "%s: head_dim must be a multiple of 8 in [8, 256], got %d", fn,
                         d->head_dim);
    if (d->layout != P3D_ROTARY_INTERLEAVED && d->layout != P3D_ROTARY_HALF)
        return set_error(P3D_ERR_INVALID_ARG, "%s: layout must be INTERLEAVED or HALF, got %d", fn,
                         (int)d->layout);
    if (d->axes < 1 || d->axes > 3)
        return set_error(P3D_ERR_INVALID_ARG, "%s: axes must be in [1, 3], got %d", fn, d->axes);
    if (d->pairs < 1 || (int64_t)2 * d->axes * d->pairs > d->head_dim)
        return set_error(P3D_ERR_SHAPE,
                         "%s: pairs must be >= 1 with 2 * axes * pairs <= head_dim: got %d axes x "
                         "%d pairs in a head of %d", fn, d->axes, d->pairs, d->head_dim);
    if (d->pos_stride < d->axes)
        return set_error(P3D_ERR_SHAPE, "%s: pos_stride must be >= axes = %d, got %d", fn,
                         d->axes, d->pos_stride);
    if (!isfinite(d->magnitude))
        return set_error(P3D_ERR_INVALID_ARG, "%s: magnitude must be finite, got %g", fn,
                         (double)d->magnitude);
    if (!(isfinite(d->eps) && d->eps > 0.f))
        return set_error(P3D_ERR_INVALID_ARG, "%s: eps must be finite and > 0, got %g", fn,
                         (double)d->eps);
    P3D_TRY(check_tensor(fn, "positions", d->positions, d->n > 0, 4));
    P3D_TRY(check_tensor(fn, "freqs", d->freqs, d->n > 0, 4));
    P3D_TRY(check_tensor(fn, "gamma", d->gamma, false));
    *a = RotaryArgs{};
    a->gamma = d->gamma;
    a->positions = d->positions;
    a->freqs = d->freqs;
    a->n = d->n;
    a->heads = d->heads;
    a->head_dim = d->head_dim;
    a->axes = d->axes;
    a->pairs = d->pairs;
    a->pos_stride = d->pos_stride;
    a->layout = d->layout;
    a->magnitude = d->magnitude;
    a->eps = d->eps;
    return P3D_OK;
}

p3d_status check_stride(const char* fn, const char* name, int64_t stride, int64_t width,
                        int epv) {
    if (stride < width)
        return set_error(P3D_ERR_SHAPE,
                         "%s: %s must be >= heads * head_dim = %lld, got %lld", fn, name,
                         (long long)width, (long long)stride);
    if (stride % epv || stride > (int64_t(1) << 30))
        return set_error(P3D_ERR_UNSUPPORTED,
                         "%s: %s must be a multiple of %d up to 2^30, got %lld", fn, name, epv,
                         (long long)stride);
    return P3D_OK;
}

// -------------------------------------------------------------- attention ---
p3d_status check_attention(const char* fn, const p3d_attn_desc* d, AttnArgs* a) {
    if (!d) return set_error(P3D_ERR_INVALID_ARG, "%s: desc is NULL", fn);
    P3D_TRY(check_dtype(fn, d->dtype));
    if (d->dtype != P3D_BF16)
        return set_error(P3D_ERR_UNSUPPORTED, "%s: only BF16 is supported, got F32", fn);
    if (d->kv_heads < 1 || d->heads < d->kv_heads || d->heads > 1024)
        return set_error(P3D_ERR_INVALID_ARG,
                         "%s: needs 1 <= kv_heads <= heads <= 1024, got %d and %d", fn,
                         d->kv_heads, d->heads);
    if (d->heads % d->kv_heads)
        return set_error(P3D_ERR_SHAPE, "%s: heads must be a multiple of kv_heads, got %d and %d",
                         fn, d->heads, d->kv_heads);
    if (d->head_dim < 8 || d->head_dim % 8 || d->head_dim > 128)
        return set_error(P3D_ERR_UNSUPPORTED,
                         "%s: head_dim must be a multiple of 8 in [8, 128], got %d", fn,
                         d->head_dim);
    if (!(isfinite(d->scale) && d->scale > 0.f))
        return set_error(P3D_ERR_INVALID_ARG, "%s: scale must be finite and > 0, got %g", fn,
                         (double)d->scale);
    if (d->scale > 0x1p127f)                 // scale log2(e) has to be finite
        return set_error(P3D_ERR_UNSUPPORTED, "%s: scale must be at most 2^127, got %g", fn,
                         (double)d->scale);
    if (d->causal != 0 && d->causal != 1)
        return set_error(P3D_ERR_INVALID_ARG, "%s: causal must be 0 or 1, got %d", fn, d->causal);
    *a = AttnArgs{};
    P3D_TRY(check_items(fn, "q_offsets", d->q_offsets, d->batch, &a->q_items));
    P3D_TRY(check_items(fn, "k_offsets", d->k_offsets, d->batch, &a->k_items));
    const int64_t nq = d->q_offsets[d->batch], nk = d->k_offsets[d->batch];
    if (nq * d->heads >= kMaxRows || nk * d->kv_heads >= kMaxRows)
        return set_error(P3D_ERR_UNSUPPORTED,
                         "%s: queries * heads and keys * kv_heads must be below 2^30, got %lld * "
                         "%d and %lld * %d", fn, (long long)nq, d->heads, (long long)nk,
                         d->kv_heads);
    a->batch = d->batch;
    a->heads = d->heads;
    a->kv_heads = d->kv_heads;
    a->head_dim = d->head_dim;
    a->causal = d->causal;
    a->scale = d->scale;
    return P3D_OK;
}

// The gradient divides lse by the scale, which has to stay finite.
p3d_status check_attention_backward(const char* fn, const p3d_attn_desc* d, AttnArgs* a) {
    P3D_TRY(check_attention(fn, d, a));
    if (d->scale < 0x1p-100f)
        return set_error(P3D_ERR_UNSUPPORTED, "%s: scale must be at least 2^-100, got %g", fn,
                         (double)d->scale);
    return P3D_OK;
}

// The bytes of a [rows, width] tensor, rows `pitch` bytes apart.
struct Rows {
    const char* name;
    const void* base;
    int64_t rows, width, pitch;
};

int64_t floor_div(int64_t a, int64_t b) { return a >= 0 ? a / b : -((b - 1 - a) / b); }

// Whether the single row `a` shares a byte with `b`: the first of b's rows that
// ends behind a's start begins before a's end.
bool row_meets(const Rows& a, const Rows& b) {
    const int64_t at = static_cast<const char*>(a.base) - static_cast<const char*>(b.base);
    const int64_t row = at < b.width ? 0 : floor_div(at - b.width, b.pitch) + 1;
    return row < b.rows && row * b.pitch < at + a.width;
}

// Whether two tensors share a byte: decided where their rows are equally far
// apart (views of one packed buffer), one of them has a single row, or both
// start at one place.
bool overlap(const Rows& a, const Rows& b) {
    if (a.rows == 0 || b.rows == 0) return false;
    if (a.base == b.base) return true;
    if (a.rows == 1) return row_meets(a, b);
    if (b.rows == 1) return row_meets(b, a);
    if (a.pitch != b.pitch) return false;
    // b's row 0 starts `column` bytes into row `down` of a's raster
    const int64_t apart = static_cast<const char*>(b.base) - static_cast<const char*>(a.base);
    const int64_t down = floor_div(apart, a.pitch), column = apart - down * a.pitch;
    const auto meet = [&](int64_t by) { return by < a.rows && by + b.rows > 0; };
    return (column < a.width && meet(down)) || (column + b.width > a.pitch && meet(down + 1));
}

p3d_status check_apart(const char* fn, const Rows& written, const Rows& other) {
    if (overlap(written, other))
        return set_error(P3D_ERR_INVALID_ARG, "%s: %s must not overlap %s", fn, written.name,
                         other.name);
    return P3D_OK;
}

}  // namespace

extern "C" {

p3d_status p3d_gated_norm(const p3d_norm_desc* desc, const void* x, const void* y, void* r,
                          void* h, void* stream) {
    const char* fn = "p3d_gated_norm";
    NormArgs a;
    ItemTable items;
    P3D_TRY(check_norm(fn, desc, &a, &items));
    P3D_TRY(check_tensor(fn, "x", x, a.n > 0));
    P3D_TRY(check_tensor(fn, "y", y, false));
    P3D_TRY(check_tensor(fn, "r", r, false));
    P3D_TRY(check_tensor(fn, "h", h, a.n > 0));
    if (r && r == h)
        return set_error(P3D_ERR_INVALID_ARG, "%s: r and h must be different tensors", fn);
    if (a.n == 0) return set_ok();
    a.x = x;
    a.y = y;
    a.r = r;
    a.h = h;
    const hipError_t e =
        launch_gated_norm(a, desc->dtype, items, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? set_ok() : hip_fail(fn, e);
}

size_t p3d_gated_norm_workspace_size(const p3d_norm_desc* desc) {
    NormArgs a;
    ItemTable items;
    if (check_norm("p3d_gated_norm_workspace_size", desc, &a, &items) != P3D_OK) return 0;
    set_ok();
    return norm_workspace(a, items);
}

p3d_status p3d_gated_norm_backward(const p3d_norm_desc* desc, const void* dh, const void* dr,
                                   const void* x, const void* y, void* dx, void* dy,
                                   float* dgate, float* dscale, float* dshift, float* dweight,
                                   float* dbias, float* dpost_weight, void* workspace,
                                   size_t workspace_bytes, void* stream) {
    const char* fn = "p3d_gated_norm_backward";
    NormArgs a;
    ItemTable items;
    P3D_TRY(check_norm(fn, desc, &a, &items));
    P3D_TRY(check_tensor(fn, "dh", dh, a.n > 0));
    P3D_TRY(check_tensor(fn, "dr", dr, false));
    P3D_TRY(check_tensor(fn, "x", x, a.n > 0));
    P3D_TRY(check_tensor(fn, "y", y, false));
    P3D_TRY(check_tensor(fn, "dx", dx, a.n > 0));
    P3D_TRY(check_tensor(fn, "dy", dy, false));
    P3D_TRY(check_tensor(fn, "dgate", dgate, false, 4));
    P3D_TRY(check_tensor(fn, "dscale", dscale, false, 4));
    P3D_TRY(check_tensor(fn, "dshift", dshift, false, 4));
    P3D_TRY(check_tensor(fn, "dweight", dweight, false, 4));
    P3D_TRY(check_tensor(fn, "dbias", dbias, false, 4));
    P3D_TRY(check_tensor(fn, "dpost_weight", dpost_weight, false, 4));
    if (a.n > 0 && !y && (dy || dgate || dpost_weight))
        return set_error(P3D_ERR_INVALID_ARG, "%s: dy, dgate and dpost_weight need y", fn);
    if (dx && dx == dy)
        return set_error(P3D_ERR_INVALID_ARG, "%s: dx and dy must be different tensors", fn);
    P3D_TRY(check_workspace(fn, "p3d_gated_norm_workspace_size", workspace, workspace_bytes,
                            norm_workspace(a, items)));
    a.x = x;
    a.y = y;
    a.dh = dh;
    a.dr = dr;
    a.dx = dx;
    a.dy = dy;
    a.dgate = dgate;
    a.dscale = dscale;
    a.dshift = dshift;
    a.dweight = dweight;
    a.dbias = dbias;
    a.dpost_weight = dpost_weight;
    a.partial = static_cast<float*>(workspace);
    const hipError_t e =
        launch_gated_norm_backward(a, desc->dtype, items, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? set_ok() : hip_fail(fn, e);
}

p3d_status p3d_rotary(const p3d_rotary_desc* desc, const void* x, int64_t x_stride, void* out,
                      int64_t out_stride, void* stream) {
    const char* fn = "p3d_rotary";
    RotaryArgs a;
    P3D_TRY(check_rotary(fn, desc, &a));
    const int epv = desc->dtype == P3D_BF16 ? 8 : 4;
    const int64_t width = (int64_t)a.heads * a.head_dim;
    P3D_TRY(check_tensor(fn, "x", x, a.n > 0));
    P3D_TRY(check_tensor(fn, "out", out, a.n > 0));
    P3D_TRY(check_stride(fn, "x_stride", x_stride, width, epv));
    P3D_TRY(check_stride(fn, "out_stride", out_stride, width, epv));
    if (x == out && x_stride != out_stride && a.n > 1)
        return set_error(P3D_ERR_SHAPE, "%s: in place, out_stride must be x_stride = %lld, got "
                         "%lld", fn, (long long)x_stride, (long long)out_stride);
    if (a.n == 0) return set_ok();
    a.x = x;
    a.x_stride = x_stride;
    a.out = out;
    a.out_stride = out_stride;
    const hipError_t e = launch_rotary(a, desc->dtype, false, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? set_ok() : hip_fail(fn, e);
}

size_t p3d_rotary_workspace_size(const p3d_rotary_desc* desc) {
    RotaryArgs a;
    if (check_rotary("p3d_rotary_workspace_size", desc, &a) != P3D_OK) return 0;
    set_ok();
    return (rotary_partial_bytes(a.n, a.heads, a.head_dim, desc->dtype) + 511) / 256 * 256;
}

p3d_status p3d_rotary_backward(const p3d_rotary_desc* desc, const void* dout,
                               int64_t dout_stride, const void* x, int64_t x_stride, void* dx,
                               int64_t dx_stride, float* dgamma, void* workspace,
                               size_t workspace_bytes, void* stream) {
    const char* fn = "p3d_rotary_backward";
    RotaryArgs a;
    P3D_TRY(check_rotary(fn, desc, &a));
    const int epv = desc->dtype == P3D_BF16 ? 8 : 4;
    const int64_t width = (int64_t)a.heads * a.head_dim;
    P3D_TRY(check_tensor(fn, "dout", dout, a.n > 0));
    P3D_TRY(check_tensor(fn, "dx", dx, a.n > 0));
    P3D_TRY(check_stride(fn, "dout_stride", dout_stride, width, epv));
    P3D_TRY(check_stride(fn, "dx_stride", dx_stride, width, epv));
    if (dx == dout && dx_stride != dout_stride && a.n > 1)
        return set_error(P3D_ERR_SHAPE, "%s: in place, dx_stride must be dout_stride = %lld, got "
                         "%lld", fn, (long long)dout_stride, (long long)dx_stride);
    if (a.gamma) {
        P3D_TRY(check_tensor(fn, "x", x, a.n > 0));
        P3D_TRY(check_stride(fn, "x_stride", x_stride, width, epv));
        if (dx == x && dx_stride != x_stride && a.n > 1)
            return set_error(P3D_ERR_SHAPE, "%s: in place, dx_stride must be x_stride = %lld, got "
                             "%lld", fn, (long long)x_stride, (long long)dx_stride);
    } else if (dgamma) {
        return set_error(P3D_ERR_INVALID_ARG, "%s: dgamma must be NULL without gamma", fn);
    }
    P3D_TRY(check_tensor(fn, "dgamma", dgamma, false, 4));
    if (dgamma)
        P3D_TRY(check_workspace(
            fn, "p3d_rotary_workspace_size", workspace, workspace_bytes,
            (rotary_partial_bytes(a.n, a.heads, a.head_dim, desc->dtype) + 511) / 256 * 256));
    a.dout = dout;
    a.dout_stride = dout_stride;
    a.x = x;
    a.x_stride = x_stride;
    a.out = dx;
    a.out_stride = dx_stride;
    a.dgamma = dgamma;
    a.partial = static_cast<float*>(workspace);
    const hipError_t e = launch_rotary(a, desc->dtype, true, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? set_ok() : hip_fail(fn, e);
}

p3d_status p3d_rotary_frequencies(double base, int32_t pairs, p3d_rotary_scaling scaling,
                                  double factor, double trained, float* freqs) {
    const char* fn = "p3d_rotary_frequencies";
    if (!(isfinite(base) && base > 1.0))
        return set_error(P3D_ERR_INVALID_ARG, "%s: base must be finite and > 1, got %g", fn, base);
    if (pairs < 1 || pairs > 128)
        return set_error(P3D_ERR_INVALID_ARG, "%s: pairs must be in [1, 128], got %d", fn, pairs);
    if (scaling < P3D_ROTARY_PLAIN || scaling > P3D_ROTARY_BY_PARTS)
        return set_error(P3D_ERR_INVALID_ARG,
                         "%s: scaling must be PLAIN, LINEAR, BASE or BY_PARTS, got %d", fn,
                         (int)scaling);
    if (scaling != P3D_ROTARY_PLAIN && !(isfinite(factor) && factor >= 1.0))
        return set_error(P3D_ERR_INVALID_ARG, "%s: factor must be finite and >= 1, got %g", fn,
                         factor);
    if (scaling == P3D_ROTARY_BASE && pairs < 2)
        return set_error(P3D_ERR_INVALID_ARG, "%s: BASE needs at least 2 pairs, got %d", fn,
                         pairs);
    if (scaling == P3D_ROTARY_BY_PARTS && !(isfinite(trained) && trained >= 1.0))
        return set_error(P3D_ERR_INVALID_ARG, "%s: trained must be finite and >= 1, got %g", fn,
                         trained);
    if (!freqs) return set_error(P3D_ERR_INVALID_ARG, "%s: freqs is NULL (host array)", fn);
    if (scaling == P3D_ROTARY_BASE) base *= pow(factor, (double)pairs / (pairs - 1));
    for (int32_t i = 0; i < pairs; ++i) {
        double f = pow(base, -(double)i / pairs);
        if (scaling == P3D_ROTARY_LINEAR) f /= factor;
        if (scaling == P3D_ROTARY_BY_PARTS) {
            const double turns = trained * f / 6.283185307179586477;
            const double keep = fmin(fmax((turns - 1.0) / 31.0, 0.0), 1.0);
            f = f * keep + f / factor * (1.0 - keep);
        }
        freqs[i] = (float)f;
    }
    return set_ok();
}

size_t p3d_attention_workspace_size(const p3d_attn_desc* desc) {
    AttnArgs a;
    if (check_attention("p3d_attention_workspace_size", desc, &a) != P3D_OK) return 0;
    set_ok();
    return (attention_plan(a).forward_bytes + 255) / 256 * 256;
}

size_t p3d_attention_backward_workspace_size(const p3d_attn_desc* desc) {
    AttnArgs a;
    if (check_attention_backward("p3d_attention_backward_workspace_size", desc, &a) != P3D_OK)
        return 0;
    set_ok();
    return (attention_plan(a).backward_bytes + 255) / 256 * 256;
}

p3d_status p3d_attention(const p3d_attn_desc* desc, const void* q, int64_t q_stride,
                         const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                         void* out, int64_t out_stride, float* lse, void* workspace,
                         size_t workspace_bytes, void* stream) {
    const char* fn = "p3d_attention";
    AttnArgs a;
    P3D_TRY(check_attention(fn, desc, &a));
    const bool queries = a.q_items.start[a.batch] > 0, keys = a.k_items.start[a.batch] > 0;
    const int64_t wq = (int64_t)a.heads * a.head_dim, wk = (int64_t)a.kv_heads * a.head_dim;
    P3D_TRY(check_tensor(fn, "q", q, queries));
    P3D_TRY(check_tensor(fn, "k", k, keys));
    P3D_TRY(check_tensor(fn, "v", v, keys));
    P3D_TRY(check_tensor(fn, "out", out, queries));
    P3D_TRY(check_tensor(fn, "lse", lse, false, 4));
    P3D_TRY(check_stride(fn, "q_stride", q_stride, wq, 8));
    P3D_TRY(check_stride(fn, "k_stride", k_stride, wk, 8));
    P3D_TRY(check_stride(fn, "v_stride", v_stride, wk, 8));
    P3D_TRY(check_stride(fn, "out_stride", out_stride, wq, 8));
    if (out && out == q && out_stride != q_stride)
        return set_error(P3D_ERR_SHAPE, "%s: in place, out_stride must be q_stride = %lld, got "
                         "%lld", fn, (long long)q_stride, (long long)out_stride);
    const AttnPlan plan = attention_plan(a);
    P3D_TRY(check_workspace(fn, "p3d_attention_workspace_size", workspace, workspace_bytes,
                            (plan.forward_bytes + 255) / 256 * 256));
    const int64_t nq = a.q_items.start[a.batch], nk = a.k_items.start[a.batch];
    const Rows written{"out", out, nq, 2 * wq, 2 * out_stride};
    P3D_TRY(check_apart(fn, written, {"k", k, nk, 2 * wk, 2 * k_stride}));
    P3D_TRY(check_apart(fn, written, {"v", v, nk, 2 * wk, 2 * v_stride}));
    if (out != q) P3D_TRY(check_apart(fn, written, {"q", q, nq, 2 * wq, 2 * q_stride}));
    a.q = q;
    a.k = k;
    a.v = v;
    a.out = out;
    a.lse = lse;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.out_stride = out_stride;
    const hipError_t e = launch_attention(a, plan, workspace, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? set_ok() : hip_fail(fn, e);
}

p3d_status p3d_attention_backward(const p3d_attn_desc* desc, const void* dout,
                                  int64_t dout_stride, const void* q, int64_t q_stride,
                                  const void* k, int64_t k_stride, const void* v,
                                  int64_t v_stride, const void* out, int64_t out_stride,
                                  const float* lse, void* dq, int64_t dq_stride, void* dk,
                                  int64_t dk_stride, void* dv, int64_t dv_stride,
                                  void* workspace, size_t workspace_bytes, void* stream) {
    const char* fn = "p3d_attention_backward";
    AttnArgs a;
    P3D_TRY(check_attention_backward(fn, desc, &a));
    const bool queries = a.q_items.start[a.batch] > 0, keys = a.k_items.start[a.batch] > 0;
    const int64_t wq = (int64_t)a.heads * a.head_dim, wk = (int64_t)a.kv_heads * a.head_dim;
    P3D_TRY(check_tensor(fn, "dout", dout, queries));
    P3D_TRY(check_tensor(fn, "q", q, queries));
    P3D_TRY(check_tensor(fn, "k", k, keys));
    P3D_TRY(check_tensor(fn, "v", v, keys));
    P3D_TRY(check_tensor(fn, "out", out, queries));
    P3D_TRY(check_tensor(fn, "lse", lse, queries, 4));
    P3D_TRY(check_tensor(fn, "dq", dq, queries));
    P3D_TRY(check_tensor(fn, "dk", dk, keys));
    P3D_TRY(check_tensor(fn, "dv", dv, keys));
    P3D_TRY(check_stride(fn, "dout_stride", dout_stride, wq, 8));
    P3D_TRY(check_stride(fn, "q_stride", q_stride, wq, 8));
    P3D_TRY(check_stride(fn, "k_stride", k_stride, wk, 8));
    P3D_TRY(check_stride(fn, "v_stride", v_stride, wk, 8));
    P3D_TRY(check_stride(fn, "out_stride", out_stride, wq, 8));
    P3D_TRY(check_stride(fn, "dq_stride", dq_stride, wq, 8));
    P3D_TRY(check_stride(fn, "dk_stride", dk_stride, wk, 8));
    P3D_TRY(check_stride(fn, "dv_stride", dv_stride, wk, 8));
    const AttnPlan plan = attention_plan(a);
    P3D_TRY(check_workspace(fn, "p3d_attention_backward_workspace_size", workspace,
                            workspace_bytes, (plan.backward_bytes + 255) / 256 * 256));
    const int64_t nq = a.q_items.start[a.batch], nk = a.k_items.start[a.batch];
    const Rows tensors[] = {{"dq", dq, nq, 2 * wq, 2 * dq_stride},
                            {"dk", dk, nk, 2 * wk, 2 * dk_stride},
                            {"dv", dv, nk, 2 * wk, 2 * dv_stride},
                            {"dout", dout, nq, 2 * wq, 2 * dout_stride},
                            {"q", q, nq, 2 * wq, 2 * q_stride},
                            {"k", k, nk, 2 * wk, 2 * k_stride},
                            {"v", v, nk, 2 * wk, 2 * v_stride},
                            {"out", out, nq, 2 * wq, 2 * out_stride},
                            {"lse", lse, nq, 4 * (int64_t)a.heads, 4 * (int64_t)a.heads}};
    for (int i = 0; i < 3; ++i)
        for (int j = i + 1; j < 9; ++j) P3D_TRY(check_apart(fn, tensors[i], tensors[j]));
    a.dout = dout;
    a.q = q;
    a.k = k;
    a.v = v;
    a.out_in = out;
    a.lse_in = lse;
    a.dq = dq;
    a.dk = dk;
    a.dv = dv;
    a.dout_stride = dout_stride;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.out_stride = out_stride;
    a.dq_stride = dq_stride;
    a.dk_stride = dk_stride;
    a.dv_stride = dv_stride;
    const hipError_t e =
        launch_attention_backward(a, plan, workspace, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? set_ok() : hip_fail(fn, e);
}

}  // extern "C"
