// model_api.hip -- the extern "C" entry points of include/p3d_model.h:
// validation of every argument before anything is enqueued, workspace sizes,
// and dispatch to the kernels.
#include <math.h>
#include <stdio.h>

#include <algorithm>
#include <initializer_list>
#include <new>
#include <utility>
#include <vector>

#include "api_checks.h"
#include "model_internal.h"

using namespace p3d;
using namespace p3d::checks;

namespace {

p3d_status check_act(const char* fn, p3d_act act) {
    if (act != P3D_ACT_NONE && act != P3D_ACT_SILU && act != P3D_ACT_GELU)
        return set_error(P3D_ERR_INVALID_ARG, "%s: act must be NONE, SILU or GELU, got %d", fn,
                         (int)act);
    return P3D_OK;
}

p3d_status check_rows(const char* fn, int64_t n) {
    if (n < 0 || n >= kMaxRows)
        return set_error(P3D_ERR_INVALID_ARG, "%s: n must be in [0, %lld), got %lld", fn,
                         (long long)kMaxRows, (long long)n);
    return P3D_OK;
}

// Elements between rows of `width` that hold `name` by `unit` elements.
p3d_status check_pitch(const char* fn, const char* name, int64_t stride, int64_t width, int unit,
                       int64_t most) {
    if (stride < width)
        return set_error(P3D_ERR_SHAPE, "%s: %s must be at least a row's %lld elements, got %lld",
                         fn, name, (long long)width, (long long)stride);
    if (stride % unit || stride > most)
        return set_error(P3D_ERR_UNSUPPORTED, "%s: %s must be a multiple of %d up to %lld, got %lld",
                         fn, name, unit, (long long)most, (long long)stride);
    return P3D_OK;
}

constexpr int64_t kMaxStride = int64_t(1) << 30;

Rows line(const char* name, const void* base, int64_t bytes) {
    return {name, base, bytes > 0 ? 1 : 0, bytes, bytes};
}

// Whether two tensors share a byte, whatever their strides. A tensor without gaps
// counts as one row, which overlap() decides against any; rows with gaps that are
// differently far apart are gone through one by one.
bool meet(Rows a, Rows b) {
    for (Rows* t : {&a, &b}) {
        if (!t->base || t->rows == 0) return false;
        if (t->pitch == t->width) *t = line(t->name, t->base, t->rows * t->width);
    }
    if (a.rows == 1 || b.rows == 1 || a.pitch == b.pitch) return overlap(a, b);
    const auto end = [](const Rows& t) {
        return static_cast<const char*>(t.base) + (t.rows - 1) * t.pitch + t.width;
    };
    if (end(a) <= b.base || end(b) <= a.base) return false;
    if (a.rows > b.rows) std::swap(a, b);
    Rows row{a.name, a.base, 1, a.width, a.width};
    for (int64_t i = 0; i < a.rows; ++i) {
        row.base = static_cast<const char*>(a.base) + i * a.pitch;
        if (row_meets(row, b)) return true;
    }
    return false;
}

// Results share nothing with each other or with what the call reads.
p3d_status check_results(const char* fn, std::initializer_list<Rows> written,
                         std::initializer_list<Rows> read) {
    for (const Rows* w = written.begin(); w != written.end(); ++w) {
        const auto refuse = [&](const Rows& other) {
            return meet(*w, other) ? set_error(P3D_ERR_INVALID_ARG, "%s: %s must not overlap %s",
                                               fn, w->name, other.name)
                                   : P3D_OK;
        };
        for (const Rows* o = w + 1; o != written.end(); ++o) P3D_TRY(refuse(*o));
        for (const Rows& o : read) P3D_TRY(refuse(o));
    }
    return P3D_OK;
}

// ------------------------------------------------------------- group norm ---
p3d_status check_group(const char* fn, const p3d_group_desc* d, GroupArgs* a) {
    if (!d) return set_error(P3D_ERR_INVALID_ARG, "%s: desc is NULL", fn);
    P3D_TRY(check_dtype(fn, d->dtype));
    P3D_TRY(check_act(fn, d->act));
    P3D_TRY(check_rows(fn, d->n));
    *a = GroupArgs{};
    P3D_TRY(check_items(fn, "offsets", d->offsets, d->batch, &a->items));
    if (d->offsets[d->batch] != d->n)
        return set_error(P3D_ERR_SHAPE, "%s: offsets[%d] must be n = %lld, got %lld", fn, d->batch,
                         (long long)d->n, (long long)d->offsets[d->batch]);
    const int unit = d->dtype == P3D_BF16 ? 8 : 4;
    if (d->channels < 1)
        return set_error(P3D_ERR_INVALID_ARG, "%s: channels must be >= 1, got %d", fn, d->channels);
    if (d->channels % unit || d->channels > 4096)
        return set_error(P3D_ERR_UNSUPPORTED,
                         "%s: channels must be a multiple of %d up to 4096, got %d", fn, unit,
                         d->channels);
    if (d->groups < 1 || d->channels % d->groups)
        return set_error(P3D_ERR_SHAPE, "%s: groups must divide channels = %d, got %d", fn,
                         d->channels, d->groups);
    if (!(isfinite(d->eps) && d->eps > 0.f))
        return set_error(P3D_ERR_INVALID_ARG, "%s: eps must be finite and > 0, got %g", fn,
                         (double)d->eps);
    P3D_TRY(check_tensor(fn, "weight", d->weight, false));
    P3D_TRY(check_tensor(fn, "bias", d->bias, false));
    a->batch = d->batch;
    a->channels = d->channels;
    a->groups = d->groups;
    a->act = d->act;
    a->eps = d->eps;
    a->weight = d->weight;
    a->bias = d->bias;
    return P3D_OK;
}

// `out` may be `in` where their rows lie alike, and shares nothing with it otherwise.
p3d_status check_in_place(const char* fn, const Rows& out, const Rows& in) {
    if (out.base && out.base == in.base && out.pitch == in.pitch) return P3D_OK;
    if (out.base && out.base == in.base && out.rows > 0)
        return set_error(P3D_ERR_SHAPE, "%s: in place, the strides of %s and %s must be equal", fn,
                         out.name, in.name);
    return check_results(fn, {out}, {in});
}

// ----------------------------------------------------------------- linear ---
p3d_status check_width(const char* fn, const char* name, int32_t width) {
    if (width < 16 || width > 65536 || width % 16)
        return set_error(width < 1 ? P3D_ERR_INVALID_ARG : P3D_ERR_UNSUPPORTED,
                         "%s: %s must be a multiple of 16 in [16, 65536], got %d", fn, name, width);
    return P3D_OK;
}

// ------------------------------------------------------------------ adamw ---
struct Span {
    uintptr_t from, to;
    int32_t tensor;
    const char* name;
    bool written;
    // "tensors[3].m", or the name alone of what belongs to none
    void word(char (&to)[64]) const {
        if (tensor < 0) snprintf(to, sizeof to, "%s", name);
        else snprintf(to, sizeof to, "tensors[%d].%s", tensor, name);
    }
};

p3d_status check_table(const char* fn, const p3d_adamw_desc* d, bool step) {
    if (!d) return set_error(P3D_ERR_INVALID_ARG, "%s: desc is NULL", fn);
    if (d->count < 0 || d->count > 65536)
        return set_error(P3D_ERR_INVALID_ARG, "%s: count must be in [0, 65536], got %d", fn,
                         d->count);
    if (d->count > 0 && !d->tensors)
        return set_error(P3D_ERR_INVALID_ARG, "%s: tensors is NULL (host array [count])", fn);
    if (d->grad_dtype != P3D_F32 && d->grad_dtype != P3D_BF16)
        return set_error(P3D_ERR_DTYPE, "%s: grad_dtype must be F32 or BF16, got %d", fn,
                         (int)d->grad_dtype);
    if (step) {
        if (d->param_dtype != P3D_F32 && d->param_dtype != P3D_BF16)
            return set_error(P3D_ERR_DTYPE, "%s: param_dtype must be F32 or BF16, got %d", fn,
                             (int)d->param_dtype);
        if (d->state_bits != 8 && d->state_bits != 32)
            return set_error(P3D_ERR_INVALID_ARG, "%s: state_bits must be 32 or 8, got %d", fn,
                             d->state_bits);
    }
    const char* bad = nullptr;
    const int32_t masters = (int32_t)std::count_if(
        d->tensors, d->tensors + d->count,
        [](const p3d_adamw_tensor& t) { return t.master != nullptr; });
    for (int32_t j = 0; j < d->count; ++j) {
        const p3d_adamw_tensor& t = d->tensors[j];
        if (t.size < 0 || t.size >= int64_t(1) << 34)
            return set_error(P3D_ERR_INVALID_ARG, "%s: tensors[%d].size must be in [0, 2^34), got "
                             "%lld", fn, j, (long long)t.size);
        const bool some = t.size > 0;
        if (some && !t.grad) bad = "grad";
        if (step && some) {
            if (!t.param) bad = "param";
            if (!t.m) bad = "m";
            if (!t.v) bad = "v";
            if (d->state_bits == 8 && !t.m_scale) bad = "m_scale";
            if (d->state_bits == 8 && !t.v_scale) bad = "v_scale";
            if (masters && !t.master) bad = "master";
        }
        if (bad)
            return set_error(P3D_ERR_INVALID_ARG, "%s: tensors[%d].%s is NULL", fn, j, bad);
        if (!aligned(t.grad, 16)) bad = "grad";
        if (step) {
            if (!aligned(t.param, 16)) bad = "param";
            if (!aligned(t.master, 16)) bad = "master";
            if (!aligned(t.m, 16)) bad = "m";
            if (!aligned(t.v, 16)) bad = "v";
            if (!aligned(t.m_scale, 4)) bad = "m_scale";
            if (!aligned(t.v_scale, 4)) bad = "v_scale";
        }
        if (bad)
            return set_error(P3D_ERR_UNSUPPORTED, "%s: tensors[%d].%s is not aligned (16 bytes; "
                             "scales: 4)", fn, j, bad);
        if (!step) continue;
        if (d->state_bits == 32 && (t.m_scale || t.v_scale))
            return set_error(P3D_ERR_INVALID_ARG, "%s: tensors[%d] has scales, which 32-bit states "
                             "do not", fn, j);
        if (!isfinite(t.weight_decay))
            return set_error(P3D_ERR_INVALID_ARG, "%s: tensors[%d].weight_decay must be finite, got "
                             "%g", fn, j, (double)t.weight_decay);
    }
    if (step && masters && d->param_dtype == P3D_F32)
        return set_error(P3D_ERR_INVALID_ARG, "%s: masters are for BF16 params", fn);
    return P3D_OK;
}

// Whether nothing that a step writes is written twice or read as anything else.
p3d_status check_spans(const char* fn, const p3d_adamw_desc* d) {
    std::vector<Span> spans;
    spans.reserve((size_t)d->count * 7 + 3);
    for (const auto& [name, base] : {std::pair<const char*, const void*>{"grad_scale", d->grad_scale},
                                     {"device_lr", d->device_lr}, {"device_step", d->device_step}}) {
        const uintptr_t at = reinterpret_cast<uintptr_t>(base);
        if (base) spans.push_back({at, at + 4, -1, name, false});
    }
    const int p = d->param_dtype == P3D_BF16 ? 2 : 4, g = d->grad_dtype == P3D_BF16 ? 2 : 4;
    const int state = d->state_bits / 8;
    for (int32_t j = 0; j < d->count; ++j) {
        const p3d_adamw_tensor& t = d->tensors[j];
        if (t.size == 0) continue;
        const auto add = [&](const char* name, const void* base, int64_t bytes, bool written) {
            const uintptr_t at = reinterpret_cast<uintptr_t>(base);
            if (base) spans.push_back({at, at + (uintptr_t)bytes, j, name, written});
        };
        const int64_t scales = (t.size + 255) / 256 * 4;
        add("param", t.param, t.size * p, true);
        add("master", t.master, t.size * 4, true);
        add("grad", t.grad, t.size * g, false);
        add("m", t.m, t.size * state, true);
        add("v", t.v, t.size * state, true);
        add("m_scale", t.m_scale, scales, true);
        add("v_scale", t.v_scale, scales, true);
    }
    std::sort(spans.begin(), spans.end(),
              [](const Span& a, const Span& b) { return a.from < b.from; });
    // the span that reaches furthest so far, of all and of the written ones
    const Span *all = nullptr, *written = nullptr;
    for (const Span& s : spans) {
        const Span* other = s.written ? all : written;
        if (other && other->to > s.from) {
            char a[64], b[64];
            s.word(a);
            other->word(b);
            return set_error(P3D_ERR_INVALID_ARG, "%s: %s must not overlap %s", fn, a, b);
        }
        if (!all || s.to > all->to) all = &s;
        if (s.written && (!written || s.to > written->to)) written = &s;
    }
    return P3D_OK;
}

size_t grad_norm_bytes(const p3d_adamw_desc& d) {
    return ((size_t)grad_norm_parts(d) * sizeof(double) + 511) / 256 * 256;
}

}  // namespace

extern "C" {

size_t p3d_group_norm_workspace_size(const p3d_group_desc* desc) {
    GroupArgs a;
    if (check_group("p3d_group_norm_workspace_size", desc, &a) != P3D_OK) return 0;
    set_ok();
    return group_norm_plan(a, desc->dtype).bytes;
}

p3d_status p3d_group_norm(const p3d_group_desc* desc, const void* x, int64_t x_stride, void* out,
                          int64_t out_stride, float* mean, float* rstd, void* workspace,
                          size_t workspace_bytes, void* stream) {
    const char* fn = "p3d_group_norm";
    GroupArgs a;
    P3D_TRY(check_group(fn, desc, &a));
    const int unit = desc->dtype == P3D_BF16 ? 8 : 4, e = 16 / unit;
    const bool some = desc->n > 0;
    P3D_TRY(check_tensor(fn, "x", x, some));
    P3D_TRY(check_tensor(fn, "out", out, some));
    P3D_TRY(check_pitch(fn, "x_stride", x_stride, a.channels, unit, kMaxStride));
    P3D_TRY(check_pitch(fn, "out_stride", out_stride, a.channels, unit, kMaxStride));
    P3D_TRY(check_tensor(fn, "mean", mean, false, 4));
    P3D_TRY(check_tensor(fn, "rstd", rstd, false, 4));
    const int64_t width = (int64_t)a.channels * e, stats = (int64_t)a.batch * a.groups * 4;
    const Rows to{"out", out, desc->n, width, out_stride * e},
        from{"x", x, desc->n, width, x_stride * e}, m = line("mean", mean, stats),
        r = line("rstd", rstd, stats), w = line("weight", a.weight, width),
        b = line("bias", a.bias, width);
    P3D_TRY(check_in_place(fn, to, from));
    P3D_TRY(check_results(fn, {to, m, r}, {w, b}));
    P3D_TRY(check_results(fn, {m}, {from}));
    P3D_TRY(check_results(fn, {r}, {from}));
    const GroupPlan plan = group_norm_plan(a, desc->dtype);
    P3D_TRY(check_workspace(fn, "p3d_group_norm_workspace_size", workspace, workspace_bytes,
                            plan.bytes));
    a.x = x;
    a.x_stride = x_stride;
    a.out = out;
    a.out_stride = out_stride;
    a.mean = mean;
    a.rstd = rstd;
    const hipError_t er =
        launch_group_norm(a, plan, desc->dtype, workspace, static_cast<hipStream_t>(stream));
    return er == hipSuccess ? set_ok() : hip_fail(fn, er);
}

p3d_status p3d_group_norm_backward(const p3d_group_desc* desc, const void* dout,
                                   int64_t dout_stride, const void* x, int64_t x_stride,
                                   const float* mean, const float* rstd, void* dx,
                                   int64_t dx_stride, float* dweight, float* dbias,
                                   void* workspace, size_t workspace_bytes, void* stream) {
    const char* fn = "p3d_group_norm_backward";
    GroupArgs a;
    P3D_TRY(check_group(fn, desc, &a));
    const int unit = desc->dtype == P3D_BF16 ? 8 : 4, e = 16 / unit;
    const bool some = desc->n > 0;
    P3D_TRY(check_tensor(fn, "dout", dout, some));
    P3D_TRY(check_tensor(fn, "x", x, some));
    P3D_TRY(check_tensor(fn, "mean", mean, true, 4));
    P3D_TRY(check_tensor(fn, "rstd", rstd, true, 4));
    P3D_TRY(check_tensor(fn, "dx", dx, some));
    P3D_TRY(check_pitch(fn, "dout_stride", dout_stride, a.channels, unit, kMaxStride));
    P3D_TRY(check_pitch(fn, "x_stride", x_stride, a.channels, unit, kMaxStride));
    P3D_TRY(check_pitch(fn, "dx_stride", dx_stride, a.channels, unit, kMaxStride));
    P3D_TRY(check_tensor(fn, "dweight", dweight, false, 4));
    P3D_TRY(check_tensor(fn, "dbias", dbias, false, 4));
    const int64_t width = (int64_t)a.channels * e, stats = (int64_t)a.batch * a.groups * 4,
                  sums = (int64_t)a.channels * 4;
    const Rows to{"dx", dx, desc->n, width, dx_stride * e},
        grad{"dout", dout, desc->n, width, dout_stride * e},
        from{"x", x, desc->n, width, x_stride * e}, m = line("mean", mean, stats),
        r = line("rstd", rstd, stats), w = line("weight", a.weight, width),
        b = line("bias", a.bias, width), dw = line("dweight", dweight, sums),
        db = line("dbias", dbias, sums);
    P3D_TRY(check_in_place(fn, to, grad));
    P3D_TRY(check_in_place(fn, to, from));
    P3D_TRY(check_results(fn, {to, dw, db}, {m, r, w, b}));
    P3D_TRY(check_results(fn, {dw}, {grad, from}));
    P3D_TRY(check_results(fn, {db}, {grad, from}));
    const GroupPlan plan = group_norm_plan(a, desc->dtype);
    P3D_TRY(check_workspace(fn, "p3d_group_norm_workspace_size", workspace, workspace_bytes,
                            plan.bytes));
    a.x = x;
    a.x_stride = x_stride;
    a.dout = dout;
    a.dout_stride = dout_stride;
    a.dx = dx;
    a.out_stride = dx_stride;
    a.mean_in = mean;
    a.rstd_in = rstd;
    a.dweight = dweight;
    a.dbias = dbias;
    const hipError_t er = launch_group_norm_backward(a, plan, desc->dtype, workspace,
                                                     static_cast<hipStream_t>(stream));
    return er == hipSuccess ? set_ok() : hip_fail(fn, er);
}

p3d_status p3d_quantize_rows(const void* x, p3d_dtype dtype, int64_t n, int32_t width,
                             int64_t x_stride, int8_t* q, int64_t q_stride, float* scale,
                             void* stream) {
    const char* fn = "p3d_quantize_rows";
    P3D_TRY(check_dtype(fn, dtype));
    P3D_TRY(check_rows(fn, n));
    P3D_TRY(check_width(fn, "width", width));
    const int unit = dtype == P3D_BF16 ? 8 : 4, e = 16 / unit;
    P3D_TRY(check_tensor(fn, "x", x, n > 0));
    P3D_TRY(check_tensor(fn, "q", q, n > 0));
    P3D_TRY(check_tensor(fn, "scale", scale, n > 0, 4));
    P3D_TRY(check_pitch(fn, "x_stride", x_stride, width, unit, kMaxStride));
    P3D_TRY(check_pitch(fn, "q_stride", q_stride, width, 16, kMaxStride));
    P3D_TRY(check_results(fn, {{"q", q, n, width, q_stride}, line("scale", scale, n * 4)},
                          {{"x", x, n, (int64_t)width * e, x_stride * e}}));
    if (n == 0) return set_ok();
    QuantizeArgs a{x, n, x_stride, q_stride, width, q, scale};
    const hipError_t er = launch_quantize_rows(a, dtype, static_cast<hipStream_t>(stream));
    return er == hipSuccess ? set_ok() : hip_fail(fn, er);
}

p3d_status p3d_linear_i8(const p3d_linear_i8_desc* desc, const int8_t* q, int64_t q_stride,
                         const float* scale, const void* residual, int64_t residual_stride,
                         void* out, int64_t out_stride, void* stream) {
    const char* fn = "p3d_linear_i8";
    if (!desc) return set_error(P3D_ERR_INVALID_ARG, "%s: desc is NULL", fn);
    P3D_TRY(check_dtype(fn, desc->dtype));
    P3D_TRY(check_act(fn, desc->act));
    P3D_TRY(check_rows(fn, desc->n));
    P3D_TRY(check_width(fn, "in_dim", desc->in_dim));
    const int64_t n = desc->n, k = desc->in_dim, d = desc->out_dim;
    if (d < 1 || d >= kMaxRows)
        return set_error(P3D_ERR_INVALID_ARG, "%s: out_dim must be in [1, 2^30), got %lld", fn,
                         (long long)d);
    if (d % 8)
        return set_error(P3D_ERR_UNSUPPORTED, "%s: out_dim must be a multiple of 8, got %lld", fn,
                         (long long)d);
    // (the kernels number their tiles, of 128 x 64 or more, in 32 bits)
    if (((n + 63) / 64) * ((d + 63) / 64) >= int64_t(1) << 24)
        return set_error(P3D_ERR_UNSUPPORTED,
                         "%s: n * out_dim, each rounded up to a multiple of 64, must be below 2^36, "
                         "got %lld * %lld", fn, (long long)n, (long long)d);
    const int unit = desc->dtype == P3D_BF16 ? 8 : 4, e = 16 / unit;
    const bool some = n > 0;
    P3D_TRY(check_tensor(fn, "weight", desc->weight, some));
    P3D_TRY(check_tensor(fn, "weight_scale", desc->weight_scale, some, 4));
    P3D_TRY(check_tensor(fn, "bias", desc->bias, false));
    P3D_TRY(check_tensor(fn, "q", q, some));
    P3D_TRY(check_tensor(fn, "scale", scale, some, 4));
    P3D_TRY(check_tensor(fn, "residual", residual, false));
    P3D_TRY(check_tensor(fn, "out", out, some));
    P3D_TRY(check_pitch(fn, "q_stride", q_stride, k, 16, int64_t(1) << 22));
    P3D_TRY(check_pitch(fn, "out_stride", out_stride, d, unit, kMaxStride));
    if (residual)
        P3D_TRY(check_pitch(fn, "residual_stride", residual_stride, d, unit, kMaxStride));
    const Rows to{"out", out, n, d * e, out_stride * e};
    P3D_TRY(check_results(fn, {to},
                          {{"q", q, n, k, q_stride}, line("weight", desc->weight, d * k),
                           line("scale", scale, n * 4),
                           line("weight_scale", desc->weight_scale, d * 4),
                           line("bias", desc->bias, d * e)}));
    if (residual)
        P3D_TRY(check_in_place(fn, to, {"residual", residual, n, d * e, residual_stride * e}));
    if (n == 0) return set_ok();
    LinearArgs a{};
    a.q = q;
    a.weight = desc->weight;
    a.scale = scale;
    a.weight_scale = desc->weight_scale;
    a.bias = desc->bias;
    a.residual = residual;
    a.out = out;
    a.n = n;
    a.q_stride = q_stride;
    a.residual_stride = residual_stride;
    a.out_stride = out_stride;
    a.in_dim = desc->in_dim;
    a.out_dim = desc->out_dim;
    a.act = desc->act;
    const hipError_t er = launch_linear_i8(a, desc->dtype, static_cast<hipStream_t>(stream));
    return er == hipSuccess ? set_ok() : hip_fail(fn, er);
}

p3d_status p3d_adamw(const p3d_adamw_desc* desc, void* stream) {
    const char* fn = "p3d_adamw";
    P3D_TRY(check_table(fn, desc, true));
    if (!(isfinite(desc->lr) && desc->lr >= 0.))
        return set_error(P3D_ERR_INVALID_ARG, "%s: lr must be finite and >= 0, got %g", fn,
                         desc->lr);
    if (!(desc->beta1 >= 0. && desc->beta1 < 1.) || !(desc->beta2 >= 0. && desc->beta2 < 1.))
        return set_error(P3D_ERR_INVALID_ARG, "%s: beta1 and beta2 must be in [0, 1), got %g and %g",
                         fn, desc->beta1, desc->beta2);
    // (as the kernels hold it: an eps that binary32 has no number for is 0)
    if (!(isfinite((float)desc->eps) && (float)desc->eps > 0.f))
        return set_error(P3D_ERR_INVALID_ARG, "%s: eps must be finite and > 0, got %g", fn,
                         desc->eps);
    if (desc->step < 1)
        return set_error(P3D_ERR_INVALID_ARG, "%s: step must be >= 1, got %lld", fn,
                         (long long)desc->step);
    P3D_TRY(check_tensor(fn, "grad_scale", desc->grad_scale, false, 4));
    P3D_TRY(check_tensor(fn, "device_lr", desc->device_lr, false, 4));
    P3D_TRY(check_tensor(fn, "device_step", desc->device_step, false, 4));
    try {
        P3D_TRY(check_spans(fn, desc));
    } catch (const std::bad_alloc&) {
        return set_error(P3D_ERR_UNSUPPORTED, "%s: no host memory to check %d tensors", fn,
                         desc->count);
    }
    const hipError_t er = launch_adamw(*desc, static_cast<hipStream_t>(stream));
    return er == hipSuccess ? set_ok() : hip_fail(fn, er);
}

size_t p3d_grad_norm_workspace_size(const p3d_adamw_desc* desc) {
    if (check_table("p3d_grad_norm_workspace_size", desc, false) != P3D_OK) return 0;
    set_ok();
    return grad_norm_bytes(*desc);
}

p3d_status p3d_grad_norm(const p3d_adamw_desc* desc, float max_norm, float* out, void* workspace,
                         size_t workspace_bytes, void* stream) {
    const char* fn = "p3d_grad_norm";
    P3D_TRY(check_table(fn, desc, false));
    if (!(max_norm > 0.f))
        return set_error(P3D_ERR_INVALID_ARG, "%s: max_norm must be > 0, got %g", fn,
                         (double)max_norm);
    P3D_TRY(check_tensor(fn, "out", out, true, 4));
    const int64_t e = desc->grad_dtype == P3D_BF16 ? 2 : 4;
    for (int32_t j = 0; j < desc->count; ++j)
        if (meet(line("out", out, 8), line("grad", desc->tensors[j].grad, desc->tensors[j].size * e)))
            return set_error(P3D_ERR_INVALID_ARG, "%s: out must not overlap tensors[%d].grad", fn, j);
    P3D_TRY(check_workspace(fn, "p3d_grad_norm_workspace_size", workspace, workspace_bytes,
                            grad_norm_bytes(*desc)));
    const hipError_t er = launch_grad_norm(*desc, max_norm, out, static_cast<double*>(workspace),
                                           static_cast<hipStream_t>(stream));
    return er == hipSuccess ? set_ok() : hip_fail(fn, er);
}

}  // extern "C"
