// api_checks.h -- argument checks that the entry points of the block's and the
// model's operators share. Host code; each returns P3D_OK or the status that
// the entry point answers with, the message set.
#pragma once

#include "block_internal.h"

namespace p3d {
namespace checks {

constexpr int64_t kMaxRows = int64_t(1) << 30;     // rows and offsets are int32 in the kernels

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline p3d_status hip_fail(const char* fn, hipError_t e) {
    return set_error(P3D_ERR_HIP, "%s: HIP launch failed: %s", fn, hipGetErrorString(e));
}

inline p3d_status check_dtype(const char* fn, p3d_dtype dt) {
    if (dt != P3D_F32 && dt != P3D_BF16)
        return set_error(P3D_ERR_DTYPE, "%s: dtype must be F32 or BF16, got %d", fn, (int)dt);
    return P3D_OK;
}

// A required (or, `needed` false, optional) device tensor.
inline p3d_status check_tensor(const char* fn, const char* name, const void* p, bool needed,
                        size_t align = 16) {
    if (needed && !p) return set_error(P3D_ERR_INVALID_ARG, "%s: %s is NULL", fn, name);
    if (!aligned(p, align))
        return set_error(P3D_ERR_UNSUPPORTED, "%s: %s must be %zu-byte aligned, got %p", fn, name,
                         align, p);
    return P3D_OK;
}

inline p3d_status check_items(const char* fn, const char* name, const int64_t* offsets, int32_t batch,
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

inline p3d_status check_workspace(const char* fn, const char* size_fn, const void* ws, size_t got,
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

// The bytes of a [rows, width] tensor, rows `pitch` bytes apart.
struct Rows {
    const char* name;
    const void* base;
    int64_t rows, width, pitch;
};

inline int64_t floor_div(int64_t a, int64_t b) { return a >= 0 ? a / b : -((b - 1 - a) / b); }

// Whether the single row `a` shares a byte with `b`: the first of b's rows that
// ends behind a's start begins before a's end.
inline bool row_meets(const Rows& a, const Rows& b) {
    const int64_t at = static_cast<const char*>(a.base) - static_cast<const char*>(b.base);
    const int64_t row = at < b.width ? 0 : floor_div(at - b.width, b.pitch) + 1;
    return row < b.rows && row * b.pitch < at + a.width;
}

// Whether two tensors share a byte: decided where their rows are equally far
// apart (views of one packed buffer), one of them has a single row, or both
// start at one place.
inline bool overlap(const Rows& a, const Rows& b) {
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

inline p3d_status check_apart(const char* fn, const Rows& written, const Rows& other) {
    if (overlap(written, other))
        return set_error(P3D_ERR_INVALID_ARG, "%s: %s must not overlap %s", fn, written.name,
                         other.name);
    return P3D_OK;
}

}  // namespace checks
}  // namespace p3d
