// model_internal.h -- launch interfaces and device helpers of the model's
// operators (include/p3d_model.h).
#pragma once

#include "block_internal.h"
#include "p3d_model.h"

namespace p3d {

// ---------------------------------------------------------------------------
// Activations. e^-u is a hardware exponential of a scaled argument (relative
// error |u| 2^-24 or so, where e^-u matters only for u of a few units) and the
// quotient a hardware reciprocal: a few roundings of binary32, far below a
// bf16 result's and within the tolerance of an F32 one.
// ---------------------------------------------------------------------------
__device__ __forceinline__ float logistic(float u) {
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(u * -1.44269504088896340736f));
}

constexpr float kGelu2 = 1.59576912160573071176f;       // 2 sqrt(2 / pi)
constexpr float kGelu3 = 0.044715f;

// act(u). GELU's tanh form is u logistic(2 sqrt(2 / pi) (u + 0.044715 u^3)).
template <int Act>
__device__ __forceinline__ float activate(float u) {
    if constexpr (Act == P3D_ACT_SILU) return u * logistic(u);
    if constexpr (Act == P3D_ACT_GELU) return u * logistic(kGelu2 * u * (1.f + kGelu3 * u * u));
    return u;
}

// act'(u).
template <int Act>
__device__ __forceinline__ float slope(float u) {
    if constexpr (Act == P3D_ACT_SILU) {
        const float p = logistic(u);
        return p * (1.f + u * (1.f - p));
    }
    if constexpr (Act == P3D_ACT_GELU) {
        // (p (1 - p) is 0 long before u^2 reaches the bound, which keeps inf from it)
        const float u2 = fminf(u * u, 1e4f);
        const float p = logistic(kGelu2 * u * (1.f + kGelu3 * u2));
        return p + u * p * (1.f - p) * kGelu2 * (1.f + 3.f * kGelu3 * u2);
    }
    return 1.f;
}

// ---------------------------------------------------------------------------
// Launch interfaces.
// ---------------------------------------------------------------------------
struct GroupArgs {
    const void *x, *dout, *weight, *bias;
    void *out, *dx;
    int64_t x_stride, dout_stride, out_stride;  // out_stride: of out or dx
    int32_t batch, channels, groups, act;
    float eps;
    float *mean, *rstd;             // forward: written or NULL
    const float *mean_in, *rstd_in;
    float *dweight, *dbias;
    ItemTable items;
};

// How a call is cut: its channels into `slices`, every item's rows into chunks,
// chunk.start[b] .. chunk.start[b + 1] item b's.
struct GroupPlan {
    int32_t small;                  // slices of the one-launch kernels, or 0: items too long
    int32_t slices, ty;             // rows of a chunk's blocks
    ItemTable chunk;
    size_t bytes;                   // of the workspace
};

GroupPlan group_norm_plan(const GroupArgs& a, p3d_dtype dt);
hipError_t launch_group_norm(const GroupArgs& a, const GroupPlan& p, p3d_dtype dt, void* ws,
                             hipStream_t s);
hipError_t launch_group_norm_backward(const GroupArgs& a, const GroupPlan& p, p3d_dtype dt,
                                      void* ws, hipStream_t s);

struct QuantizeArgs {
    const void* x;
    int64_t n, x_stride, q_stride;
    int32_t width;
    int8_t* q;
    float* scale;
};

hipError_t launch_quantize_rows(const QuantizeArgs& a, p3d_dtype dt, hipStream_t s);

struct LinearArgs {
    const int8_t *q, *weight;
    const float *scale, *weight_scale;
    const void *bias, *residual;
    void* out;
    int64_t n, q_stride, residual_stride, out_stride;
    int32_t in_dim, out_dim, act;
};

hipError_t launch_linear_i8(const LinearArgs& a, p3d_dtype dt, hipStream_t s);

// Partial sums of squares that p3d_grad_norm's workspace holds.
int64_t grad_norm_parts(const p3d_adamw_desc& d);
hipError_t launch_grad_norm(const p3d_adamw_desc& d, float max_norm, float* out, double* parts,
                            hipStream_t s);
hipError_t launch_adamw(const p3d_adamw_desc& d, hipStream_t s);

}  // namespace p3d
