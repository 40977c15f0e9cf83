// block_internal.h -- device helpers and launch interfaces of the
// transformer-block operators (include/p3d_block.h). Device code here needs
// no bit-exact order of operations, so these sources let the compiler fuse
// multiply-adds.
#pragma once

#include "p3d_internal.h"
#include "p3d_block.h"

#pragma clang fp contract(fast)

namespace p3d {

// The thread's last error message (api.hip owns it).
p3d_status set_error(p3d_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
p3d_status set_ok();

// Compute units of the chip: launches are cut for it on the host, so that
// workspace sizes need no device.
constexpr int kComputeUnits = 256;

// Row ranges of the batch items, in the kernel arguments.
struct ItemTable {
    int32_t start[P3D_MAX_BATCH + 1];
};

// ---------------------------------------------------------------------------
// Sums and maxima over the lanes of a group of 2^k lanes, the result in every
// lane: quad permutes and mirrors inside 16 lanes, then swaps of 16-lane rows
// and of halves. Every lane adds the same two partial results, so all lanes
// hold the same bits.
// ---------------------------------------------------------------------------
template <int Ctrl>
__device__ __forceinline__ float dpp(float v) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), Ctrl, 0xf, 0xf, true));
}

__device__ __forceinline__ float other_row16(float v, float& own) {
    auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    own = __uint_as_float(r[0]);
    return __uint_as_float(r[1]);
}

__device__ __forceinline__ float other_half(float v, float& own) {
    auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    own = __uint_as_float(r[0]);
    return __uint_as_float(r[1]);
}

template <int Lanes>
__device__ __forceinline__ float lane_sum(float v) {
    static_assert(Lanes == 1 || Lanes == 2 || Lanes == 4 || Lanes == 8 || Lanes == 16 ||
                  Lanes == 32 || Lanes == 64, "lane group");
    float a;
    if constexpr (Lanes >= 2) v += dpp<0xB1>(v);         // quad_perm [1, 0, 3, 2]
    if constexpr (Lanes >= 4) v += dpp<0x4E>(v);         // quad_perm [2, 3, 0, 1]
    if constexpr (Lanes >= 8) v += dpp<0x141>(v);        // row_half_mirror
    if constexpr (Lanes >= 16) v += dpp<0x140>(v);       // row_mirror
    if constexpr (Lanes >= 32) { const float b = other_row16(v, a); v = a + b; }
    if constexpr (Lanes >= 64) { const float b = other_half(v, a); v = a + b; }
    return v;
}

__device__ __forceinline__ float lane_max(float v) {
    float a;
    v = fmaxf(v, dpp<0xB1>(v));
    v = fmaxf(v, dpp<0x4E>(v));
    v = fmaxf(v, dpp<0x141>(v));
    v = fmaxf(v, dpp<0x140>(v));
    { const float b = other_row16(v, a); v = fmaxf(a, b); }
    { const float b = other_half(v, a); v = fmaxf(a, b); }
    return v;
}

// ---------------------------------------------------------------------------
// 16-byte vectors of elements as floats: 8 bf16 or 4 binary32.
// ---------------------------------------------------------------------------
struct Bf16 { uint16_t bits; };

template <typename T> struct Vec;
template <> struct Vec<Bf16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void widen(uint4 v, float (&f)[8]) {
        f[0] = bf16lo(v.x); f[1] = bf16hi(v.x); f[2] = bf16lo(v.y); f[3] = bf16hi(v.y);
        f[4] = bf16lo(v.z); f[5] = bf16hi(v.z); f[6] = bf16lo(v.w); f[7] = bf16hi(v.w);
    }
    static __device__ __forceinline__ uint4 narrow(const float (&f)[8]) {
        return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                          pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
    }
};
template <> struct Vec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void widen(uint4 v, float (&f)[4]) {
        f[0] = __uint_as_float(v.x); f[1] = __uint_as_float(v.y);
        f[2] = __uint_as_float(v.z); f[3] = __uint_as_float(v.w);
    }
    static __device__ __forceinline__ uint4 narrow(const float (&f)[4]) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                          __float_as_uint(f[3]));
    }
};

// ---------------------------------------------------------------------------
// Launch interfaces.
// ---------------------------------------------------------------------------
struct NormArgs {
    const void *x, *y, *gate, *scale, *shift, *weight, *bias, *post_weight;
    void *r, *h;
    int64_t n, mod_stride;
    int32_t batch, dim, pre, post;
    float res_scale, eps;
    // backward
    const void *dh, *dr;
    void *dx, *dy;
    float *dgate, *dscale, *dshift, *dweight, *dbias, *dpost_weight;
    float* partial;             // [chunks][3][dim] column sums, then [batch][3][dim]
};

hipError_t launch_gated_norm(const NormArgs& a, p3d_dtype dt, const ItemTable& items,
                             hipStream_t s);
hipError_t launch_gated_norm_backward(const NormArgs& a, p3d_dtype dt, const ItemTable& items,
                                      hipStream_t s);
// Row chunks of the backward launch: chunk_start[b] .. chunk_start[b + 1] are
// item b's. Returns the rows per chunk.
int64_t norm_chunks(int64_t n, int32_t batch, const ItemTable& items, ItemTable* chunk_start);

struct RotaryArgs {
    const void *x, *dout, *gamma;
    void *out;                  // out, or dx
    const int32_t* positions;
    const float* freqs;
    int64_t n, x_stride, dout_stride, out_stride;
    int32_t heads, head_dim, axes, pairs, pos_stride, layout;
    float magnitude, eps;
    float *dgamma, *partial;
};

hipError_t launch_rotary(const RotaryArgs& a, p3d_dtype dt, bool backward, hipStream_t s);
size_t rotary_partial_bytes(int64_t n, int32_t heads, int32_t head_dim, p3d_dtype dt);

struct AttnArgs {
    const void *q, *k, *v, *out_in, *dout;
    void *out, *dq, *dk, *dv;
    float* lse;                 // forward: written or NULL
    const float* lse_in;
    int64_t q_stride, k_stride, v_stride, out_stride, dout_stride, dq_stride, dk_stride,
        dv_stride;
    int32_t batch, heads, kv_heads, head_dim, causal;
    float scale;
    ItemTable q_items, k_items;
};

// How a forward or backward launch is cut (host-only; sizes the workspace).
struct AttnPlan {
    bool single;                // every item's rows fit one wave: the waves split the keys
    int32_t share;              // single: keys of a part
    int32_t few;                // every item has at most 32 few keys (1 or 2): they stay in LDS
    int32_t per_tile;           // query rows of a tile
    int32_t units;              // row tiles x key heads
    int32_t whole, parts;       // units run whole; parts of the keys of every later one
    int32_t dq_splits, dk_splits; // backward: parts of the keys for dq, of the rows for dk, dv
    size_t forward_bytes, backward_bytes;
};

AttnPlan attention_plan(const AttnArgs& a);
void plan_attention_backward(const AttnArgs& a, AttnPlan* p);
hipError_t launch_attention(const AttnArgs& a, const AttnPlan& p, void* ws, hipStream_t s);
hipError_t launch_attention_backward(const AttnArgs& a, const AttnPlan& p, void* ws,
                                     hipStream_t s);

}  // namespace p3d
