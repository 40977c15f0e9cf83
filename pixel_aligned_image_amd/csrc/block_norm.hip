// block_norm.hip -- p3d_gated_norm and p3d_gated_norm_backward: the step
// between two branches of a transformer block (include/p3d_block.h).
//
//   t = post(y) post_weight,  r = x + s gate t,
//   h = (pre(r) weight + bias)(1 + scale) + shift
//
// Both directions read every tensor once and keep a row in registers between
// the read and the last write: the forward call moves 4 planes (x, y in; r, h
// out), the backward call 6 (x, y, dh, dr in; dx, dy out), and nothing else
// grows with the rows. Both are bound by memory: 100,000 rows of 1536 bf16
// take 222 us forward (5.5 TB/s), 200,000 rows 448 us and backward 739 us (5.0
// TB/s; its loop reads two registers back from memory); 4096 rows of 1024
// binary32 14 and 26 us (22 when the caches hold them) with 5 us of sums; 5 rows
// 5 us, a launch. A row belongs to a group of
// 16, 32, 64 or 256 threads, the smallest that holds it in at most VPT
// 16-byte vectors each, so that its sums stay inside a wave wherever they can
// (DPP, no LDS) and no lane idles on narrow rows.
//
// The variance is the mean of squared deviations from the mean already known
// (the row is in registers, so the second pass is free), not a difference of
// two large sums.
#include <algorithm>

#include "block_internal.h"

namespace p3d {

// About four workgroups per CU, and at least 16 rows each, so that the chunk
// sums (12 bytes per column and chunk, written and read once) stay small
// beside the rows (4096 rows: 23 + 4.6 us with 16, 21 + 6.1 with 8, 26 + 9.4
// with 4).
int64_t norm_chunks(int64_t n, int32_t batch, const ItemTable& items, ItemTable* chunks) {
    const int64_t most = 4 * kComputeUnits;
    const int64_t rpc = std::max<int64_t>((n + most - 1) / most, 16);
    int32_t at = 0;
    for (int32_t b = 0; b < batch; ++b) {
        chunks->start[b] = at;
        at += (int32_t)((items.start[b + 1] - items.start[b] + rpc - 1) / rpc);
    }
    for (int32_t b = batch; b <= P3D_MAX_BATCH; ++b) chunks->start[b] = at;
    return rpc;
}

namespace {

constexpr int kThreads = 256;

// Item of a row: the last one that starts at or before it.
__device__ __forceinline__ int item_of(const ItemTable& t, int batch, int64_t row) {
    int lo = 0, hi = batch;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (t.start[mid] <= row) lo = mid; else hi = mid;
    }
    return lo;
}

// Sum over the TPR threads of a row. For TPR == kThreads, `red` holds one
// float per wave and the two barriers keep its uses apart.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* red) {
    if constexpr (TPR <= 64) {
        return lane_sum<TPR>(v);
    } else {
        v = lane_sum<64>(v);
        __syncthreads();
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
        __syncthreads();
        return (red[0] + red[1]) + (red[2] + red[3]);
    }
}

// A thread's vectors of a row: vector u * TPR + t, zeros past the row's end.
template <typename T, int VPT, int TPR>
struct RowVec {
    static constexpr int N = Vec<T>::N;
    float f[VPT][N];

    __device__ __forceinline__ void widen(const uint4 (&q)[VPT]) {
#pragma unroll
        for (int u = 0; u < VPT; ++u) Vec<T>::widen(q[u], f[u]);
    }
};

// A row's vectors as they lie, zeros past its end and where there is no
// tensor or (`live`) no row.
template <int VPT, int TPR>
__device__ __forceinline__ void load_row(uint4 (&q)[VPT], const void* base, int64_t row, int nv,
                                         int t, bool live = true) {
    const uint4* p = reinterpret_cast<const uint4*>(base) + row * nv;
    const int vectors = base && live ? nv : 0;
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
        const int v = u * TPR + t;
        q[u] = v < vectors ? p[v] : make_uint4(0, 0, 0, 0);
    }
}

// One vector of a per-column parameter, `other` where it is absent.
template <typename T>
__device__ __forceinline__ void param(const void* base, int64_t offset, int v, int nv,
                                      float other, float (&f)[Vec<T>::N]) {
    if (base) {
        const uint4* p = reinterpret_cast<const uint4*>(base) + offset;
        Vec<T>::widen(v < nv ? p[v] : make_uint4(0, 0, 0, 0), f);
    } else {
#pragma unroll
        for (int e = 0; e < Vec<T>::N; ++e) f[e] = other;
    }
}

// One value of a per-column parameter, `other` where it is absent.
template <typename T>
__device__ __forceinline__ float column(const void* base, int64_t i, float other) {
    if (!base) return other;
    if constexpr (sizeof(T) == 4) return reinterpret_cast<const float*>(base)[i];
    else return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(base)[i] << 16);
}

// What a vector's columns are multiplied or shifted by.
template <int N>
__device__ __forceinline__ void factors(const float* lds, int v, float (&f)[N]) {
#pragma unroll
    for (int e = 0; e < N; e += 4) {
        const float4 q = *reinterpret_cast<const float4*>(lds + v * N + e);
        f[e] = q.x, f[e + 1] = q.y, f[e + 2] = q.z, f[e + 3] = q.w;
    }
}

// v <- (v - mean) / deviation in place (0 past the row's end); returns the
// reciprocal deviation (1 for NONE).
template <typename T, int VPT, int TPR>
__device__ __forceinline__ float normalise(RowVec<T, VPT, TPR>& v, int kind, int nv, int t,
                                           float inv_dim, float eps, float* red) {
    constexpr int N = Vec<T>::N;
    if (kind == P3D_NORM_NONE) return 1.0f;
    if (kind == P3D_NORM_LAYER) {
        float s = 0.f;
#pragma unroll
        for (int u = 0; u < VPT; ++u)
#pragma unroll
            for (int e = 0; e < N; ++e) s += v.f[u][e];
        const float mean = row_sum<TPR>(s, red) * inv_dim;
#pragma unroll
        for (int u = 0; u < VPT; ++u) {
            const bool in = u * TPR + t < nv;
#pragma unroll
            for (int e = 0; e < N; ++e) v.f[u][e] = in ? v.f[u][e] - mean : 0.f;
        }
    }
    float q = 0.f;
#pragma unroll
    for (int u = 0; u < VPT; ++u)
#pragma unroll
        for (int e = 0; e < N; ++e) q += v.f[u][e] * v.f[u][e];
    const float rstd = 1.0f / sqrtf(row_sum<TPR>(q, red) * inv_dim + eps);
#pragma unroll
    for (int u = 0; u < VPT; ++u)
#pragma unroll
        for (int e = 0; e < N; ++e) v.f[u][e] *= rstd;
    return rstd;
}

// d <- the gradient of the norm's input from the gradient d of its output n:
// rstd (d - n mean(d n) - mean(d)), the last term for LAYER only (0 past the
// row's end).
template <typename T, int VPT, int TPR>
__device__ __forceinline__ void normalise_backward(RowVec<T, VPT, TPR>& d,
                                                   const RowVec<T, VPT, TPR>& n, int kind,
                                                   float rstd, int nv, int t, float inv_dim,
                                                   float* red) {
    constexpr int N = Vec<T>::N;
    if (kind == P3D_NORM_NONE) return;
    float s = 0.f, q = 0.f;
#pragma unroll
    for (int u = 0; u < VPT; ++u)
#pragma unroll
        for (int e = 0; e < N; ++e) {
            s += d.f[u][e];
            q += d.f[u][e] * n.f[u][e];
        }
    const float dot = row_sum<TPR>(q, red) * inv_dim;
    const float mean = kind == P3D_NORM_LAYER ? row_sum<TPR>(s, red) * inv_dim : 0.f;
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
        const bool in = u * TPR + t < nv;
#pragma unroll
        for (int e = 0; e < N; ++e)
            d.f[u][e] = in ? rstd * (d.f[u][e] - n.f[u][e] * dot - mean) : 0.f;
    }
}

// A row's vectors out; `nt`: past the caches.
template <typename T, int VPT, int TPR>
__device__ __forceinline__ void store_row(const RowVec<T, VPT, TPR>& r, void* base, int64_t row,
                                          int nv, int t, bool nt) {
    uint4* p = reinterpret_cast<uint4*>(base) + row * nv;
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
        const int v = u * TPR + t;
        if (v >= nv) continue;
        const uint4 q = Vec<T>::narrow(r.f[u]);
        if (nt) store_nt16(p + v, q);
        else p[v] = q;
    }
}

template <typename T, int VPT, int TPR>
__global__ __launch_bounds__(kThreads) void gated_norm_kernel(NormArgs a, ItemTable items,
                                                              bool nt) {
    constexpr int N = Vec<T>::N;
    __shared__ float red[4];
    const int t = threadIdx.x % TPR;
    const int nv = a.dim / N;
    const float inv_dim = 1.0f / (float)a.dim;
    // a row's threads take every turn of the loop together
    for (int64_t row = (int64_t)blockIdx.x * (kThreads / TPR) + threadIdx.x / TPR; row < a.n;
         row += (int64_t)gridDim.x * (kThreads / TPR)) {
        const int64_t mod = item_of(items, a.batch, row) * (a.mod_stride / N);
        uint4 raw_x[VPT], raw_y[VPT];
        load_row<VPT, TPR>(raw_x, a.x, row, nv, t);
        load_row<VPT, TPR>(raw_y, a.y, row, nv, t);
        RowVec<T, VPT, TPR> x;
        x.widen(raw_x);
        if (a.y) {
            RowVec<T, VPT, TPR> y;
            y.widen(raw_y);
            normalise(y, a.post, nv, t, inv_dim, a.eps, red);
#pragma unroll
            for (int u = 0; u < VPT; ++u) {
                const int v = u * TPR + t;
                float g[N], w[N];
                param<T>(a.gate, mod, v, nv, 1.f, g);
                param<T>(a.post_weight, 0, v, nv, 1.f, w);
#pragma unroll
                for (int e = 0; e < N; ++e) x.f[u][e] += a.res_scale * g[e] * (y.f[u][e] * w[e]);
            }
        }
        if (a.r) store_row(x, a.r, row, nv, t, nt);
        normalise(x, a.pre, nv, t, inv_dim, a.eps, red);
#pragma unroll
        for (int u = 0; u < VPT; ++u) {
            const int v = u * TPR + t;
            float w[N], b[N], sc[N], sh[N];
            param<T>(a.weight, 0, v, nv, 1.f, w);
            param<T>(a.bias, 0, v, nv, 0.f, b);
            param<T>(a.scale, mod, v, nv, 0.f, sc);
            param<T>(a.shift, mod, v, nv, 0.f, sh);
#pragma unroll
            for (int e = 0; e < N; ++e)
                x.f[u][e] = (x.f[u][e] * w[e] + b[e]) * (1.0f + sc[e]) + sh[e];
        }
        store_row(x, a.h, row, nv, t, nt);
    }
}

// The three column sums that every parameter gradient is made of, per item:
// A = sum dh n, S = sum dh, G = sum dr t^ (n, t^ the normalised r and y). A
// workgroup walks one chunk of one item's rows with its sums in registers and
// what its columns are multiplied by in LDS, put together once; x and y of the
// next row are loaded, still packed, while a row is worked on, dh and dr before
// the statistics that come ahead of them. It joins its row groups through LDS
// in a fixed order and writes [3][dim] binary32 values; no atomics, so the
// sums' order never changes.
template <typename T, int VPT, int TPR>
__global__ __launch_bounds__(kThreads, VPT* Vec<T>::N <= 24 ? 2 : 1) void gated_norm_backward_kernel(
    NormArgs a, ItemTable items, ItemTable chunks, int64_t rows_per_chunk, bool nt) {
    constexpr int N = Vec<T>::N;
    constexpr int R = kThreads / TPR;        // rows in flight
    __shared__ float red[4];
    // [2][dim], read 16 bytes at a time, then [R][TPR * VPT * N]
    extern __shared__ __align__(16) float cols[];
    float* mul = cols;                       // weight (1 + scale)
    float* lift = cols + a.dim;              // res_scale gate post_weight
    const int t = threadIdx.x % TPR, group = threadIdx.x / TPR;
    const int nv = a.dim / N;
    const float inv_dim = 1.0f / (float)a.dim;
    const int item = item_of(chunks, a.batch, blockIdx.x);
    const int64_t first = items.start[item] +
                          (int64_t)((int)blockIdx.x - chunks.start[item]) * rows_per_chunk;
    const int64_t end = min(first + rows_per_chunk, (int64_t)items.start[item + 1]);

    // (a group past the last row reads nothing, stores nothing and adds nothing:
    // another group may have written that row's results over its inputs)
    int64_t row = first + group;
    uint4 next_x[VPT], next_y[VPT];
    load_row<VPT, TPR>(next_x, a.x, row, nv, t, row < end);
    load_row<VPT, TPR>(next_y, a.y, row, nv, t, row < end);
    const int64_t mod = item * a.mod_stride;
    for (int c = threadIdx.x; c < a.dim; c += kThreads) {
        mul[c] = column<T>(a.weight, c, 1.f) * (1.0f + column<T>(a.scale, mod + c, 0.f));
        lift[c] = a.res_scale * column<T>(a.gate, mod + c, 1.f) *
                  column<T>(a.post_weight, c, 1.f);
    }
    __syncthreads();

    float sums[3][VPT][N];
#pragma unroll
    for (int k = 0; k < 3; ++k)
#pragma unroll
        for (int u = 0; u < VPT; ++u)
#pragma unroll
            for (int e = 0; e < N; ++e) sums[k][u][e] = 0.f;

    // every thread takes the turns of the workgroup's first row
    for (int64_t top = first; top < end; top += R, row += R) {
        const bool live = row < end;
        RowVec<T, VPT, TPR> x, y, d;
        uint4 raw_d[VPT], raw_r[VPT];
        load_row<VPT, TPR>(raw_d, a.dh, row, nv, t, row < end);
        load_row<VPT, TPR>(raw_r, a.dr, row, nv, t, row < end);
        x.widen(next_x);
        if (a.y) y.widen(next_y);
        load_row<VPT, TPR>(next_x, a.x, row + R, nv, t, row + R < end);
        load_row<VPT, TPR>(next_y, a.y, row + R, nv, t, row + R < end);
        float y_rstd = 1.f;
        if (a.y) {
            y_rstd = normalise(y, a.post, nv, t, inv_dim, a.eps, red);
#pragma unroll
            for (int u = 0; u < VPT; ++u) {
                float g[N];
                factors<N>(lift, min(u * TPR + t, nv - 1), g);
#pragma unroll
                for (int e = 0; e < N; ++e) x.f[u][e] += g[e] * y.f[u][e];
            }
        }
        const float rstd = normalise(x, a.pre, nv, t, inv_dim, a.eps, red);
        d.widen(raw_d);
#pragma unroll
        for (int u = 0; u < VPT; ++u) {
            float m[N];
            factors<N>(mul, min(u * TPR + t, nv - 1), m);
#pragma unroll
            for (int e = 0; e < N; ++e) {
                sums[0][u][e] += live ? d.f[u][e] * x.f[u][e] : 0.f;
                sums[1][u][e] += live ? d.f[u][e] : 0.f;
                d.f[u][e] *= m[e];
            }
        }
        normalise_backward(d, x, a.pre, rstd, nv, t, inv_dim, red);
        if (a.dr) {
#pragma unroll
            for (int u = 0; u < VPT; ++u) {
                float f[N];
                Vec<T>::widen(raw_r[u], f);
#pragma unroll
                for (int e = 0; e < N; ++e) d.f[u][e] += f[e];
            }
        }
        if (live) store_row(d, a.dx, row, nv, t, nt);
        if (a.y) {
#pragma unroll
            for (int u = 0; u < VPT; ++u) {
                float g[N];
                factors<N>(lift, min(u * TPR + t, nv - 1), g);
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    sums[2][u][e] += live ? d.f[u][e] * y.f[u][e] : 0.f;
                    d.f[u][e] *= g[e];
                }
            }
            if (a.dy) {
                normalise_backward(d, y, a.post, y_rstd, nv, t, inv_dim, red);
                if (live) store_row(d, a.dy, row, nv, t, nt);
            }
        }
    }

    if (!a.partial) return;
    float* joint = cols + 2 * a.dim;
    float* out = a.partial + (int64_t)blockIdx.x * 3 * a.dim;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        __syncthreads();
#pragma unroll
        for (int u = 0; u < VPT; ++u)
#pragma unroll
            for (int e = 0; e < N; ++e)
                joint[(group * VPT * TPR + u * TPR + t) * N + e] = sums[k][u][e];
        __syncthreads();
        for (int c = threadIdx.x; c < a.dim; c += kThreads) {
            float s = 0.f;
            for (int g = 0; g < R; ++g) s += joint[g * VPT * TPR * N + c];
            out[k * a.dim + c] = s;
        }
    }
}

// Joins an item's chunks: 32 columns by 32 chunk lanes per workgroup, each
// lane a fixed share of the chunks.
constexpr int kJoinCols = 32, kJoinLanes = 32;

template <typename T>
__global__ __launch_bounds__(kJoinCols* kJoinLanes) void norm_join_kernel(NormArgs a,
                                                                          ItemTable chunks,
                                                                          float* item_sums) {
    __shared__ float part[3][kJoinLanes][kJoinCols + 1];
    const int col = threadIdx.x % kJoinCols, lane = threadIdx.x / kJoinCols;
    const int c = blockIdx.x * kJoinCols + col;
    const int item = blockIdx.y;
    const int64_t D = a.dim;
    float s[3] = {0.f, 0.f, 0.f};
    if (c < D) {
#pragma unroll 4
        for (int q = chunks.start[item] + lane; q < chunks.start[item + 1]; q += kJoinLanes) {
            const float* p = a.partial + q * 3 * D + c;
#pragma unroll
            for (int k = 0; k < 3; ++k) s[k] += p[k * D];
        }
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) part[k][lane][col] = s[k];
    __syncthreads();
    if (lane || c >= D) return;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        s[k] = 0.f;
        for (int l = 0; l < kJoinLanes; ++l) s[k] += part[k][l][col];
    }
    const float A = s[0], S = s[1], G = s[2];
    const int64_t at = item * D + c;
    const float gate = column<T>(a.gate, item * a.mod_stride + c, 1.f);
    const float scale = 1.0f + column<T>(a.scale, item * a.mod_stride + c, 0.f);
    if (a.dgate) a.dgate[at] = a.res_scale * column<T>(a.post_weight, c, 1.f) * G;
    if (a.dscale)
        a.dscale[at] = column<T>(a.weight, c, 1.f) * A + column<T>(a.bias, c, 0.f) * S;
    if (a.dshift) a.dshift[at] = S;
    if (item_sums) {
        float* o = item_sums + (int64_t)item * 3 * D + c;
        o[0] = scale * A;
        o[D] = scale * S;
        o[2 * D] = a.res_scale * gate * G;
    } else {                                 // one item: its sums are the whole
        if (a.dweight) a.dweight[c] = scale * A;
        if (a.dbias) a.dbias[c] = scale * S;
        if (a.dpost_weight) a.dpost_weight[c] = a.res_scale * gate * G;
    }
}

// The [dim] parameters' gradients: the items' shares added in item order.
__global__ __launch_bounds__(kThreads) void norm_items_kernel(NormArgs a,
                                                              const float* item_sums) {
    const int c = blockIdx.x * kThreads + threadIdx.x;
    if (c >= a.dim) return;
    const int64_t D = a.dim;
    float s[3] = {0.f, 0.f, 0.f};
    for (int b = 0; b < a.batch; ++b)
#pragma unroll
        for (int k = 0; k < 3; ++k) s[k] += item_sums[(b * 3 + k) * D + c];
    if (a.dweight) a.dweight[c] = s[0];
    if (a.dbias) a.dbias[c] = s[1];
    if (a.dpost_weight) a.dpost_weight[c] = s[2];
}

// Results go past the caches where the call's tensors do not fit the 256 MB of
// last-level cache anyway (100,000 rows of 1536 bf16: 260 -> 229 us); below
// that the next call finds them there.
bool past_caches(const NormArgs& a, int planes, int bytes) {
    return a.n * a.dim * planes * bytes > (int64_t(256) << 20);
}

template <typename T, int VPT, int TPR>
hipError_t forward_as(const NormArgs& a, const ItemTable& items, hipStream_t s) {
    const int64_t rows = kThreads / TPR;
    // (a launch holds under 2^32 threads)
    const int64_t blocks = std::min<int64_t>((a.n + rows - 1) / rows, int64_t(1) << 22);
    gated_norm_kernel<T, VPT, TPR><<<dim3((unsigned)blocks), dim3(kThreads), 0, s>>>(
        a, items, past_caches(a, 4, 16 / Vec<T>::N));
    return hipGetLastError();
}

template <typename T, int VPT, int TPR>
hipError_t backward_as(const NormArgs& a, const ItemTable& items, const ItemTable& chunks,
                       int64_t rows_per_chunk, hipStream_t s) {
    const size_t lds = (2 * a.dim + kThreads * VPT * Vec<T>::N) * sizeof(float);
    gated_norm_backward_kernel<T, VPT, TPR>
        <<<dim3((unsigned)chunks.start[a.batch]), dim3(kThreads), lds, s>>>(
            a, items, chunks, rows_per_chunk, past_caches(a, 6, 16 / Vec<T>::N));
    return hipGetLastError();
}

// The group of threads of a row of `nv` vectors, and its vectors per thread:
// the smallest group that keeps a row's values in registers (the backward call
// also its three sums: 24 columns a thread), else the whole workgroup. Backward,
// bf16 rows of 1536 take 755 us for 200,000 in a wave and 850 in a workgroup;
// binary32 rows of 1536, whose packed vectors are twice as many registers, 991
// us for 77,367 in a wave (71 registers spilled) and 600 in a workgroup.
template <typename T>
hipError_t forward_of(const NormArgs& a, const ItemTable& items, hipStream_t s) {
    const int nv = a.dim / Vec<T>::N;
    if (nv <= 16) return forward_as<T, 1, 16>(a, items, s);
    if (nv <= 32) return forward_as<T, 1, 32>(a, items, s);
    if (nv <= 64) return forward_as<T, 1, 64>(a, items, s);
    if (nv <= 128) return forward_as<T, 2, 64>(a, items, s);
    if (nv <= 192) return forward_as<T, 3, 64>(a, items, s);
    if (nv <= 256) return forward_as<T, 4, 64>(a, items, s);
    if constexpr (Vec<T>::N == 4) {
        if (nv <= 384) return forward_as<T, 6, 64>(a, items, s);
        if (nv > 1024) return forward_as<T, 8, 256>(a, items, s);
    }
    if (nv <= 512) return forward_as<T, 2, 256>(a, items, s);
    return forward_as<T, 4, 256>(a, items, s);
}

template <typename T>
hipError_t backward_of(const NormArgs& a, const ItemTable& items, const ItemTable& chunks,
                       int64_t rpc, hipStream_t s) {
    const int nv = a.dim / Vec<T>::N;
    if (nv <= 16) return backward_as<T, 1, 16>(a, items, chunks, rpc, s);
    if (nv <= 32) return backward_as<T, 1, 32>(a, items, chunks, rpc, s);
    if (nv <= 64) return backward_as<T, 1, 64>(a, items, chunks, rpc, s);
    if (nv <= 128) return backward_as<T, 2, 64>(a, items, chunks, rpc, s);
    if (nv <= 192) return backward_as<T, 3, 64>(a, items, chunks, rpc, s);
    if constexpr (Vec<T>::N == 4) {
        if (nv <= 256) return backward_as<T, 4, 64>(a, items, chunks, rpc, s);
        if (nv > 1024) return backward_as<T, 8, 256>(a, items, chunks, rpc, s);
    }
    if (nv <= 256) return backward_as<T, 1, 256>(a, items, chunks, rpc, s);
    if (nv <= 512) return backward_as<T, 2, 256>(a, items, chunks, rpc, s);
    return backward_as<T, 4, 256>(a, items, chunks, rpc, s);
}

}  // namespace

hipError_t launch_gated_norm(const NormArgs& a, p3d_dtype dt, const ItemTable& items,
                             hipStream_t s) {
    return dt == P3D_BF16 ? forward_of<Bf16>(a, items, s) : forward_of<float>(a, items, s);
}

hipError_t launch_gated_norm_backward(const NormArgs& args, p3d_dtype dt, const ItemTable& items,
                                      hipStream_t s) {
    NormArgs a = args;
    ItemTable chunks;
    const int64_t rpc = norm_chunks(a.n, a.batch, items, &chunks);
    const bool shared = a.dweight || a.dbias || a.dpost_weight;
    const bool sums = shared || a.dgate || a.dscale || a.dshift;
    if (!sums) a.partial = nullptr;
    if (chunks.start[a.batch] > 0) {
        const hipError_t e = dt == P3D_BF16 ? backward_of<Bf16>(a, items, chunks, rpc, s)
                                            : backward_of<float>(a, items, chunks, rpc, s);
        if (e != hipSuccess) return e;
    }
    if (!sums) return hipSuccess;
    float* item_sums = shared && a.batch > 1
                           ? a.partial + (int64_t)chunks.start[a.batch] * 3 * a.dim
                           : nullptr;
    const dim3 grid((unsigned)((a.dim + kJoinCols - 1) / kJoinCols), (unsigned)a.batch);
    if (dt == P3D_BF16)
        norm_join_kernel<Bf16><<<grid, dim3(kJoinCols * kJoinLanes), 0, s>>>(a, chunks, item_sums);
    else
        norm_join_kernel<float><<<grid, dim3(kJoinCols * kJoinLanes), 0, s>>>(a, chunks, item_sums);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !item_sums) return e;
    norm_items_kernel<<<dim3((unsigned)((a.dim + kThreads - 1) / kThreads)), dim3(kThreads), 0, s>>>(
        a, item_sums);
    return hipGetLastError();
}

}  // namespace p3d
