// block_rotary.hip -- p3d_rotary and p3d_rotary_backward: rms-normed heads
// turned by the tokens' positions (include/p3d_block.h).
//
// Every element e of a head becomes  x^[e] C[e] + x^[e'] S[e],  e' the other
// element of its pair, C = m cos, S = -m sin for the first of the pair and
// +m sin for the second; (C, S) = (1, 0) past the turned part. The gradient is
// the same with S negated. Both directions read and write every element once
// and are bound by memory: 100,000 tokens of 24 bf16 heads of 128 take 220 us
// (5.6 TB/s), and backward with the gains' gradient 392 us (4.7 TB/s: its 253
// registers leave two waves a SIMD to keep loads in flight) and 7 for the sums;
// 4096 tokens of 32 binary32 heads of 64 17 and 28 us (14 and 26 when the caches
// hold them) and 4 for the sums, held up by the loads of the few rows of a chunk.
//
// A group of P2 lanes (a power of two) holds one head, one 16-byte vector per
// lane, so its rms sum stays inside a wave. The angles of a token do not
// depend on the head: the workgroup computes each token's cosines and sines
// once into LDS (angle position * frequency in turns, reduced in binary64) and
// every thread then keeps the C and S of its vector in registers over the
// heads it walks. Pairs of the half layout, which need not be a whole number
// of vectors apart, meet through LDS inside the wave.
#include <algorithm>

#include "block_internal.h"

namespace p3d {

namespace {

constexpr int kThreads = 256;
constexpr int kKeep = 4;                 // heads per thread of the backward kernel

// cos and sin of the angle pos * freq radians. The product of an int32 and a
// binary32 is exact to 2^-53 in binary64, so the fraction of a turn is good
// to 2^-22 at the largest position there is.
__device__ __forceinline__ float2 phase(int32_t pos, float freq) {
    const double turns = (double)pos * (double)freq * 0.15915494309189533577;
    const float f = (float)(turns - rint(turns));
    float2 r;
    sincospif(2.0f * f, &r.y, &r.x);
    return r;
}

// This wave's LDS stores are seen by its own later loads.
__device__ __forceinline__ void wave_lds_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// The angles of `count` tokens from token t0 on: table[k * P + p].
__device__ __forceinline__ void fill_phases(const RotaryArgs& a, int64_t t0, int count, int P,
                                            float2* table) {
    for (int q = threadIdx.x; q < count * P; q += kThreads) {
        const int k = q / P, p = q - k * P;
        const int axis = (p >= a.pairs) + (p >= 2 * a.pairs);
        const int64_t t = t0 + k;
        table[q] = t < a.n ? phase(a.positions[t * a.pos_stride + axis],
                                   a.freqs[p - axis * a.pairs])
                           : make_float2(1.f, 0.f);
    }
}

// C and S of the elements of vector v, from one token's row of the table;
// `turn` is +1 (forward) or -1 (gradient).
template <int N>
__device__ __forceinline__ void coefficients(const RotaryArgs& a, const float2* row, int v, int P,
                                             float turn, float (&C)[N], float (&S)[N]) {
#pragma unroll
    for (int e = 0; e < N; ++e) {
        const int at = v * N + e;
        const bool half = a.layout == P3D_ROTARY_HALF;
        const bool second = half ? at >= P : (e & 1);
        const int p = half ? (second ? at - P : at) : at >> 1;
        const float2 cs = row[p < P ? p : 0];
        const bool in = at < 2 * P;
        C[e] = in ? a.magnitude * cs.x : 1.f;
        S[e] = in ? (second ? turn : -turn) * a.magnitude * cs.y : 0.f;
    }
}

// x <- x C + partner S. `slot` is the group's head in LDS (half layout).
template <int N>
__device__ __forceinline__ void turn_pairs(const RotaryArgs& a, float (&x)[N], int v, int P,
                                           const float (&C)[N], const float (&S)[N],
                                           float* slot, bool live) {
    float y[N];
    if (a.layout == P3D_ROTARY_HALF) {
        wave_lds_fence();                    // the last head's partners are read
        if (live) {
#pragma unroll
            for (int e = 0; e < N; e += 4)
                *reinterpret_cast<float4*>(slot + v * N + e) =
                    make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
        }
        wave_lds_fence();
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const int at = v * N + e;
            const int q = at >= P ? at - P : at + P;
            y[e] = live && at < 2 * P ? slot[q] : 0.f;
        }
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e) y[e] = x[e ^ 1];
    }
#pragma unroll
    for (int e = 0; e < N; ++e) x[e] = x[e] * C[e] + y[e] * S[e];
}

template <typename T>
__device__ __forceinline__ uint4 load_vec(const void* base, int64_t element, bool live) {
    constexpr int E = 16 / Vec<T>::N;
    return live ? *reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(base) +
                                                  element * E)
                : make_uint4(0, 0, 0, 0);
}

// `nt`: past the caches.
template <typename T>
__device__ __forceinline__ void store_vec(void* base, int64_t element, uint4 v, bool nt) {
    constexpr int E = 16 / Vec<T>::N;
    uint4* p = reinterpret_cast<uint4*>(reinterpret_cast<char*>(base) + element * E);
    if (nt) store_nt16(p, v);
    else *p = v;
}

// The forward call, and (turn = -1, no gamma) the gradient of the rotation
// alone. A token's heads are walked by `head_slots` groups; the host takes a
// wave's worth of groups per token when there are tokens enough to fill the
// chip and a workgroup's worth when there are not.
template <typename T, int P2>
__global__ __launch_bounds__(kThreads) void rotary_kernel(RotaryArgs a, int head_slots,
                                                          float turn, bool nt) {
    constexpr int N = Vec<T>::N;
    constexpr int kSlots = kThreads / P2;
    extern __shared__ float2 table[];                    // [tokens of the workgroup][P]
    __shared__ alignas(16) float heads_lds[kSlots * P2 * N];
    const int P = a.axes * a.pairs;
    const int tokens = kSlots / head_slots;
    const int v = threadIdx.x % P2, slot = threadIdx.x / P2;
    const int mine = slot / head_slots, h0 = slot - mine * head_slots;
    const float inv_dim = 1.0f / (float)a.head_dim;
    for (int64_t t0 = (int64_t)blockIdx.x * tokens; t0 < a.n; t0 += (int64_t)gridDim.x * tokens) {
        __syncthreads();                     // the last tokens' table is read
        fill_phases(a, t0, tokens, P, table);
        __syncthreads();
        const int64_t t = t0 + mine;
        const bool live = t < a.n && v * N < a.head_dim;
        float C[N], S[N];
        coefficients<N>(a, table + mine * P, v, P, turn, C, S);
        // the next head's vectors are on their way while one is turned
        const int64_t row = t * a.x_stride + v * N;
        uint4 next_x = load_vec<T>(a.x, row + (int64_t)h0 * a.head_dim, live && h0 < a.heads);
        uint4 next_g = load_vec<T>(a.gamma, (int64_t)h0 * a.head_dim + v * N,
                                   a.gamma && live && h0 < a.heads);
        for (int h = h0; h < a.heads; h += head_slots) {
            float x[N], g[N];
            Vec<T>::widen(next_x, x);
            Vec<T>::widen(next_g, g);
            const int64_t ahead = (int64_t)(h + head_slots) * a.head_dim;
            const bool more = live && h + head_slots < a.heads;
            next_x = load_vec<T>(a.x, row + ahead, more);
            next_g = load_vec<T>(a.gamma, ahead + v * N, a.gamma && more);
            if (a.gamma) {
                float q = 0.f;
#pragma unroll
                for (int e = 0; e < N; ++e) q += x[e] * x[e];
                const float rstd = 1.0f / sqrtf(lane_sum<P2>(q) * inv_dim + a.eps);
#pragma unroll
                for (int e = 0; e < N; ++e) x[e] *= rstd * g[e];
            }
            turn_pairs<N>(a, x, v, P, C, S, heads_lds + slot * P2 * N, live);
            if (live)
                store_vec<T>(a.out, t * a.out_stride + (int64_t)h * a.head_dim + v * N,
                             Vec<T>::narrow(x), nt);
        }
    }
}

// The gradient with gamma. A workgroup walks one chunk of tokens; a thread
// keeps kKeep heads' shares of dgamma in registers, the token lanes join
// through LDS in a fixed order at the end, and the chunks' sums are joined by
// rotary_join_kernel.
template <typename T, int P2>
__global__ __launch_bounds__(kThreads) void rotary_backward_kernel(RotaryArgs a, int head_slots,
                                                                   int token_lanes, int batch,
                                                                   int64_t tokens_per_chunk,
                                                                   bool nt) {
    constexpr int N = Vec<T>::N;
    constexpr int kSlots = kThreads / P2;
    extern __shared__ float2 table[];                    // [batch * token_lanes][P]
    __shared__ alignas(16) float heads_lds[kSlots * P2 * N];
    const int P = a.axes * a.pairs;
    const int v = threadIdx.x % P2, slot = threadIdx.x / P2;
    const int lane_t = slot / head_slots, hs = slot - lane_t * head_slots;
    const int head0 = blockIdx.y * head_slots * kKeep + hs;
    const int64_t first = blockIdx.x * tokens_per_chunk;
    const int64_t end = min(first + tokens_per_chunk, a.n);
    const float inv_dim = 1.0f / (float)a.head_dim;

    float acc[kKeep][N];
#pragma unroll
    for (int k = 0; k < kKeep; ++k)
#pragma unroll
        for (int e = 0; e < N; ++e) acc[k][e] = 0.f;

    // The heads' scales stay in registers, packed; the next token's vectors
    // are on their way while one token is worked on.
    const bool mine = lane_t < token_lanes && v * N < a.head_dim;
    uint4 gamma[kKeep], next_d[kKeep], next_x[kKeep];
    auto fetch = [&](int64_t t) {
#pragma unroll
        for (int k = 0; k < kKeep; ++k) {
            const int h = head0 + k * head_slots;
            const int64_t col = (int64_t)h * a.head_dim + v * N;
            const bool there = mine && h < a.heads && t < end;
            next_d[k] = load_vec<T>(a.dout, t * a.dout_stride + col, there);
            next_x[k] = load_vec<T>(a.x, t * a.x_stride + col, there);
        }
    };
#pragma unroll
    for (int k = 0; k < kKeep; ++k) {
        const int h = head0 + k * head_slots;
        gamma[k] = load_vec<T>(a.gamma, (int64_t)h * a.head_dim + v * N, mine && h < a.heads);
    }
    fetch(first + lane_t);

    for (int64_t b0 = first; b0 < end; b0 += batch * token_lanes) {
        __syncthreads();
        fill_phases(a, b0, batch * token_lanes, P, table);
        __syncthreads();
        for (int u = 0; u < batch; ++u) {
            const int at = u * token_lanes + lane_t;
            const int64_t t = b0 + at;
            const bool here = mine && t < end;
            float C[N], S[N];
            coefficients<N>(a, table + (lane_t < token_lanes ? at : 0) * P, v, P, -1.f, C, S);
            float d[kKeep][N], x[kKeep][N];
#pragma unroll
            for (int k = 0; k < kKeep; ++k) {
                Vec<T>::widen(next_d[k], d[k]);
                Vec<T>::widen(next_x[k], x[k]);
            }
            fetch(t + token_lanes);
#pragma unroll
            for (int k = 0; k < kKeep; ++k) {
                const int h = head0 + k * head_slots;
                const bool live = here && h < a.heads;
                float g[N];
                Vec<T>::widen(gamma[k], g);
                turn_pairs<N>(a, d[k], v, P, C, S, heads_lds + slot * P2 * N, live);
                float q = 0.f, dot = 0.f;
#pragma unroll
                for (int e = 0; e < N; ++e) q += x[k][e] * x[k][e];
                const float rstd = 1.0f / sqrtf(lane_sum<P2>(q) * inv_dim + a.eps);
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    x[k][e] *= rstd;
                    acc[k][e] += d[k][e] * x[k][e];
                    d[k][e] *= g[e];
                    dot += d[k][e] * x[k][e];
                }
                dot = lane_sum<P2>(dot) * inv_dim;
#pragma unroll
                for (int e = 0; e < N; ++e) d[k][e] = rstd * (d[k][e] - x[k][e] * dot);
                if (live)
                    store_vec<T>(a.out, t * a.out_stride + (int64_t)h * a.head_dim + v * N,
                                 Vec<T>::narrow(d[k]), nt);
            }
        }
    }

    if (!a.partial) return;
    const int64_t width = (int64_t)a.heads * a.head_dim;
#pragma unroll
    for (int k = 0; k < kKeep; ++k) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < N; ++e) heads_lds[(slot * P2 + v) * N + e] = acc[k][e];
        __syncthreads();
        const int h = head0 + k * head_slots;
        if (lane_t == 0 && h < a.heads && v * N < a.head_dim) {
            float s[N];
#pragma unroll
            for (int e = 0; e < N; ++e) s[e] = acc[k][e];
            for (int l = 1; l < token_lanes; ++l)
#pragma unroll
                for (int e = 0; e < N; ++e)
                    s[e] += heads_lds[((l * head_slots + hs) * P2 + v) * N + e];
            float* o = a.partial + blockIdx.x * width + (int64_t)h * a.head_dim + v * N;
#pragma unroll
            for (int e = 0; e < N; ++e) o[e] = s[e];
        }
    }
}

constexpr int kJoinCols = 16, kJoinLanes = 64;

__global__ __launch_bounds__(kJoinCols* kJoinLanes) void rotary_join_kernel(const float* partial,
                                                                            int chunks,
                                                                            int width,
                                                                            float* out) {
    __shared__ float part[kJoinLanes][kJoinCols + 1];
    const int col = threadIdx.x % kJoinCols, lane = threadIdx.x / kJoinCols;
    const int c = blockIdx.x * kJoinCols + col;
    float s = 0.f;
    if (c < width)
#pragma unroll 4
        for (int q = lane; q < chunks; q += kJoinLanes) s += partial[(int64_t)q * width + c];
    part[lane][col] = s;
    __syncthreads();
    if (lane || c >= width) return;
    s = 0.f;
    for (int l = 0; l < kJoinLanes; ++l) s += part[l][col];
    out[c] = s;
}

// The smallest power of two of lanes that holds a head's vectors.
int group_lanes(int head_dim, int per_vector) {
    int p = 1;
    while (p * per_vector < head_dim) p *= 2;
    return p;
}

// How the backward launch is cut.
struct Cut {
    int p2, head_slots, token_lanes, head_blocks, batch;
    int64_t tokens_per_chunk;
    int chunks;
};

Cut backward_cut(int64_t n, int heads, int head_dim, int per_vector) {
    Cut c;
    c.p2 = group_lanes(head_dim, per_vector);
    const int slots = kThreads / c.p2;
    const int wanted = (heads + kKeep - 1) / kKeep;
    c.head_slots = wanted < slots ? wanted : slots;
    c.token_lanes = slots / c.head_slots;
    c.head_blocks = (heads + kKeep * c.head_slots - 1) / (kKeep * c.head_slots);
    c.batch = c.token_lanes >= 16 ? 1 : 16 / c.token_lanes;
    // about four workgroups per CU, at least 16 tokens each (4096 tokens of 32
    // binary32 heads of 64: 26.6 us, 28.4 with 8 tokens, 40.7 with 32)
    const int64_t most = 4 * kComputeUnits / c.head_blocks > 0 ? 4 * kComputeUnits / c.head_blocks
                                                               : 1;
    c.tokens_per_chunk = (n + most - 1) / most;
    if (c.tokens_per_chunk < 16) c.tokens_per_chunk = 16;
    c.chunks = (int)((n + c.tokens_per_chunk - 1) / c.tokens_per_chunk);
    return c;
}

// Results go past the caches where the call's tensors do not fit the 256 MB of
// last-level cache anyway, as those of the gated norm do.
bool past_caches(const RotaryArgs& a, int planes, int bytes) {
    return a.n * a.heads * a.head_dim * planes * bytes > (int64_t(256) << 20);
}

template <typename T, int P2>
hipError_t forward_as(const RotaryArgs& a, float turn, hipStream_t s) {
    const int slots = kThreads / P2;
    // one wave per token while that gives every CU a workgroup
    int head_slots = P2 >= 64 ? 1 : 64 / P2;
    if (a.n * head_slots < (int64_t)kComputeUnits * slots) head_slots = slots;
    const int tokens = slots / head_slots;
    const size_t lds = (size_t)tokens * a.axes * a.pairs * sizeof(float2);
    // (a launch holds under 2^32 threads)
    const int64_t blocks = std::min<int64_t>((a.n + tokens - 1) / tokens, int64_t(1) << 22);
    rotary_kernel<T, P2><<<dim3((unsigned)blocks), dim3(kThreads), lds, s>>>(
        a, head_slots, turn, past_caches(a, 2, 16 / Vec<T>::N));
    return hipGetLastError();
}

template <typename T, int P2>
hipError_t backward_as(const RotaryArgs& a, const Cut& c, hipStream_t s) {
    const size_t lds = (size_t)c.batch * c.token_lanes * a.axes * a.pairs * sizeof(float2);
    rotary_backward_kernel<T, P2>
        <<<dim3((unsigned)c.chunks, (unsigned)c.head_blocks), dim3(kThreads), lds, s>>>(
            a, c.head_slots, c.token_lanes, c.batch, c.tokens_per_chunk,
            past_caches(a, 3, 16 / Vec<T>::N));
    return hipGetLastError();
}

template <typename T>
hipError_t launch_as(const RotaryArgs& a, bool backward, hipStream_t s) {
    const bool full = backward && a.gamma;
    const float turn = backward ? -1.f : 1.f;
    const Cut c = backward_cut(a.n, a.heads, a.head_dim, Vec<T>::N);
#define P3D_ROTARY_CASE(P) \
    case P: return full ? backward_as<T, P>(a, c, s) : forward_as<T, P>(a, turn, s)
    switch (c.p2) {
        P3D_ROTARY_CASE(1);
        P3D_ROTARY_CASE(2);
        P3D_ROTARY_CASE(4);
        P3D_ROTARY_CASE(8);
        P3D_ROTARY_CASE(16);
        P3D_ROTARY_CASE(32);
        default: break;
    }
#undef P3D_ROTARY_CASE
    return full ? backward_as<T, 64>(a, c, s) : forward_as<T, 64>(a, turn, s);
}

}  // namespace

size_t rotary_partial_bytes(int64_t n, int32_t heads, int32_t head_dim, p3d_dtype dt) {
    const Cut c = backward_cut(n, heads, head_dim, dt == P3D_BF16 ? 8 : 4);
    return (size_t)c.chunks * heads * head_dim * sizeof(float);
}

hipError_t launch_rotary(const RotaryArgs& args, p3d_dtype dt, bool backward, hipStream_t s) {
    RotaryArgs a = args;
    if (!a.dgamma) a.partial = nullptr;
    if (a.n > 0) {
        // the gradient of the rotation alone is the rotation back
        if (backward && !a.gamma) { a.x = a.dout; a.x_stride = a.dout_stride; }
        const hipError_t e = dt == P3D_BF16 ? launch_as<Bf16>(a, backward, s)
                                            : launch_as<float>(a, backward, s);
        if (e != hipSuccess) return e;
    }
    if (!a.dgamma) return hipSuccess;
    const Cut c = backward_cut(a.n, a.heads, a.head_dim, dt == P3D_BF16 ? 8 : 4);
    const int width = a.heads * a.head_dim;
    rotary_join_kernel<<<dim3((unsigned)((width + kJoinCols - 1) / kJoinCols)),
                         dim3(kJoinCols * kJoinLanes), 0, s>>>(a.partial, c.chunks, width,
                                                             a.dgamma);
    return hipGetLastError();
}

}  // namespace p3d
