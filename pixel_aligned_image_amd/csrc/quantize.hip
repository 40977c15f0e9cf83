// quantize.hip -- p3d_quantize_rows: rows in 8-bit integers with a scale each.
//
//   s = max |x| * (1 / 127),  q = x / s to the nearest integer, ties to even
//
// A row is read once: it stays in registers between its maximum and its
// quotients. Memory bound (3 bytes a bf16 element; 105 us for 100,000 rows of 2048,
// 5.8 TB/s) only if an element costs fewer than 20 operations, so the quotient has
// to be cheap and exact. x (1 / s) is off by two roundings of 127 at most: where it
// is further than that from the middle between two integers, the nearest to it is
// the nearest to x / s. A wave with an element nearer to a middle (8 % of rows of
// 2048) takes the remainder x - q s, which one fused operation gives without
// rounding.
#include <algorithm>

#include "model_internal.h"

namespace p3d {

namespace {

constexpr int kThreads = 256;

// Eight neighbouring elements as they lie.
template <typename T> struct Raw;
template <> struct Raw<Bf16> {
    uint4 v;
    __device__ __forceinline__ void load(const void* p) { v = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void clear() { v = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void widen(float (&f)[8]) const { Vec<Bf16>::widen(v, f); }
};
template <> struct Raw<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const void* p) {
        a = reinterpret_cast<const float4*>(p)[0];
        b = reinterpret_cast<const float4*>(p)[1];
    }
    __device__ __forceinline__ void clear() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void widen(float (&f)[8]) const {
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
};

// Largest of 64 lanes' numbers. Magnitudes compare as their bits do, NaN above
// infinity above every number.
__device__ __forceinline__ uint32_t wave_umax(uint32_t v) {
    const auto step = [&](float other) { v = max(v, __float_as_uint(other)); };
    step(dpp<0xB1>(__uint_as_float(v)));
    step(dpp<0x4E>(__uint_as_float(v)));
    step(dpp<0x141>(__uint_as_float(v)));
    step(dpp<0x140>(__uint_as_float(v)));
    auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = max(r[0], r[1]);
    r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return max(r[0], r[1]);
}

// x / s to the nearest integer, ties to even, for |x| <= 127.5 s. The
// remainder x - q s is exact (both are multiples of the smaller's last place,
// and it is no larger than s), so comparing it with s / 2 decides.
__device__ __forceinline__ int nearest(float x, float s, float inv) {
    const float q = rintf(x * inv);
    const float r = fmaf(-q, s, x), half = 0.5f * s;
    const int n = (int)q;
    const int up = r > half || (r == half && (n & 1)), down = r < -half || (r == -half && (n & 1));
    return n + up - down;
}

// Waves of a row: 1, 4 or 16; V vectors of 8 elements a thread.
template <typename T, int Waves, int V>
__global__ __launch_bounds__(Waves > 4 ? 64 * Waves : kThreads) void quantize_kernel(
    QuantizeArgs a) {
    constexpr int kRow = 64 * Waves;                            // threads of a row
    constexpr int kBlock = Waves > 4 ? kRow : kThreads;
    __shared__ uint32_t tops[kBlock / 64];
    const int t = threadIdx.x % kRow, nv = a.width / 8;
    for (int64_t row0 = (int64_t)blockIdx.x * (kBlock / kRow); row0 < a.n;
         row0 += (int64_t)gridDim.x * (kBlock / kRow)) {
        const int64_t row = row0 + threadIdx.x / kRow;
        const bool live = row < a.n;
        const T* x = reinterpret_cast<const T*>(a.x) + row * a.x_stride;
        Raw<T> raw[V];
#pragma unroll
        for (int u = 0; u < V; ++u) {
            const int v = u * kRow + t;
            if (live && v < nv) raw[u].load(x + v * 8);
            else raw[u].clear();
        }
        uint32_t top = 0;
#pragma unroll
        for (int u = 0; u < V; ++u) {
            float f[8];
            raw[u].widen(f);
#pragma unroll
            for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(f[e]) & 0x7fffffffu);
        }
        top = wave_umax(top);
        if constexpr (Waves > 1) {
            if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = top;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < Waves; ++w)
                top = max(top, tops[threadIdx.x / kRow * Waves + w]);
            __syncthreads();                // (the next row writes them again)
        }
        if (!live) continue;
        const bool finite = top < 0x7f800000u;
        const float s = finite ? __uint_as_float(top) * (1.f / 127.f) : NAN;
        if (t == 0) a.scale[row] = s;
        const bool some = s > 0.f;
        // (a reciprocal needs s well above the smallest numbers; else the
        // quotient itself, limited, as its divisor has few bits)
        const bool tiny = s < 0x1p-100f;
        const float inv = 1.f / s;
        int8_t* q = a.q + row * a.q_stride;
        const auto store = [&](int u, uint32_t lo, uint32_t hi) {
            const int v = u * kRow + t;
            if (v < nv) *reinterpret_cast<uint2*>(q + v * 8) = make_uint2(lo, hi);
        };
        if (some && !tiny) {
            // (kMagic has 1 as its last place: adding it rounds to an integer,
            // ties to even, whose low byte is the sum's)
            constexpr float kMagic = 12582912.f;
            uint32_t w[V][2];
            float far = 0.f;
#pragma unroll
            for (int u = 0; u < V; ++u) {
                float f[8];
                raw[u].widen(f);
                uint32_t n[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float x = f[e] * inv, m = x + kMagic;
                    far = fmaxf(far, fabsf(x - (m - kMagic)));
                    n[e] = __float_as_uint(m);
                }
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    w[u][h] = __builtin_amdgcn_perm(
                        __builtin_amdgcn_perm(n[4 * h + 3], n[4 * h + 2], 0x0c0c0400),
                        __builtin_amdgcn_perm(n[4 * h + 1], n[4 * h], 0x0c0c0400), 0x05040100);
            }
            if (__ballot(far > 0.5f - 0x1p-14f) == 0) {
#pragma unroll
                for (int u = 0; u < V; ++u) store(u, w[u][0], w[u][1]);
                continue;
            }
        }
#pragma unroll
        for (int u = 0; u < V; ++u) {
            float f[8];
            raw[u].widen(f);
            uint32_t w[2] = {0, 0};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                int n = 0;
                if (some)
                    n = tiny ? (int)fminf(fmaxf((float)rint((double)f[e] / (double)s), -127.f),
                                          127.f)
                             : nearest(f[e], s, inv);
                w[e >> 2] |= (uint32_t)(n & 0xff) << (8 * (e & 3));
            }
            store(u, w[0], w[1]);
        }
    }
}

template <typename T, int Waves, int V>
hipError_t launch(const QuantizeArgs& a, hipStream_t s) {
    constexpr int kBlock = Waves > 4 ? 64 * Waves : kThreads, kRows = kBlock / (64 * Waves);
    const int64_t blocks = std::min<int64_t>((a.n + kRows - 1) / kRows, 1 << 20);
    quantize_kernel<T, Waves, V><<<(unsigned)blocks, kBlock, 0, s>>>(a);
    return hipGetLastError();
}

// A row's threads hold up to 32 elements each where there are rows for all waves,
// 8 where there are few and their latency counts (binary32 always: 32 take too many
// registers). At 2048 elements of bf16, 8 and 32 a thread: 11.6 and 14.3 us for 7000
// rows, 29 and 28 for 20,000, 131 and 122 for 100,000; of binary32 12.5 and 15.1, 34
// and 37 (20,000), 87 and 97 (50,000). At 8192 of bf16: 9.0 and 10.2 us for 1000, 26
// and 25 for 4000, 123 and 105 for 20,000.
template <typename T>
hipError_t quantize_of(const QuantizeArgs& a, hipStream_t s) {
    const int64_t all = a.n * a.width;
    if (a.width <= 512) return launch<T, 1, 1>(a, s);
    if (a.width <= 1024) return launch<T, 1, 2>(a, s);
    if (a.width <= 2048) {
        if constexpr (sizeof(T) == 2)
            if (all > int64_t(1) << 25) return launch<T, 1, 4>(a, s);
        return launch<T, 4, 1>(a, s);
    }
    if (a.width <= 8192)
        return all > int64_t(1) << 24 ? launch<T, 4, 4>(a, s) : launch<T, 16, 1>(a, s);
    if (a.width <= 32768) return launch<T, 16, 4>(a, s);
    return launch<T, 16, 8>(a, s);
}

}  // namespace

hipError_t launch_quantize_rows(const QuantizeArgs& a, p3d_dtype dt, hipStream_t s) {
    return dt == P3D_BF16 ? quantize_of<Bf16>(a, s) : quantize_of<float>(a, s);
}

}  // namespace p3d
