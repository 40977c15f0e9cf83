// adamw.hip -- p3d_adamw and p3d_grad_norm: the AdamW step over many tensors
// and the gradient norm it is clipped by.
//
//   m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2
//   w = w (1 - lr decay) - lr / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// One pass over the data: memory bound at 28 bytes an element (binary32
// weights and states) down to 10 (bf16 weights, 8-bit states): 217 us for 44
// million elements of 28 bytes, 5.7 TB/s, and 153 us for 88 million of 10, 5.9, where
// the vector units are as busy; the norm of 88 million bf16 gradients takes 30 us by
// itself and 47 after a step. The tensors' table travels in the kernel arguments,
// kTensors a launch; a workgroup takes one chunk of one tensor, which its lanes find
// among the tensors' first chunks, so that a launch over many small tensors fills
// the chip as a large one does.
//
// 8-bit states: a thread holds 8 neighbouring elements and 32 neighbouring
// threads a block of 256 that shares a scale, so a block's largest state is a
// maximum over half a wave and the states are read and written once.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "model_internal.h"

namespace p3d {

namespace {

constexpr int kThreads = 256, kPer = 8;             // elements of a thread, neighbours
constexpr int kTensors = 64;                        // of a launch: 5 KB of arguments
constexpr int64_t kChunk = (int64_t)kThreads * kPer;
constexpr int kNormLoads = 8;                       // 16 bytes each, of a thread and a chunk
constexpr int64_t kMaxGrid = int64_t(1) << 23;      // (a grid has fewer than 2^32 threads)

struct Entry {
    void* param;
    float* master;
    const void* grad;
    void *m, *v;
    float *m_scale, *v_scale;
    int64_t size;
    uint32_t key;               // of the tensor's random bits, or its number's share of it where
                                // t is the device's
    float keep;                 // 1 - lr decay, or decay where lr is the device's
};

struct Step {
    float b1, b2, c1, c2;       // c = 1 - b
    float rate;                 // lr / (1 - b1^t)
    float norm;                 // 1 / sqrt(1 - b2^t)
    float eps;                  // (these three times lift)
    int32_t count;
    double lift;
    double lr, log_b1, log_b2;  // (log2) where lr or t are the device's
    int64_t t;
    uint64_t seed;
    const float* grad_scale;
    const float* device_lr;
    const int32_t* device_step;
};

struct Table {
    Entry e[kTensors];
    uint32_t first[kTensors];   // chunk of the launch
};

// The last tensor whose chunks start at or before `chunk`: a lane looks at one
// (a search would wait for a load per step).
__device__ __forceinline__ int tensor_of(const Table& t, int count, uint32_t chunk) {
    static_assert(kTensors <= 64, "a lane a tensor");
    const int lane = threadIdx.x & 63;
    const uint64_t starts = __ballot(lane < count && t.first[lane < count ? lane : 0] <= chunk);
    return __builtin_amdgcn_readfirstlane(63 - __clzll((long long)starts));
}

__host__ __device__ __forceinline__ uint32_t mix(uint32_t x) {
    x ^= x >> 15;
    x *= 0xB504F335u;
    x ^= x >> 13;
    x *= 0xDDB3D743u;
    return x ^ (x >> 16);
}

// What a call's seed gives to its tensors' keys.
__host__ __device__ __forceinline__ uint32_t seed_key(uint64_t seed) {
    return mix((uint32_t)seed) ^ (uint32_t)(seed >> 32);
}

// ------------------------------------------------- vectors of 8 elements ---
__device__ __forceinline__ void widen8(const Bf16* p, float (&f)[8]) {
    Vec<Bf16>::widen(*reinterpret_cast<const uint4*>(p), f);
}
__device__ __forceinline__ void widen8(const float* p, float (&f)[8]) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}
// (past the caches: 231 us, not 252, where 44 million elements of 28 bytes stream by)
__device__ __forceinline__ void narrow8(Bf16* p, const float (&f)[8]) {
    store_nt16(p, Vec<Bf16>::narrow(f));
}
__device__ __forceinline__ void narrow8(float* p, const float (&f)[8]) {
    const float a[4] = {f[0], f[1], f[2], f[3]}, b[4] = {f[4], f[5], f[6], f[7]};
    store_nt16(p, Vec<float>::narrow(a));
    store_nt16(p + 4, Vec<float>::narrow(b));
}
__device__ __forceinline__ float widen1(Bf16 v) { return __uint_as_float((uint32_t)v.bits << 16); }
__device__ __forceinline__ float widen1(float v) { return v; }
__device__ __forceinline__ Bf16 narrow1(float f, Bf16) {
    return Bf16{(uint16_t)(pack_bf16x2(f, 0.f) & 0xffffu)};
}
__device__ __forceinline__ float narrow1(float f, float) { return f; }

// The `live` (0..8) elements from p on; zeros behind them.
template <typename T>
__device__ __forceinline__ void read8(const void* base, int64_t i, int live, float (&f)[8]) {
    const T* p = reinterpret_cast<const T*>(base) + i;
    if (live == 8) {
        widen8(p, f);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = e < live ? widen1(p[e]) : 0.f;
    }
}
template <typename T>
__device__ __forceinline__ void write8(void* base, int64_t i, int live, const float (&f)[8]) {
    T* p = reinterpret_cast<T*>(base) + i;
    if (live == 8) {
        narrow8(p, f);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < live) p[e] = narrow1(f[e], T{});
    }
}

__device__ __forceinline__ uint2 codes8(const void* base, int64_t i, int live) {
    const uint8_t* p = reinterpret_cast<const uint8_t*>(base) + i;
    if (live == 8) return *reinterpret_cast<const uint2*>(p);
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e < live) w[e >> 2] |= (uint32_t)p[e] << (8 * (e & 3));
    return make_uint2(w[0], w[1]);
}
__device__ __forceinline__ void write_codes8(void* base, int64_t i, int live, uint2 c) {
    uint8_t* p = reinterpret_cast<uint8_t*>(base) + i;
    if (live == 8) {
        *reinterpret_cast<uint2*>(p) = c;
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e < live) p[e] = (uint8_t)((e < 4 ? c.x : c.y) >> (8 * (e & 3)));
}

// e4m3 numbers as floats: the hardware's conversion, two at a time.
__device__ __forceinline__ void decode8(uint2 c, float by, float (&f)[8]) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    const f32x2 v[4] = {__builtin_amdgcn_cvt_pk_f32_fp8((int)c.x, false),
                        __builtin_amdgcn_cvt_pk_f32_fp8((int)c.x, true),
                        __builtin_amdgcn_cvt_pk_f32_fp8((int)c.y, false),
                        __builtin_amdgcn_cvt_pk_f32_fp8((int)c.y, true)};
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = v[e >> 1][e & 1] * by;
}

// The e4m3 number that the 16 random bits in `high`'s upper half choose of the
// two around q, limited to 448, into byte `At` of `word`: the hardware's
// conversion adds random bits 31 .. 12 to the 20 mantissa bits that it drops (a
// carry moves on to the next exponent as it should), below 2^-6 to the bits
// below 2^-9.
template <int At>
__device__ __forceinline__ uint32_t encode(float q, uint32_t high, uint32_t word) {
    return (uint32_t)__builtin_amdgcn_cvt_sr_fp8_f32(__builtin_amdgcn_fmed3f(q, -448.f, 448.f),
                                                     high, (int)word, At);
}

// The largest of 32 neighbouring lanes' numbers, in each of them. Magnitudes
// compare as their bits do: NaN is above infinity, and that above the rest.
__device__ __forceinline__ uint32_t half_max(uint32_t v) {
    const auto step = [&](float other) { v = max(v, __float_as_uint(other)); };
    step(dpp<0xB1>(__uint_as_float(v)));
    step(dpp<0x4E>(__uint_as_float(v)));
    step(dpp<0x141>(__uint_as_float(v)));
    step(dpp<0x140>(__uint_as_float(v)));
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    return max(r[0], r[1]);
}

// A block's scale, from its largest state, and what its states are multiplied
// by. A state that is not finite leaves a scale that is not.
__device__ __forceinline__ void block_scale(uint32_t largest, float& scale, float& by) {
    float top = __uint_as_float(largest);
    if (top < 0x1p-100f) top = 0.f;
    scale = top * (1.f / 448.f);
    by = top == 0.f ? 0.f : (1.f / top) * 448.f;
}

// The correctly rounded root of v in [2^-100, inf): a hardware reciprocal root,
// one step of its refinement, and the remainder's correction. (The compiler's
// own handles every number, in twice the operations.)
__device__ __forceinline__ float normal_root(float v) {
    const float y = __builtin_amdgcn_rsqf(v);
    float s = v * y, h = 0.5f * y;
    const float r = fmaf(-h, s, 0.5f);
    s = fmaf(s, r, s);
    h = fmaf(h, r, h);
    return fmaf(fmaf(-s, s, v), h, s);
}

// The states' update as the interface words it: one rounding an operation, so
// that states in 8 bits come out the same bit for bit wherever they are computed
// (a last place would move one in a million over a border).
__device__ __forceinline__ void moments(const Step& s, float x, float& m, float& v) {
#pragma clang fp contract(off)
    const float a = s.b1 * m, b = s.c1 * x;
    m = a + b;
    const float c = s.b2 * v, d = s.c2 * x;
    const float e = d * x;
    v = c + e;
}

template <typename P, typename G, bool Master, int Bits>
__global__ __launch_bounds__(kThreads) void adamw_kernel(Table table, Step s) {
    float by = 1.f;
    if (s.grad_scale) {
        by = *s.grad_scale;
        if (!(fabsf(by) < INFINITY)) return;
    }
    const int at = tensor_of(table, s.count, blockIdx.x);
    const Entry& t = table.e[at];
    float keep = t.keep;
    uint32_t key = t.key;
    if (s.device_lr || s.device_step) {
        // (1 - b^t with t log2 b: binary64 leaves 1 - 0.999 its 13 digits)
        const double lr = s.device_lr ? (double)*s.device_lr : s.lr;
        int64_t n = s.device_step ? (int64_t)*s.device_step : s.t;
        n = n < 1 ? 1 : n;
        keep = (float)(1. - lr * (double)t.keep);
        s.rate = (float)(s.lift * (lr / (1. - exp2((double)n * s.log_b1))));
        s.norm = (float)(s.lift * (1. / sqrt(1. - exp2((double)n * s.log_b2))));
        if (Bits == 8 && s.device_step) key = mix(key ^ seed_key(s.seed + (uint64_t)n));
    }
    const int64_t i = (int64_t)(blockIdx.x - table.first[at]) * kChunk + threadIdx.x * kPer;
    const int64_t left = t.size - i;
    const int live = left >= kPer ? kPer : left > 0 ? (int)left : 0;
    // (in 8 bits a wave stays whole: its lanes exchange the maximum)
    if (Bits == 32 ? live == 0 : __ballot(live > 0) == 0) return;
    float g[8], m[8], v[8], w[8];
    read8<G>(t.grad, i, live, g);
    if constexpr (Master) read8<float>(t.master, i, live, w);
    else read8<P>(t.param, i, live, w);
    if constexpr (Bits == 32) {
        read8<float>(t.m, i, live, m);
        read8<float>(t.v, i, live, v);
    } else {
        const uint2 cm = codes8(t.m, i, live), cv = codes8(t.v, i, live);
        const float sm = live ? t.m_scale[i >> 8] : 0.f, sv = live ? t.v_scale[i >> 8] : 0.f;
        decode8(cm, sm, m);
        decode8(cv, sv, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= v[e];
    }
    float root[8];
    if constexpr (Bits == 32) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float x = g[e] * by;
            m[e] = s.b1 * m[e] + s.c1 * x;
            v[e] = s.b2 * v[e] + s.c2 * x * x;
            root[e] = sqrtf(v[e]);
            w[e] = w[e] * keep - s.rate * m[e] / (root[e] * s.norm + s.eps);
        }
    } else {
        float least = INFINITY, most = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            moments(s, g[e] * by, m[e], v[e]);
            least = fminf(least, v[e]);
            most = fmaxf(most, v[e]);
        }
        // (a NaN, which these two pass over, stays one in either root)
        if (__ballot(least < 0x1p-100f || most == INFINITY) == 0) {
#pragma unroll
            for (int e = 0; e < 8; ++e) root[e] = normal_root(v[e]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) root[e] = sqrtf(v[e]);
        }
        // (the hardware's reciprocal takes and gives normal numbers: see `lift_of`)
#pragma unroll
        for (int e = 0; e < 8; ++e)
            w[e] = w[e] * keep -
                   s.rate * m[e] * __builtin_amdgcn_rcpf(root[e] * s.norm + s.eps);
    }
    if constexpr (Master) write8<float>(t.master, i, live, w);
    write8<P>(t.param, i, live, w);
    if constexpr (Bits == 32) {
        write8<float>(t.m, i, live, m);
        write8<float>(t.v, i, live, v);
    } else {
        uint32_t tm = 0, tv = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            tm = max(tm, __float_as_uint(m[e]) & 0x7fffffffu);
            tv = max(tv, __float_as_uint(root[e]) & 0x7fffffffu);
        }
        float sm, sv, bm, bv;
        block_scale(half_max(tm), sm, bm);
        block_scale(half_max(tv), sv, bv);
        uint32_t cm[2] = {0, 0}, cv[2] = {0, 0};
        const uint32_t base = (uint32_t)i * 0x9E3779B1u;
        const uint32_t high = (uint32_t)((uint64_t)i >> 32) * 0xDDB3D743u ^ key;
        const auto one = [&](auto at) {
            constexpr int e = decltype(at)::value;
            const uint32_t bits = mix((base + e * 0x9E3779B1u) ^ high);
            // a root that is not 0 is at least the smallest number
            float q = root[e] * bv;
            q = q > 0.f ? fmaxf(q, 0x1p-9f) : q;
            cm[e >> 2] = encode<(e & 3)>(m[e] * bm, bits << 16, cm[e >> 2]);
            cv[e >> 2] = encode<(e & 3)>(q, bits & 0xffff0000u, cv[e >> 2]);
        };
        one(std::integral_constant<int, 0>());
        one(std::integral_constant<int, 1>());
        one(std::integral_constant<int, 2>());
        one(std::integral_constant<int, 3>());
        one(std::integral_constant<int, 4>());
        one(std::integral_constant<int, 5>());
        one(std::integral_constant<int, 6>());
        one(std::integral_constant<int, 7>());
        write_codes8(t.m, i, live, make_uint2(cm[0], cm[1]));
        write_codes8(t.v, i, live, make_uint2(cv[0], cv[1]));
        if ((threadIdx.x & 31) == 0 && live) {
            t.m_scale[i >> 8] = sm;
            t.v_scale[i >> 8] = sv;
        }
    }
}

// ------------------------------------------------------------------- norm ---

// At most kNormGrid workgroups a launch take its chunks in turn, a chunk's loads
// all on their way before the first is used. Squares and sums are binary64, so
// that no gradient's square leaves the numbers.
constexpr int64_t kNormGrid = 6 * kComputeUnits;
constexpr int64_t norm_chunk(p3d_dtype dt) {
    return (int64_t)kThreads * kNormLoads * (dt == P3D_BF16 ? 8 : 4);
}

template <typename G>
__global__ __launch_bounds__(kThreads) void norm_parts_kernel(Table table, int count,
                                                              uint32_t chunks,
                                                              double* __restrict__ parts) {
    constexpr int N = Vec<G>::N;
    constexpr int64_t kAll = (int64_t)kThreads * kNormLoads * N;
    __shared__ double wave[kThreads / 64];
    double sums[4] = {0., 0., 0., 0.};
    const auto add = [&](uint4 q) {
        float g[N];
        Vec<G>::widen(q, g);
#pragma unroll
        for (int e = 0; e < N; ++e) sums[e & 3] = fma((double)g[e], (double)g[e], sums[e & 3]);
    };
    for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
        const int at = tensor_of(table, count, c);
        const Entry& t = table.e[at];
        const int64_t i0 = (int64_t)(c - table.first[at]) * kAll;
        const G* g = reinterpret_cast<const G*>(t.grad);
        if (t.size - i0 >= kAll) {
            const uint4* p = reinterpret_cast<const uint4*>(g + i0) + threadIdx.x;
            uint4 q[kNormLoads];
#pragma unroll
            for (int r = 0; r < kNormLoads; ++r) q[r] = p[r * kThreads];
#pragma unroll
            for (int r = 0; r < kNormLoads; ++r) add(q[r]);
            continue;
        }
        for (int64_t i = i0 + threadIdx.x * N; i < t.size; i += (int64_t)kThreads * N) {
            if (t.size - i >= N) {
                add(*reinterpret_cast<const uint4*>(g + i));
            } else {
                for (int64_t k = i; k < t.size; ++k) {
                    const double x = (double)widen1(g[k]);
                    sums[0] = fma(x, x, sums[0]);
                }
            }
        }
    }
    double sum = (sums[0] + sums[1]) + (sums[2] + sums[3]);
    for (int off = 1; off < 64; off <<= 1) sum += __shfl_xor(sum, off);
    if ((threadIdx.x & 63) == 0) wave[threadIdx.x >> 6] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        sum = 0.;
        for (int k = 0; k < kThreads / 64; ++k) sum += wave[k];
        parts[blockIdx.x] = sum;
    }
}

__global__ __launch_bounds__(1024) void norm_join_kernel(const double* __restrict__ parts,
                                                         int64_t n, float max_norm,
                                                         float* __restrict__ out) {
    __shared__ double wave[16];
    double sum = 0.;
#pragma unroll 8
    for (int64_t i = threadIdx.x; i < n; i += 1024) sum += parts[i];
    for (int off = 1; off < 64; off <<= 1) sum += __shfl_xor(sum, off);
    if ((threadIdx.x & 63) == 0) wave[threadIdx.x >> 6] = sum;
    __syncthreads();
    if (threadIdx.x) return;
    sum = 0.;
    for (int k = 0; k < 16; ++k) sum += wave[k];
    const double norm = sqrt(sum);
    out[0] = (float)norm;
    // (finite as out[0] has it: the two say the same of a norm beyond binary32)
    out[1] = !(out[0] < INFINITY) ? NAN
             : norm > (double)max_norm ? (float)((double)max_norm / norm) : 1.f;
}

// ----------------------------------------------------------------- launch ---
// The tensors in launches of at most kTensors, numbered from `chunk` elements
// on: `run(table, count, chunks)` for each. A tensor's own chunks fit a grid by
// its size's limit.
template <typename Run>
hipError_t in_launches(const p3d_adamw_desc& d, int64_t chunk, Run run) {
    Table t;
    int count = 0;
    int64_t chunks = 0;
    const auto flush = [&]() {
        if (chunks == 0) {
            count = 0;
            return hipSuccess;
        }
        const hipError_t e = run(t, count, chunks);
        count = 0;
        chunks = 0;
        return e;
    };
    const uint32_t key = seed_key(d.seed);
    for (int32_t j = 0; j < d.count; ++j) {
        const p3d_adamw_tensor& x = d.tensors[j];
        if (x.size == 0) continue;
        const int64_t more = (x.size + chunk - 1) / chunk;
        if (count == kTensors || chunks + more > kMaxGrid) {
            const hipError_t e = flush();
            if (e != hipSuccess) return e;
        }
        t.first[count] = (uint32_t)chunks;
        Entry& to = t.e[count++];
        to.param = x.param;
        to.master = x.master;
        to.grad = x.grad;
        to.m = x.m;
        to.v = x.v;
        to.m_scale = x.m_scale;
        to.v_scale = x.v_scale;
        to.size = x.size;
        to.key = (uint32_t)j * 0x9E3779B1u;
        if (!d.device_step) to.key = mix(to.key ^ key);
        to.keep = d.device_lr || d.device_step ? x.weight_decay
                                               : (float)(1. - d.lr * (double)x.weight_decay);
        chunks += more;
    }
    return flush();
}

template <typename P, typename G, bool Master>
hipError_t adamw_bits(const p3d_adamw_desc& d, const Step& step, hipStream_t s) {
    return in_launches(d, kChunk, [&](const Table& t, int count, int64_t chunks) {
        Step here = step;
        here.count = count;
        if (d.state_bits == 8)
            adamw_kernel<P, G, Master, 8><<<(unsigned)chunks, kThreads, 0, s>>>(t, here);
        else
            adamw_kernel<P, G, Master, 32><<<(unsigned)chunks, kThreads, 0, s>>>(t, here);
        return hipGetLastError();
    });
}

template <typename G>
hipError_t adamw_grad(const p3d_adamw_desc& d, const Step& step, bool master, hipStream_t s) {
    if (d.param_dtype == P3D_F32) return adamw_bits<float, G, false>(d, step, s);
    return master ? adamw_bits<Bf16, G, true>(d, step, s) : adamw_bits<Bf16, G, false>(d, step, s);
}

// What the update's factor, the root's and eps are multiplied by, a power of two, so
// that the hardware's reciprocal serves every eps that binary32 holds: of a number
// below 2^-126 it gives infinity (and 0 times that is NaN, where an element without a
// gradient has nothing to divide), of one above 2^126 0. Denominators lie between eps
// and eps + 2^91, as a root is below 2^64 and its factor below 2^27. 32-bit states
// are divided.
double lift_of(const p3d_adamw_desc& d) {
    if (d.state_bits != 8) return 1.;
    return d.eps < 0x1p-126 ? 0x1p24 : d.eps > 0x1p100 ? 0x1p-64 : 1.;
}

}  // namespace

// (a launch's chunks, of which it has at most kNormGrid parts, in as many
// launches as the table takes; more would be room for nothing)
int64_t grad_norm_parts(const p3d_adamw_desc& d) {
    int64_t n = 0;
    (void)in_launches(d, norm_chunk(d.grad_dtype), [&](const Table&, int, int64_t chunks) {
        n += std::min(chunks, kNormGrid);
        return hipSuccess;
    });
    return n;
}

hipError_t launch_grad_norm(const p3d_adamw_desc& d, float max_norm, float* out, double* parts,
                            hipStream_t s) {
    int64_t at = 0;
    const int64_t chunk = norm_chunk(d.grad_dtype);
    const hipError_t e = in_launches(d, chunk, [&](const Table& t, int count, int64_t chunks) {
        const int64_t grid = std::min(chunks, kNormGrid);
        if (d.grad_dtype == P3D_BF16)
            norm_parts_kernel<Bf16>
                <<<(unsigned)grid, kThreads, 0, s>>>(t, count, (uint32_t)chunks, parts + at);
        else
            norm_parts_kernel<float>
                <<<(unsigned)grid, kThreads, 0, s>>>(t, count, (uint32_t)chunks, parts + at);
        at += grid;
        return hipGetLastError();
    });
    if (e != hipSuccess) return e;
    norm_join_kernel<<<1, 1024, 0, s>>>(parts, at, max_norm, out);
    return hipGetLastError();
}

hipError_t launch_adamw(const p3d_adamw_desc& d, hipStream_t s) {
    bool master = false;
    for (int32_t j = 0; j < d.count; ++j) master = master || d.tensors[j].master;
    Step step{};
    step.b1 = (float)d.beta1;
    step.b2 = (float)d.beta2;
    step.c1 = (float)(1. - d.beta1);
    step.c2 = (float)(1. - d.beta2);
    step.lift = lift_of(d);
    step.rate = (float)(step.lift * (d.lr / (1. - std::pow(d.beta1, (double)d.step))));
    step.norm = (float)(step.lift * (1. / std::sqrt(1. - std::pow(d.beta2, (double)d.step))));
    step.eps = (float)(step.lift * d.eps);
    step.lr = d.lr;
    step.log_b1 = std::log2(d.beta1);
    step.log_b2 = std::log2(d.beta2);
    step.t = d.step;
    step.seed = d.seed;
    step.grad_scale = d.grad_scale;
    step.device_lr = d.device_lr;
    step.device_step = d.device_step;
    return d.grad_dtype == P3D_BF16 ? adamw_grad<Bf16>(d, step, master, s)
                                    : adamw_grad<float>(d, step, master, s);
}

}  // namespace p3d
