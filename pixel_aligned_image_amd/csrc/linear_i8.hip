// linear_i8.hip -- p3d_linear_i8: products of 8-bit integers on the matrix
// cores with the scales, bias, activation and residual in the epilogue.
//
//   out[i, d] = act((sum_k q[i, k] w[d, k]) s_i t_d + b_d) + r[i, d]
//
// Tiles of out features x tokens, the weights as the row operand of
// v_mfma_i32_32x32x32_i8 (a lane holds 16 neighbouring integers of one row,
// half l / 32 of 32) and the tokens as the column operand, so that a lane's
// results are neighbouring features of one token. K advances in chunks of 128
// integers: rows of 128 bytes in LDS, 16-byte slots swizzled so that 16 lanes
// reading one slot of 16 neighbouring rows meet every bank once.
#include "attn_tile.h"
#include "model_internal.h"

namespace p3d {

namespace {

using attn::dma16_from;
using attn::lds_offset;
using attn::tile_barrier;

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

constexpr int kThreads = 256;
constexpr int kStep = 128;                      // integers of K in a stage

__device__ __forceinline__ i32x16 mfma(i32x4 a, i32x4 b, i32x16 c) {
    return __builtin_amdgcn_mfma_i32_32x32x32_i8(a, b, c, 0, 0, 0);
}

// Eight neighbouring outputs of a token: scales, bias, activation, residual.
template <typename T, int Act>
struct Finish {
    float t[8], b[8];               // of the features

    __device__ __forceinline__ void load(const LinearArgs& a, int d) {
#pragma unroll
        for (int e = 0; e < 8; ++e) t[e] = a.weight_scale[d + e];
        if (a.bias) {
            read(a.bias, d, b);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) b[e] = 0.f;
        }
    }
    static __device__ __forceinline__ void read(const void* base, int64_t i, float (&f)[8]) {
        if constexpr (sizeof(T) == 2) {
            Vec<Bf16>::widen(*reinterpret_cast<const uint4*>(
                                 reinterpret_cast<const uint16_t*>(base) + i), f);
        } else {
            const float4* p = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(base) + i);
            const float4 x = p[0], y = p[1];
            f[0] = x.x; f[1] = x.y; f[2] = x.z; f[3] = x.w;
            f[4] = y.x; f[5] = y.y; f[6] = y.z; f[7] = y.w;
        }
    }
    __device__ __forceinline__ void write(const LinearArgs& a, int64_t token, int d, float s,
                                          float (&f)[8]) const {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = activate<Act>(f[e] * s * t[e] + b[e]);
        if (a.residual) {
            float r[8];
            read(a.residual, token * a.residual_stride + d, r);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] += r[e];
        }
        const int64_t to = token * a.out_stride + d;
        if constexpr (sizeof(T) == 2) {
            *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.out) + to) =
                Vec<Bf16>::narrow(f);
        } else {
            float4* p = reinterpret_cast<float4*>(reinterpret_cast<float*>(a.out) + to);
            p[0] = make_float4(f[0], f[1], f[2], f[3]);
            p[1] = make_float4(f[4], f[5], f[6], f[7]);
        }
    }
};

// ------------------------------------------------------------------ tiles ---
// Four waves, 2 x 2 of them, each BI x BJ blocks of 32 features x 32 tokens.
template <int BI, int BJ>
struct Shape {
    static constexpr int M = 64 * BI, N = 64 * BJ;              // features, tokens
    static constexpr int kStage = (M + N) * kStep;              // bytes
    static constexpr int kPitch = BI * 32 + 4;                  // floats of a staged token
    static constexpr int kStaged = 4 * 32 * kPitch * 4;
    static constexpr int kLds = 2 * kStage > kStaged ? 2 * kStage : kStaged;
};

__device__ __forceinline__ int swizzle(int row) { return (row >> 1) & 7; }

// Rows [0, Rows) of a tile from `base` on (rows past `last` repeat it; what they
// give is not stored), into LDS at `to`: a uniform base and a 32-bit offset a
// lane (rows are at most 2^22 bytes apart). Of a last chunk that K ends in only
// the `slots` that exist are loaded; `Zero` puts zeros into the others. (One
// operand's zeros are enough: integers have no NaN.) The lane number is opaque:
// offsets made ahead of the loop would take registers that the products need.
template <int Rows, bool Zero>
__device__ __forceinline__ void load_tile(const int8_t* base, int stride, int last, int slots,
                                          char* lds, int wave, int lane) {
    const uint32_t to = lds_offset(lds);
    asm volatile("" : "+v"(lane));
    const int slot = (lane & 7) ^ swizzle(wave * 8 + (lane >> 3));  // (of every row below)
    const auto offset = [&](int i) {
        return (uint32_t)(min((i * 4 + wave) * 8 + (lane >> 3), last) * stride + slot * 16);
    };
    if (slots >= 8) {
#pragma unroll
        for (int i = 0; i < Rows / 32; ++i)
            dma16_from(base, offset(i), to + (i * 4 + wave) * 8 * kStep);
        return;
    }
#pragma unroll 1
    for (int i = 0; i < Rows / 32; ++i) {
        const int r0 = (i * 4 + wave) * 8;
        if (slot < slots) dma16_from(base, offset(i), to + r0 * kStep);
        else if (Zero)
            reinterpret_cast<uint4*>(lds)[r0 * 8 + lane] = make_uint4(0, 0, 0, 0);
    }
}

typedef const __attribute__((address_space(3))) char lds_char;

__device__ __forceinline__ uint32_t frag_base(const char* tile, int row0, int lane) {
    const int r = lane & 31;
    uint32_t at = lds_offset(tile) + (row0 + r) * kStep + (((lane >> 5) ^ swizzle(r)) << 4);
    asm volatile("" : "+v"(at));
    return at;
}

template <int B>
__device__ __forceinline__ void read_frags(uint32_t base, int step, i32x4 (&f)[B]) {
    lds_char* p = (lds_char*)(uintptr_t)(base ^ (32 * step));
#pragma unroll
    for (int i = 0; i < B; ++i)
        f[i] = *(const __attribute__((address_space(3))) i32x4*)(p + i * 32 * kStep);
}

template <typename T, int Act, int BI, int BJ>
__global__ __launch_bounds__(kThreads, (BI * BJ > 8 ? 1 : 2)) void linear_kernel(
    LinearArgs a, int tiles_m, int tiles) {
    using S = Shape<BI, BJ>;
    extern __shared__ __align__(256) char lds[];    // (fragments reach a slot by an exclusive or)
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    // Workgroups go round the 8 dies: each die takes a run of tiles, features
    // fastest, so that a token tile is read into one die's L2 once.
    const int per = (tiles + 7) / 8;
    const int tile = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
    if (tile >= tiles || (int)(blockIdx.x >> 3) >= per) return;
    const int m0 = tile % tiles_m * S::M;
    const int64_t n0 = (int64_t)(tile / tiles_m) * S::N;
    const int last_m = a.out_dim - 1 - m0;
    const int last_n = a.n - n0 < S::N ? (int)(a.n - n0) - 1 : S::N - 1;
    const int8_t *wm0 = a.weight + (int64_t)m0 * a.in_dim, *qn0 = a.q + n0 * a.q_stride;
    const int stages = (a.in_dim + kStep - 1) / kStep;

    const auto load = [&](int st) {
        char* to = lds + (st & 1) * S::kStage;
        const int slots = (a.in_dim - st * kStep) / 16;
        load_tile<S::M, true>(wm0 + st * kStep, a.in_dim, last_m, slots, to, wave, lane);
        load_tile<S::N, false>(qn0 + st * kStep, (int)a.q_stride, last_n, slots, to + S::M * kStep,
                               wave, lane);
    };

    i32x16 acc[BI][BJ];
#pragma unroll
    for (int i = 0; i < BI; ++i)
#pragma unroll
        for (int j = 0; j < BJ; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;

    const int wm = (wave & 1) * BI * 32, wn = (wave >> 1) * BJ * 32;
    const uint32_t fa = frag_base(lds, wm, lane), fb = frag_base(lds + S::M * kStep, wn, lane);
    i32x4 fm[2][BI], fn[2][BJ];

    load(0);
    tile_barrier();
    read_frags<BI>(fa, 0, fm[0]);
    read_frags<BJ>(fb, 0, fn[0]);
    if (stages > 1) load(1);
    for (int st = 0; st < stages; ++st) {
        const uint32_t at = (st & 1) * S::kStage, other = S::kStage - at;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int cur = s & 1, nxt = cur ^ 1;
            if (s < 3) {
                read_frags<BI>(fa + at, s + 1, fm[nxt]);
                read_frags<BJ>(fb + at, s + 1, fn[nxt]);
            } else if (st + 1 < stages) {
                // The next stage has come, and every wave has its last
                // fragments of this one: its place is free.
                tile_barrier();
                read_frags<BI>(fa + other, 0, fm[nxt]);
                read_frags<BJ>(fb + other, 0, fn[nxt]);
                if (st + 2 < stages) load(st + 2);
            }
#pragma unroll
            for (int i = 0; i < BI; ++i)
#pragma unroll
                for (int j = 0; j < BJ; ++j)
                    acc[i][j] = mfma(fm[cur][i], fn[cur][j], acc[i][j]);
        }
    }
    tile_barrier();                     // the tiles' place is the epilogue's

    // A wave turns 32 tokens at a time in LDS, so that a token's features
    // leave in 16-byte pieces of whole rows.
    float* stage = reinterpret_cast<float*>(lds) + wave * 32 * S::kPitch;
    constexpr int kAcross = BI * 4, kDown = 64 / kAcross;       // lanes of a token, tokens at once
    const int d = m0 + wm + (lane % kAcross) * 8;
    Finish<T, Act> finish;
    if (d < a.out_dim) finish.load(a, d);
#pragma unroll
    for (int j = 0; j < BJ; ++j) {
#pragma unroll
        for (int i = 0; i < BI; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const i32x16& v = acc[i][j];
                *reinterpret_cast<float4*>(stage + (lane & 31) * S::kPitch + i * 32 + q * 8 +
                                           (lane >> 5) * 4) =
                    make_float4((float)v[4 * q], (float)v[4 * q + 1], (float)v[4 * q + 2],
                                (float)v[4 * q + 3]);
            }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll 2
        for (int r = lane / kAcross; r < 32; r += kDown) {
            const int64_t token = n0 + wn + j * 32 + r;
            const float* from = stage + r * S::kPitch + (lane % kAcross) * 8;
            const float4 x = *reinterpret_cast<const float4*>(from),
                         y = *reinterpret_cast<const float4*>(from + 4);
            float f[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
            if (token < a.n && d < a.out_dim) finish.write(a, token, d, a.scale[token], f);
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
}

// -------------------------------------------------------------- few tokens ---
// At most 16 B tokens: the weights are the traffic. 16 features a workgroup,
// its 8 waves a part of K each, fragments straight from memory (a weight is
// used once); the parts are added up as integers, in LDS.
constexpr int kFewWaves = 8, kFewSteps = 4;

template <typename T, int Act, int B>
__global__ __launch_bounds__(64 * kFewWaves) void linear_few_kernel(LinearArgs a) {
    __shared__ int part[kFewWaves][16 * B][16 + 1];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int row = lane & 15, d0 = blockIdx.x * 16;
    const int steps = (a.in_dim + 63) / 64;
    const int each = (steps + kFewWaves - 1) / kFewWaves;
    const int first = wave * each, end = first + each < steps ? first + each : steps;
    const int wd = d0 + row < a.out_dim ? d0 + row : a.out_dim - 1;
    const int8_t* w = a.weight + (int64_t)wd * a.in_dim + (lane >> 4) * 16;
    const int8_t* x[B];
    i32x4 acc[B];
#pragma unroll
    for (int b = 0; b < B; ++b) {
        const int64_t token = b * 16 + row;
        x[b] = a.q + (token < a.n ? token : a.n - 1) * a.q_stride + (lane >> 4) * 16;
        acc[b] = i32x4{0, 0, 0, 0};
    }
    const i32x4 zero = {0, 0, 0, 0};
    for (int k = first; k < end; k += kFewSteps) {
        i32x4 fw[kFewSteps], fx[kFewSteps][B];
#pragma unroll
        for (int u = 0; u < kFewSteps; ++u) {
            const int at = (k + u) * 64;
            const bool in = k + u < end && at + (lane >> 4) * 16 < a.in_dim;
            fw[u] = in ? *reinterpret_cast<const i32x4*>(w + at) : zero;
#pragma unroll
            for (int b = 0; b < B; ++b)
                fx[u][b] = in ? *reinterpret_cast<const i32x4*>(x[b] + at) : zero;
        }
#pragma unroll
        for (int u = 0; u < kFewSteps; ++u)
#pragma unroll
            for (int b = 0; b < B; ++b)
                acc[b] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[u], fx[u][b], acc[b], 0, 0, 0);
    }
    // (column lane % 16, a token; rows 4 (lane / 16) + r, features)
#pragma unroll
    for (int b = 0; b < B; ++b)
#pragma unroll
        for (int r = 0; r < 4; ++r) part[wave][b * 16 + row][(lane >> 4) * 4 + r] = acc[b][r];
    __syncthreads();
    for (int i = threadIdx.x; i < 16 * B * 2; i += 64 * kFewWaves) {
        const int token = i >> 1, d = (i & 1) * 8;
        if (token >= a.n || d0 + d >= a.out_dim) continue;
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            int s = 0;
#pragma unroll
            for (int k = 0; k < kFewWaves; ++k) s += part[k][token][d + e];
            f[e] = (float)s;
        }
        Finish<T, Act> finish;
        finish.load(a, d0 + d);
        finish.write(a, token, d0 + d, a.scale[token], f);
    }
}

// ----------------------------------------------------------------- launch ---
template <typename T, int Act, int BI, int BJ>
hipError_t tiles_of(const LinearArgs& a, hipStream_t s) {
    using S = Shape<BI, BJ>;
    const int64_t tiles_m = (a.out_dim + S::M - 1) / S::M, tiles_n = (a.n + S::N - 1) / S::N;
    const int64_t tiles = tiles_m * tiles_n;
    const unsigned grid = (unsigned)((tiles + 7) / 8 * 8);
    linear_kernel<T, Act, BI, BJ>
        <<<grid, kThreads, S::kLds, s>>>(a, (int)tiles_m, (int)tiles);
    return hipGetLastError();
}

template <typename T, int Act>
hipError_t linear_of(const LinearArgs& a, hipStream_t s) {
    const unsigned few = (unsigned)((a.out_dim + 15) / 16);
    if (a.n <= 16) linear_few_kernel<T, Act, 1><<<few, 64 * kFewWaves, 0, s>>>(a);
    else if (a.n <= 32) linear_few_kernel<T, Act, 2><<<few, 64 * kFewWaves, 0, s>>>(a);
    else if (a.n <= 64) linear_few_kernel<T, Act, 4><<<few, 64 * kFewWaves, 0, s>>>(a);
    else {
        const auto tiles = [&](int m) {
            return ((a.out_dim + m - 1) / m) * ((a.n + m - 1) / m);
        };
        if (tiles(256) >= kComputeUnits) return tiles_of<T, Act, 4, 4>(a, s);
        if (tiles(128) >= kComputeUnits / 2) return tiles_of<T, Act, 2, 2>(a, s);
        return tiles_of<T, Act, 1, 1>(a, s);
    }
    return hipGetLastError();
}

template <typename T>
hipError_t linear_act(const LinearArgs& a, hipStream_t s) {
    if (a.act == P3D_ACT_SILU) return linear_of<T, P3D_ACT_SILU>(a, s);
    if (a.act == P3D_ACT_GELU) return linear_of<T, P3D_ACT_GELU>(a, s);
    return linear_of<T, P3D_ACT_NONE>(a, s);
}

}  // namespace

hipError_t launch_linear_i8(const LinearArgs& a, p3d_dtype dt, hipStream_t s) {
    return dt == P3D_BF16 ? linear_act<Bf16>(a, s) : linear_act<float>(a, s);
}

}  // namespace p3d
