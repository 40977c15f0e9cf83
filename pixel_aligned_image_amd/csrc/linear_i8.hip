// linear_i8.hip -- p3d_linear_i8: products of 8-bit integers on the matrix
// cores with the scales, bias, activation and residual in the epilogue.
//
//   out[i, d] = act((sum_k q[i, k] w[d, k]) s_i t_d + b_d) + r[i, d]
//
// Tiles of out features x tokens, the weights as the row operand of
// v_mfma_i32_32x32x32_i8 (a lane holds 16 neighbouring integers of one row,
// half l / 32 of 32) and the tokens as the column operand, so that a lane's
// results are neighbouring features of one token. K advances in stages of 64
// integers, four of them in LDS: while one is multiplied the next has arrived
// and two more are on their way, which covers the memory's latency with one
// workgroup on a CU. Measured: 100,000 x 2048 x 1536 in 323 to 333 us,
// 1.9 PFLOP/s, 12,289 x 1536 x 6144 in 134 us, 1.73, and with GELU in 154 (a
// library's bare products: 1.72 to 1.83 and 1.52 to 1.61). The clock is 1.9 GHz under
// this load, the matrix cores are busy 48 % of the time (in the library's product 45)
// and the waves stand at waits for 36: which of these bounds it is not shown.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "attn_tile.h"
#include "model_internal.h"

namespace p3d {

namespace {

using attn::dma16_from;
using attn::lds_offset;
using attn::tile_barrier;

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

constexpr int kStep = 64, kSlots = kStep / 16;  // integers and 16-byte slots of a row in a stage
constexpr int kStages = 4;                      // in LDS

__device__ __forceinline__ i32x16 mfma(i32x4 a, i32x4 b, i32x16 c) {
    return __builtin_amdgcn_mfma_i32_32x32x32_i8(a, b, c, 0, 0, 0);
}

// Eight neighbouring numbers of a row as they lie.
template <typename T>
struct Eight {
    uint4 v[sizeof(T) / 2];

    __device__ __forceinline__ void load(const void* base, int64_t i) {
        const uint4* p = reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(base) +
                                                        i * (int64_t)sizeof(T));
#pragma unroll
        for (int k = 0; k < (int)sizeof(T) / 2; ++k) v[k] = p[k];
    }
    __device__ __forceinline__ void widen(float (&f)[8]) const {
        if constexpr (sizeof(T) == 2) {
            Vec<Bf16>::widen(v[0], f);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint4& q = v[e >> 2];
                f[e] = __uint_as_float((e & 3) == 0 ? q.x : (e & 3) == 1 ? q.y
                                                        : (e & 3) == 2 ? q.z : q.w);
            }
        }
    }
};

// Eight neighbouring outputs of a token: scales, bias, activation, residual.
template <typename T, int Act>
struct Finish {
    float t[8], b[8];               // of the features

    __device__ __forceinline__ void load(const LinearArgs& a, int d) {
#pragma unroll
        for (int e = 0; e < 8; ++e) t[e] = a.weight_scale[d + e];
        if (a.bias) {
            Eight<T> q;
            q.load(a.bias, d);
            q.widen(b);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) b[e] = 0.f;
        }
    }
    // (f: the sums times the token's scale)
    template <bool Res>
    __device__ __forceinline__ void write(const LinearArgs& a, int64_t token, int d,
                                          const Eight<T>& residual, float (&f)[8]) const {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = activate<Act>(f[e] * t[e] + b[e]);
        if constexpr (Res) {
            float r[8];
            residual.widen(r);
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
// WM x WN waves, each BI x BJ blocks of 32 features x 32 tokens.
template <int BI_, int BJ_, int WM_, int WN_>
struct Shape {
    static constexpr int BI = BI_, BJ = BJ_, WM = WM_, kWaves = WM_ * WN_, kThreads = 64 * kWaves;
    static constexpr int M = WM_ * BI * 32, N = WN_ * BJ * 32;  // features, tokens
    // Loads of a wave and a stage, 16 rows each, the same number for every wave:
    // rows past the tile's repeat its last one and are not read.
    static constexpr int kRound = 16 * kWaves;
    static constexpr int LM = (M + kRound - 1) / kRound, LN = (N + kRound - 1) / kRound;
    static constexpr int kRowsM = LM * kRound, kStage = (kRowsM + LN * kRound) * kStep;  // bytes
    // The epilogue turns kTurn blocks of features at a time, behind the first two
    // stages' place.
    static constexpr int kTurn = BI % 2 ? 1 : 2, kPitch = kTurn * 32 + 4;   // floats of a token
    static constexpr int kTurned = 2 * kStage + kWaves * 32 * kPitch * 4;
    static constexpr int kLds = kStages * kStage > kTurned ? kStages * kStage : kTurned;
    static constexpr int kPerCu = 160 * 1024 / kLds;            // workgroups
};

// Slot c of row r of a stage sits at c ^ swizzle(r): 16 lanes that read one
// slot of 16 neighbouring rows (64 bytes each) meet every bank once.
__device__ __forceinline__ int swizzle(int row) { return (row >> 2) & (kSlots - 1); }

typedef const __attribute__((address_space(3))) char lds_char;

// 16 bytes of LDS from `at`, a register, and a constant distance on.
__device__ __forceinline__ i32x4 read_frag(uint32_t at, int on) {
    return *(const __attribute__((address_space(3))) i32x4*)((lds_char*)(uintptr_t)at + on);
}

// The order of a stage's instructions is the source's: the fragments and loads
// of what comes next stand between the products, one at a time.
__device__ __forceinline__ void pin() { __builtin_amdgcn_sched_barrier(0); }

__device__ __forceinline__ void meet() { asm volatile("s_barrier" ::: "memory"); }

// A workgroup takes tiles in turn. The next tile's first two stages are on their
// way while this one's results are turned and stored, which hides the memory's
// latency at a tile's start and its own stores. With a residual (Res), that of a
// turn is loaded as the turn before is stored, in the registers that its half of
// the features' scales and biases leave: 381 us for 100,000 x 2048 x 1536, 429 where
// it was loaded as it was added, 330 without one. (The same code for both kept those
// registers from the stages: 346 us without one.)
template <typename T, int Act, bool Res, typename S>
__global__ __launch_bounds__(S::kThreads, 2) void linear_kernel(LinearArgs a, int tiles_m,
                                                               int tiles) {
    constexpr int BI = S::BI, BJ = S::BJ, LM = S::LM, LN = S::LN, kLoads = LM + LN;
    extern __shared__ __align__(256) char lds[];    // (fragments reach a slot by an exclusive or)
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    // Workgroups go round the 8 dies: each die takes a run of tiles, features
    // fastest, so that a token tile is read into one die's L2 once; in bands of at
    // most 8 feature tiles, whose weights stay there meanwhile (12,289 x 1536 x 6144:
    // 143 us without bands, 135 with).
    const int per = (tiles + 7) / 8, turn = gridDim.x >> 3;
    const int first = (blockIdx.x & 7) * per, end = min(first + per, tiles);
    int tile = first + (blockIdx.x >> 3);
    if (tile >= end) return;
    const int tiles_n = tiles / tiles_m, bands = (tiles_m + 7) / 8;
    const int wide = (tiles_m + bands - 1) / bands;
    const int stages = (a.in_dim + kStep - 1) / kStep;

    // Loads: 16 rows an instruction, a uniform base and a 32-bit offset a lane
    // (rows are at most 2^22 bytes apart). Rows past the last repeat it; what
    // they give is not stored. Slots past K, in the last stage, repeat the
    // row's first there; the weights' fragments of those are cleared.
    const int row = wave * 16 + (lane >> 2), slot = (lane & 3) ^ swizzle(row);
    const int last_slots = (a.in_dim - (stages - 1) * kStep) / 16;
    const int back = slot < last_slots ? 0 : slot * 16;
    int m0, off_m[LM], off_n[LN];
    int64_t n0;
    const int8_t *wm0, *qn0;
    const auto begin = [&](int t) {
        const int band = t / (wide * tiles_n), in = t - band * wide * tiles_n;
        const int width = min(wide, tiles_m - band * wide), down = in / width;
        m0 = (band * wide + in - down * width) * S::M;
        n0 = (int64_t)down * S::N;
        wm0 = a.weight + (int64_t)m0 * a.in_dim;
        qn0 = a.q + n0 * a.q_stride;
        const int last_m = min(a.out_dim - m0, S::M) - 1;
        const int last_n = a.n - n0 < S::N ? (int)(a.n - n0) - 1 : S::N - 1;
#pragma unroll
        for (int i = 0; i < LM; ++i)
            off_m[i] = min(i * S::kRound + row, last_m) * a.in_dim + slot * 16;
#pragma unroll
        for (int j = 0; j < LN; ++j)
            off_n[j] = min(j * S::kRound + row, last_n) * (int)a.q_stride + slot * 16;
    };
    const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_offset(lds)) + wave * 16 * kStep;
    // load `l` (0 .. kLoads) of this wave's share of stage st
    const auto load = [&](int st, int l) {
        const uint32_t to = lds0 + (st & (kStages - 1)) * S::kStage + l * S::kRound * kStep;
        if (l < LM) dma16_from(wm0 + st * kStep, off_m[l < LM ? l : 0], to);
        else dma16_from(qn0 + st * kStep, off_n[l < LM ? 0 : l - LM], to);
    };
    const auto before_load = [&](int st) {
        if (st == stages - 1) {
#pragma unroll
            for (int i = 0; i < LM; ++i) off_m[i] -= back;
#pragma unroll
            for (int j = 0; j < LN; ++j) off_n[j] -= back;
        }
    };
    const auto load_stage = [&](int st) {
        if (st >= stages) return;
        before_load(st);
#pragma unroll
        for (int l = 0; l < kLoads; ++l) load(st, l);
    };

    i32x16 acc[BI][BJ];
    const int wm = wave % S::WM * BI * 32, wn = wave / S::WM * BJ * 32;
    const int r32 = lane & 31;
    uint32_t at = ((lane >> 5) ^ swizzle(r32)) << 4;
    at += lds_offset(lds) + r32 * kStep;
    const uint32_t fa = at + wm * kStep, fb = at + (S::kRowsM + wn) * kStep;
    i32x4 fm[2][BI], fn[2][BJ];
    // where step s of stage st has this lane's fragments; fragment f of it
    struct Place { uint32_t m, n; };
    const auto place = [&](int st, int s) {
        const uint32_t stage = (st & (kStages - 1)) * S::kStage;
        Place p{(fa ^ (32 * s)) + stage, (fb ^ (32 * s)) + stage};
        asm volatile("" : "+v"(p.m), "+v"(p.n));
        return p;
    };
    const auto read = [&](const Place& p, int s, int f) {
        if (f < BI) fm[s][f < BI ? f : 0] = read_frag(p.m, f * 32 * kStep);
        else fn[s][f < BI ? 0 : f - BI] = read_frag(p.n, (f - BI) * 32 * kStep);
    };
    const auto clear = [&](int s) {                 // what lies past K
        if (2 * s + (lane >> 5) >= last_slots)
#pragma unroll
            for (int i = 0; i < BI; ++i) fm[s][i] = i32x4{0, 0, 0, 0};
    };

    // A stage: two steps of 32. `flying`: later stages' loads that stay on
    // their way when the next one has to be there.
    constexpr int kProducts = BI * BJ, kFrags = BI + BJ;
    const auto stage = [&](int st, auto flying, auto loads, auto next) {
        constexpr bool kLoad = decltype(loads)::value, kNext = decltype(next)::value;
        if constexpr (!kNext) clear(0);
        if constexpr (kLoad) before_load(st + kStages);
        const Place here = place(st, 1), then = place(st + 1, 0);
#pragma unroll
        for (int p = 0, f = 0; p < kProducts; ++p) {
            acc[p / BJ][p % BJ] = mfma(fm[0][p / BJ], fn[0][p % BJ], acc[p / BJ][p % BJ]);
#pragma unroll
            for (; f < kFrags && f * kProducts < (p + 1) * 2 * kFrags; ++f) read(here, 1, f);
            pin();
        }
        // Every wave has its fragments of this stage, so its place is free, and
        // the next stage has come.
        if constexpr (kNext) {
            attn::wave_wait<decltype(flying)::value * kLoads>();
            meet();
        } else {
            clear(1);
        }
        pin();
#pragma unroll
        for (int p = 0, f = 0, l = 0; p < kProducts; ++p) {
            acc[p / BJ][p % BJ] = mfma(fm[1][p / BJ], fn[1][p % BJ], acc[p / BJ][p % BJ]);
            if constexpr (kNext) {
#pragma unroll
                for (; f < kFrags && f * kProducts < (p + 1) * 2 * kFrags; ++f) read(then, 0, f);
            }
            if constexpr (kLoad) {
#pragma unroll
                for (; l < kLoads && l * kProducts < (2 * p + 2 - kProducts) * kLoads; ++l)
                    load(st + kStages, l);
            }
            pin();
        }
    };
    using std::integral_constant;
    using Yes = std::true_type;
    using No = std::false_type;

    // The epilogue: lanes of a token, tokens at once, turns of the features.
    constexpr int kAcross = S::kTurn * 4, kDown = 64 / kAcross, kTurns = BI / S::kTurn;
    constexpr int kRows = 32 / kDown;               // tokens of a lane in a turn
    const auto turn_h = [](int u) { return Res ? u / BJ : u % kTurns; };
    const auto turn_j = [](int u) { return Res ? u % BJ : u / kTurns; };
    float* turned = reinterpret_cast<float*>(lds + 2 * S::kStage) + wave * 32 * S::kPitch;

    begin(tile);
    load_stage(0);
    load_stage(1);
    for (;;) {
        // What the epilogue needs (first): the scales of the lane's tokens, and those of
        // eight of its features in every turn.
        const int d0 = m0 + wm + (lane % kAcross) * 8;
        const int64_t token0 = n0 + wn;
        Finish<T, Act> finish[kTurns];
#pragma unroll
        for (int h = 0; h < (Res ? 1 : kTurns); ++h)
            if (d0 + h * S::kTurn * 32 < a.out_dim) finish[h].load(a, d0 + h * S::kTurn * 32);
        float scale[BJ];
#pragma unroll
        for (int j = 0; j < BJ; ++j) {
            const int64_t token = token0 + j * 32 + r32;
            scale[j] = a.scale[token < a.n ? token : a.n - 1];
        }
        load_stage(2);
        load_stage(3);
#pragma unroll
        for (int i = 0; i < BI; ++i)
#pragma unroll
            for (int j = 0; j < BJ; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;
        // (older than the last two stages' loads: the first two's, the tile
        // before's stores and the scales)
        if (stages >= 4) attn::wave_wait<2 * kLoads>();
        else attn::wave_wait<0>();
        meet();
#pragma unroll
        for (int f = 0; f < kFrags; ++f) read(place(0, 0), 0, f);
        int st = 0;
        for (; st + kStages < stages; ++st) stage(st, integral_constant<int, 2>(), Yes(), Yes());
        if (stages - st >= 4) stage(st++, integral_constant<int, 2>(), No(), Yes());
        if (stages - st >= 3) stage(st++, integral_constant<int, 1>(), No(), Yes());
        if (stages - st >= 2) stage(st++, integral_constant<int, 0>(), No(), Yes());
        stage(st, integral_constant<int, 0>(), No(), No());
        // (loads of every lane, kept inside the tensor: what a lane left out would be a
        // register to keep)
        Eight<T> residual[kRows];
        const auto fetch = [&](int u, int k) {
            const int d = min(d0 + turn_h(u) * S::kTurn * 32, a.out_dim - 8);
            const int64_t token = token0 + turn_j(u) * 32 + lane / kAcross + k * kDown;
            residual[k].load(a.residual,
                             (token < a.n ? token : a.n - 1) * a.residual_stride + d);
        };
        if constexpr (Res) {
#pragma unroll
            for (int k = 0; k < kRows; ++k) fetch(0, k);
#pragma unroll
            for (int h = 1; h < kTurns; ++h)
                finish[h].load(a, min(d0 + h * S::kTurn * 32, a.out_dim - 8));
        }
        tile_barrier();                 // nothing reads or writes the stages now

        tile += turn;
        const bool more = tile < end;
        if (more) {
            begin(tile);
            load_stage(0);
            load_stage(1);
        }
        // A wave turns 32 tokens and kTurn blocks of features at a time in LDS, so
        // that a token's features leave in 16-byte pieces of whole lines.
#pragma unroll
        for (int u = 0; u < kTurns * BJ; ++u) {
            const int h = turn_h(u), j = turn_j(u);
#pragma unroll
            for (int i = 0; i < S::kTurn; ++i)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const i32x16& v = acc[h * S::kTurn + i][j];
                    *reinterpret_cast<float4*>(turned + r32 * S::kPitch + i * 32 + q * 8 +
                                               (lane >> 5) * 4) =
                        make_float4((float)v[4 * q] * scale[j], (float)v[4 * q + 1] * scale[j],
                                    (float)v[4 * q + 2] * scale[j],
                                    (float)v[4 * q + 3] * scale[j]);
                }
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            const int d = d0 + h * S::kTurn * 32;
#pragma unroll
            for (int k = 0; k < kRows; ++k) {
                const int r = lane / kAcross + k * kDown;
                const int64_t token = token0 + j * 32 + r;
                const float* from = turned + r * S::kPitch + (lane % kAcross) * 8;
                const float4 x = *reinterpret_cast<const float4*>(from),
                             y = *reinterpret_cast<const float4*>(from + 4);
                float f[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
                if (token < a.n && d < a.out_dim)
                    finish[h].template write<Res>(a, token, d, residual[k], f);
                if constexpr (Res)
                    if (u + 1 < kTurns * BJ) fetch(u + 1, k);
            }
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        }
        if (!more) return;
        meet();                         // the turned tile's place is the stages' again
    }
}

// -------------------------------------------------------------- few tokens ---
// At most 16 B tokens: the weights are the traffic. 16 features a workgroup,
// its 8 waves a part of K each, fragments straight from memory (a weight is
// used once); the parts are added up as integers, in LDS. 5 and 16 tokens of 6144
// features to 1536 take 8.1 us (with the host's part), in tiles 18.6, 64 tokens
// 16.2 and 19.8; where K is short the host's part is all there is of either.
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
            f[e] = (float)s * a.scale[token];
        }
        Finish<T, Act> finish;
        finish.load(a, d0 + d);
        Eight<T> residual;
        if (a.residual) {
            residual.load(a.residual, token * a.residual_stride + d0 + d);
            finish.template write<true>(a, token, d0 + d, residual, f);
        } else {
            finish.template write<false>(a, token, d0 + d, residual, f);
        }
    }
}

// ----------------------------------------------------------------- launch ---
template <typename S>
int64_t tiles_in(const LinearArgs& a) {
    return ((a.out_dim + S::M - 1) / S::M) * ((a.n + S::N - 1) / S::N);
}

template <typename T, int Act, typename S, bool Added = true>
hipError_t tiles_of(const LinearArgs& a, hipStream_t s) {
    const int64_t tiles = tiles_in<S>(a);
    const int64_t grid = std::min<int64_t>((tiles + 7) / 8 * 8, S::kPerCu * kComputeUnits);
    const int tiles_m = (a.out_dim + S::M - 1) / S::M;
    if constexpr (Added)
        if (a.residual) {
            linear_kernel<T, Act, true, S>
                <<<(unsigned)grid, S::kThreads, S::kLds, s>>>(a, tiles_m, (int)tiles);
            return hipGetLastError();
        }
    linear_kernel<T, Act, false, S>
        <<<(unsigned)grid, S::kThreads, S::kLds, s>>>(a, tiles_m, (int)tiles);
    return hipGetLastError();
}

template <typename T, int Act>
hipError_t linear_of(const LinearArgs& a, hipStream_t s) {
    const unsigned few = (unsigned)((a.out_dim + 15) / 16);
    const bool fits = few <= (1u << 22);            // (a grid has fewer than 2^32 threads)
    if (fits && a.n <= 16) linear_few_kernel<T, Act, 1><<<few, 64 * kFewWaves, 0, s>>>(a);
    else if (fits && a.n <= 32) linear_few_kernel<T, Act, 2><<<few, 64 * kFewWaves, 0, s>>>(a);
    else if (fits && a.n <= 64) linear_few_kernel<T, Act, 4><<<few, 64 * kFewWaves, 0, s>>>(a);
    else {
        // Rounds of tiles over the chip, times a round's length: us where K is 2048,
        // of a full round and of one with a tile or two (what is left of a round runs
        // at a higher clock). Measured: 27 us in B and 29 to 41 in the others for
        // 7000 x 2048 x 1536, 49 in B and 54 to 67 for 12,289, 66 in A and 76 to 97
        // for 20,000, 12 in D and 13 to 24 for 1500, 8.7 in E and 10 to 22 for 300.
        // The lengths' ratios hardly change with K (1024 and 6144 choose alike). C not
        // with a residual, whose first loads a tile of so few columns does not cover:
        // 19 us without one and 23.4 with it, D 20.6 and 21.8 (4000 x 2048 x 1536).
        using A = Shape<4, 2, 2, 4>;        // 256 features x 256 tokens
        using B = Shape<2, 3, 4, 2>;        // 256 x 192
        using C = Shape<4, 1, 2, 4>;        // 256 x 128
        using D = Shape<2, 2, 2, 2>;        // 128 x 128
        using E = Shape<2, 1, 2, 2>;        // 128 x 64
        const auto time = [](int64_t tiles, double full, double least) {
            const int64_t rest = tiles % kComputeUnits;
            const double last = least + (full - least) * rest / kComputeUnits;
            return (double)(tiles / kComputeUnits) * full + (rest ? last : 0.);
        };
        const double times[] = {
            time(tiles_in<A>(a), 34., 22.), time(tiles_in<B>(a), 28.4, 18.),
            a.residual ? INFINITY : time(tiles_in<C>(a), 21., 13.5),
            time(tiles_in<D>(a), 11.3, 8.5), time(tiles_in<E>(a), 7.4, 6.6)};
        switch (std::min_element(times, times + 5) - times) {
            case 0: return tiles_of<T, Act, A>(a, s);
            case 1: return tiles_of<T, Act, B>(a, s);
            case 2: return tiles_of<T, Act, C, false>(a, s);
            case 3: return tiles_of<T, Act, D>(a, s);
            default: return tiles_of<T, Act, E>(a, s);
        }
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
