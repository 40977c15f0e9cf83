// attention_bwd.hip -- p3d_attention_backward (include/p3d_block.h). With the
// forward call's lse the probabilities are one exponential away from the
// scores, P = exp(scale S - lse), so both kernels recompute them tile by tile:
//
//   dq kernel     a wave holds 32 query rows and walks the keys:
//                 dS^T = P^T (V dO^T - D),  dQ^T += K^T dS^T
//                 with D_i = dout_i . out_i, and on the way sums up
//                 D_i = sum_j P_ij (dout_i . v_j)
//   dkv kernel    a wave holds 32 keys and walks the query rows, with that D:
//                 dV^T += dO^T P,  dK^T += Q^T dS
//
// A result is off by its own rounding to bf16, by that of dS or P (as large) and
// by D's, which out's rounding and that of the forward call's P have moved: half
// as large where a row sees some ten keys, and less as the root of their
// number. All three make 1.57 times the first alone on items of 11 keys, 1.43
// on long ones. Rows that see few keys therefore take dS as the sum of two bf16
// factors (1.24 there; another product on fragments already read, 40 % more
// time if every row did), items of a single tile of keys sum D up before dq uses
// it (1.78 -> 1.0 on three keys), and dk takes the D that the dq kernel sums up
// (1.42). dk and dv of a key that one or two rows see carry the rounding of
// those rows' dS and P whole: 1.4 as a mean, up to 1.64 over 300 drawn cases.
//
// Each product's second factor is the softmax tile as the first product left
// it in registers (attn_tile.h). The scores are computed twice, once per
// kernel (7 products instead of 5): the alternative, adding dQ from the dkv
// kernel with atomics, changes results from run to run and moves 4 bytes per
// 1280 operations through the caches.
//
// Where few tiles face a long axis the walked axis is cut into parts whose
// binary32 sums go to the workspace and are joined by join_kernel.
//
// Causal, 12,289 tokens, 12 heads of 128 on 4: dq 0.68 ms, dkv 0.86 ms, 1.03 and
// 1.07 PFLOP/s of seen pairs. dq is bound by its matrix and vector instructions
// together (a SIMD's units are busy 51 and 46 % of the time), dkv by waits of
// its two waves a SIMD beside them (54 and 30 %). Heads of 64 (7000 queries, 2 x
// 1029 keys, 16 heads: dq 75 us, dkv 80 and join 12) fill neither unit: 24 and
// 39 % of dq's time, 33 and 32 % of dkv's. Their waves stand at a wait or a
// barrier for 36 and 26 % of theirs, and the last round is not full.
#include <algorithm>
#include <type_traits>

#include "attn_tile.h"

namespace p3d {

namespace {

using namespace attn;

constexpr int kWaves = 4;
constexpr int kHeld = 32 * kWaves;       // rows (dq) or keys (dkv) held by a workgroup
constexpr int kWalk = 64;                // keys of a tile that the dq kernel walks
constexpr int kFineKeys = 256;           // rows seeing at most so many take dS in two factors

struct BwdArgs {
    AttnArgs a;
    ItemTable tiles;                     // first tile of every item, of rows or keys
    Group group;
    int splits;
    float *minus_lse, *minus_d;          // [heads][nq], then -inf and 0
    float *part, *part2;                 // [splits][n * heads][head_dim]: dq, or dk and dv
    float* part_d;                       // [splits][nq * heads]
};

// A held tile's binary32 sums to the workspace; `row` counts (token, head).
template <int HD>
__device__ __forceinline__ void store_sums(const f32x16 (&o)[Tile<HD>::kBlocks], float* out,
                                           int hd, int lane) {
    const int h = lane >> 5;
#pragma unroll
    for (int b = 0; b < Tile<HD>::kBlocks; ++b)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int d = 32 * b + 8 * j + 4 * h;
            if (d < hd)
                *reinterpret_cast<float4*>(out + d) = make_float4(
                    o[b][4 * j], o[b][4 * j + 1], o[b][4 * j + 2], o[b][4 * j + 3]);
        }
}

// Issue orders. The two products of `Steps` steps: `Ahead` + 4 LDS reads, then
// a matrix instruction and a read in turn.
template <int Steps, int Ahead>
__device__ __forceinline__ void products_in_turn() {
    __builtin_amdgcn_sched_group_barrier(0x100, Ahead + 4, 0);
#pragma unroll
    for (int i = 0; i < 2 * Steps; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
}

// Two sets of `N` matrix instructions on transposed fragments, each set behind
// its half of `2 Vector` vector instructions: the second half goes under the
// first set.
template <int N, int Vector>
__device__ __forceinline__ void sums_in_turn() {
    __builtin_amdgcn_sched_group_barrier(0x100, 8, 0);
    __builtin_amdgcn_sched_group_barrier(0x002, Vector, 0);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
        __builtin_amdgcn_sched_group_barrier(0x002, (Vector + N - 1) / N, 0);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
    }
}

// (Heads of 64, three waves a SIMD: three registers are kept in memory outside
// the loop.)
template <int HD>
__global__ __launch_bounds__(64 * kWaves, HD <= 64 ? 3 : 2) void dq_kernel(BwdArgs f) {
    using T = Tile<HD>;
    __shared__ alignas(kTileAlign) uint4 kt[2][kWalk * T::kChunks];
    __shared__ alignas(kTileAlign) uint4 vt[2][kWalk * T::kChunks];
    const AttnArgs& a = f.a;
    const int lane = threadIdx.x & 63, h = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int chunks = a.head_dim >> 3;

    const int tile = blockIdx.x / a.kv_heads, kv_head = blockIdx.x - tile * a.kv_heads;
    const int item = item_of_tile(f.tiles, a.batch, tile);
    const int tiles = f.tiles.start[item + 1] - f.tiles.start[item];
    const int nth = tile - f.tiles.start[item];
    const uint32_t row0 = (uint32_t)(a.causal ? tiles - 1 - nth : nth) * kHeld;
    const int q0 = a.q_items.start[item], nq = a.q_items.start[item + 1] - q0;
    const int k0 = a.k_items.start[item], nk = a.k_items.start[item + 1] - k0;
    const uint32_t rows = (uint32_t)nq * f.group.size;

    const uint32_t row = row0 + 32 * wave + (lane & 31);
    const bool live = row < rows;
    uint32_t token, member;
    f.group.split(live ? row : 0, token, member);
    const int head = kv_head * f.group.size + member;
    int part = (nk + f.splits - 1) / f.splits;
    part = (part + kWalk - 1) / kWalk * kWalk;
    const int begin = (int)min((int64_t)blockIdx.y * part, (int64_t)nk);
    int end = (int)min((int64_t)begin + part, (int64_t)nk);
    int limit = end, fewest = nk;            // fewest: keys that the tile's first row sees
    if (a.causal) {
        limit = min(end, live ? (int)token + nk - nq + 1 : end);
        uint32_t first, last, m;
        f.group.split(row0, first, m);
        f.group.split(min(row0 + kHeld, rows) - 1, last, m);
        fewest = (int)first + nk - nq + 1;
        end = min(end, (int)last + nk - nq + 1);
    }
    const int all_see = __builtin_amdgcn_readfirstlane(limit);

    // the first tile travels while the rows' own values are loaded
    if (chunks < T::kChunks) {
        for (int i = 0; i < 2; ++i) {
            T::clear(kt[i], kWalk, 64 * kWaves, threadIdx.x);
            T::clear(vt[i], kWalk, 64 * kWaves, threadIdx.x);
        }
        __syncthreads();
    }
    const uint16_t* kb = reinterpret_cast<const uint16_t*>(a.k) + (int64_t)k0 * a.k_stride +
                         kv_head * a.head_dim;
    const uint16_t* vb = reinterpret_cast<const uint16_t*>(a.v) + (int64_t)k0 * a.v_stride +
                         kv_head * a.head_dim;
    // rows past the item's last key repeat it; their dS is 0
    auto fetch = [&](int buf, int key) {
        T::template load<kWalk, kWaves>(kt[buf], wave, lane, chunks, [&](int r) {
            return reinterpret_cast<const uint4*>(kb + (int64_t)min(key + r, nk - 1) * a.k_stride);
        });
        T::template load<kWalk, kWaves>(vt[buf], wave, lane, chunks, [&](int r) {
            return reinterpret_cast<const uint4*>(vb + (int64_t)min(key + r, nk - 1) * a.v_stride);
        });
    };
    if (begin < end) fetch(0, begin);

    bf16x8_t q[T::kSteps], dout[T::kSteps];
    load_query<HD>(q,
                   reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(a.q) +
                                                  (int64_t)(q0 + (int)token) * a.q_stride +
                                                  head * a.head_dim),
                   live, chunks, lane);
    load_query<HD>(dout,
                   reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(a.dout) +
                                                  (int64_t)(q0 + (int)token) * a.dout_stride +
                                                  head * a.head_dim),
                   live, chunks, lane);
    // What the score and dP products of the row start from in the dkv kernel:
    // -lse / scale, so that P = exp2(scale log2(e) (S - lse / scale)), and -D. A
    // row that sees no key starts from -inf: its P is 0. Here D = dout . out.
    const float c = a.scale * kLog2e;
    const int64_t stat = (int64_t)a.q_items.start[a.batch] * head + q0 + (int)token;
    float lse = -INFINITY, minus_d = 0.f;
    if (live) {
        lse = a.lse_in[(int64_t)(q0 + (int)token) * a.heads + head];
        const uint4* o = reinterpret_cast<const uint4*>(
            reinterpret_cast<const uint16_t*>(a.out_in) +
            (int64_t)(q0 + (int)token) * a.out_stride + head * a.head_dim);
#pragma unroll
        for (int k = 0; k < T::kSteps; ++k) {
            const int chunk = 2 * k + h;
            if (chunk >= chunks) continue;
            float x[8], y[8];
            Vec<Bf16>::widen(o[chunk], x);
            Vec<Bf16>::widen(__builtin_bit_cast(uint4, dout[k]), y);
#pragma unroll
            for (int e = 0; e < 8; ++e) minus_d -= x[e] * y[e];
        }
    }
    {
        float own;
        const float other = other_half(minus_d, own);
        minus_d = own + other;
    }
    float minus_lse2 = lse == -INFINITY ? -INFINITY : -lse * kLog2e;
    if (live && lane < 32 && blockIdx.y == 0)
        f.minus_lse[stat] = lse == -INFINITY ? -INFINITY : -lse / a.scale;
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) {
        const int64_t past = (int64_t)a.heads * a.q_items.start[a.batch];
        f.minus_lse[past] = -INFINITY;
        f.minus_d[past] = 0.f;
    }
    settle(q);
    settle(dout);
    asm volatile("" : "+v"(minus_lse2), "+v"(minus_d));

    f32x16 dq[T::kBlocks];
#pragma unroll
    for (int b = 0; b < T::kBlocks; ++b) dq[b] = zero16();
    auto products = [&](f32x16& s, f32x16& dp, uint32_t k_at, uint32_t v_at, int b) {
        s = zero16();
        dp = zero16();
#pragma unroll
        for (int k = 0; k < T::kSteps; ++k) {
            s = mfma(T::row_frag(k_at, 32 * b, k), q[k], s);
            dp = mfma(T::row_frag(v_at, 32 * b, k), dout[k], dp);
        }
    };
    auto mask = [&](f32x16& s, int key) {
        const int left = limit - key - 4 * h;
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (acc_row(i, 0) >= left) s[i] = -INFINITY;
    };
    // dS as a bf16 factor (fine: as the sum of two), and this lane's share of D
    float sum_d = 0.f;
    auto gradient = [&](auto fine, f32x16& s, const f32x16& dp, bf16x8_t* hi, bf16x8_t* lo) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float p = __builtin_amdgcn_exp2f(fmaf(s[i], c, minus_lse2));
            sum_d = fmaf(p, dp[i], sum_d);
            const float g = p * (dp[i] + minus_d);
            hi[i >> 3][i & 7] = (__bf16)g;
            if constexpr (decltype(fine)::value)
                lo[i >> 3][i & 7] = (__bf16)(g - (float)hi[i >> 3][i & 7]);
        }
    };
    auto walk = [&](auto fine, bool masked, int buf, int key) {
        constexpr bool kFine = decltype(fine)::value;
        constexpr int kVector = kFine ? 136 : 88;        // vector instructions of gradient()
        const uint32_t k_at = T::row_base(kt[buf], lane), v_at = T::row_base(vt[buf], lane);
        f32x16 s0, dp0, s1, dp1;
        __builtin_amdgcn_s_setprio(1);       // (as in the forward kernel)
        products(s0, dp0, k_at, v_at, 0);
        products_in_turn<T::kSteps, 4>();
        __builtin_amdgcn_s_setprio(0);
        if (masked) mask(s0, key);
        // the second block's products under the first one's exponentials
        products(s1, dp1, k_at, v_at, 1);
        bf16x8_t hi[4], lo[4];
        gradient(fine, s0, dp0, hi, lo);
        __builtin_amdgcn_sched_group_barrier(0x100, 4, 0);
#pragma unroll
        for (int i = 0; i < 2 * T::kSteps; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x002, kVector / (2 * T::kSteps) + 1, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
        if (masked) mask(s1, key + 32);
        const uint32_t k_tr = T::tr_base(kt[buf], lane);
        gradient(fine, s1, dp1, hi + 2, lo + 2);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            bf16x8_t frag[T::kBlocks];
#pragma unroll
            for (int d = 0; d < T::kBlocks; ++d) frag[d] = T::tr_frag(k_tr, 16 * t, d);
#pragma unroll
            for (int d = 0; d < T::kBlocks; ++d) dq[d] = mfma(frag[d], hi[t], dq[d]);
            if constexpr (kFine)
#pragma unroll
                for (int d = 0; d < T::kBlocks; ++d) dq[d] = mfma(frag[d], lo[t], dq[d]);
        }
        __builtin_amdgcn_sched_group_barrier(0x100, 8, 0);
#pragma unroll
        for (int i = 0; i < (kFine ? 8 : 4) * T::kBlocks; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, kFine ? 1 : 2, 0);
            __builtin_amdgcn_sched_group_barrier(
                0x002, kVector / ((kFine ? 4 : 2) * T::kBlocks) + 1, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    auto walk_all = [&](auto fine) {
        int buf = 0;
        for (int key = begin; key < end; key += kWalk, buf ^= 1) {
            tile_barrier();
            if (key + kWalk < end) fetch(buf ^ 1, key + kWalk);
            walk(fine, key + kWalk > all_see, buf, key);
        }
    };
    // Rows of a single tile of keys are short enough for out's rounding to show
    // in D (dq 1.78 times its own rounding off with three keys): they sum D up
    // before they use it.
    if (nk <= kWalk && begin < end) {
        tile_barrier();
        const uint32_t k_at = T::row_base(kt[0], lane), v_at = T::row_base(vt[0], lane);
        float sum = 0.f;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            f32x16 s, dp;
            products(s, dp, k_at, v_at, b);
            mask(s, 32 * b);
#pragma unroll
            for (int i = 0; i < 16; ++i)
                sum = fmaf(__builtin_amdgcn_exp2f(fmaf(s[i], c, minus_lse2)), dp[i], sum);
        }
        float own;
        const float other = other_half(sum, own);
        minus_d = -(own + other);
    }
    // (by the item and the rows, not by this part's keys: how the launch is cut
    // does not change a rounding)
    if (fewest <= kFineKeys) walk_all(std::true_type{});
    else walk_all(std::false_type{});

    // A row that sees one key has P = 1 and dS = 0; P (dP - D) leaves a few
    // 2^-24 of dP there, which would be all of dq.
    if (live && (a.causal ? (int)token + nk - nq : nk - 1) == 0)
#pragma unroll
        for (int b = 0; b < T::kBlocks; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i) dq[b][i] *= 0.f;

    float own;
    const float other = other_half(sum_d, own);
    sum_d = own + other;
    const int64_t out_row = (int64_t)(q0 + (int)token) * a.heads + head;
    if (f.splits > 1) {
        const int64_t all = (int64_t)a.q_items.start[a.batch] * a.heads;
        if (live) {
            store_sums<HD>(dq, f.part + (blockIdx.y * all + out_row) * a.head_dim, a.head_dim,
                           lane);
            if (lane < 32) f.part_d[blockIdx.y * all + out_row] = sum_d;
        }
        return;
    }
    if (live && lane < 32) f.minus_d[stat] = -sum_d;
    tile_barrier();
    const float by = a.scale;
    uint4* stage = wave < 2 ? kt[wave] : vt[wave - 2];
    store_rows<HD>(dq, by, stage, chunks, lane, [&](int r) -> uint4* {
        const uint32_t at = row0 + 32 * wave + r;
        if (at >= rows) return nullptr;
        uint32_t t, m;
        f.group.split(at, t, m);
        return reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.dq) +
                                        (int64_t)(q0 + (int)t) * a.dq_stride +
                                        (kv_head * f.group.size + m) * a.head_dim);
    });
}

// Walks the rows of one key head's query heads, head by head, in tiles of 32
// tokens (64 for narrow heads: half the barriers): every tile is a run of
// tokens of one head, loaded as it lies.
//
// The wave's two sums take 128 registers for heads of 128 and its keys 32. Its
// values stay in LDS: 32 registers more would leave two waves a SIMD nothing
// to read fragments ahead into, and every matrix instruction would wait for
// LDS (one wave a SIMD, with registers to spare, is held up by its own issue).
// Heads of 64 leave room for three waves a SIMD (98 -> 89 us for 2 x 1029
// keys, at the price of one register kept in memory outside the loop) and for
// tiles of 64 rows (89 -> 85 us).
template <int HD>
__global__ __launch_bounds__(64 * kWaves, HD <= 64 ? 3 : 2) void dkv_kernel(BwdArgs f) {
    using T = Tile<HD>;
    constexpr int kRows = HD <= 64 ? 64 : 32;
    // [buffer][q rows, dout rows]
    __shared__ alignas(kTileAlign) uint4 tiles[2][2 * kRows * T::kChunks];
    __shared__ alignas(kTileAlign) uint4 values[kHeld * T::kChunks];
    __shared__ alignas(16) float stats[2][2][64];        // [buffer][-lse / scale, -D]
    const AttnArgs& a = f.a;
    const int lane = threadIdx.x & 63, h = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int chunks = a.head_dim >> 3;

    // Causal: the parts of the longest tiles first, so that the last ones to
    // run are short (12,289 tokens: 961 us the other way round, 878 this way).
    // Otherwise part by part, so that neighbours walk the same rows (2 x 1029
    // keys: 104 and 96 us).
    const int units = gridDim.x / f.splits;
    const int unit = a.causal ? blockIdx.x / f.splits : blockIdx.x % units;
    const int part = a.causal ? blockIdx.x % f.splits : blockIdx.x / units;
    const int tile = unit / a.kv_heads, kv_head = unit - tile * a.kv_heads;
    const int item = item_of_tile(f.tiles, a.batch, tile);
    const int key0 = (tile - f.tiles.start[item]) * kHeld;
    const int q0 = a.q_items.start[item], nq = a.q_items.start[item + 1] - q0;
    const int k0 = a.k_items.start[item], nk = a.k_items.start[item + 1] - k0;
    const int group = f.group.size;

    if (chunks < T::kChunks) {
        for (int i = 0; i < 2; ++i) T::clear(tiles[i], 2 * kRows, 64 * kWaves, threadIdx.x);
        T::clear(values, kHeld, 64 * kWaves, threadIdx.x);
        __syncthreads();
    }
    const int key = key0 + 32 * wave + (lane & 31);
    const bool live = key < nk;
    // Tokens from `from` on see this lane's key, from `all_from` on all of the
    // wave's, and none before the first tile sees any of the workgroup's.
    int first = 0, from = 0, all_from = 0;
    if (a.causal) {
        from = min(max(key - (nk - nq), 0), nq);
        all_from = min(max(key0 + 32 * wave + 31 - (nk - nq), 0), nq);
        first = min(max(key0 - (nk - nq), 0), nq) / kRows;
    }
    // This part of the tiles, numbered over (head, token tile), is the same
    // for every workgroup of the key head, and is walked from its end: they
    // read the same rows at the same time, from their XCD's L2, whatever
    // their causal first tile is. (Walking up from it, 56 % of the reads of
    // 12,289 tokens missed L2.)
    const int per_head = (nq + kRows - 1) / kRows;
    const int64_t all = (int64_t)per_head * group;
    const int low = (int)(all * part / f.splits);
    const int high = (int)(all * (part + 1) / f.splits);
    const int last_member = low < high ? low / per_head : 0;
    int member = low < high ? (high - 1) / per_head : -1;
    int at_tile = min(per_head, high - member * per_head) - 1;
    auto settle_tile = [&] {                 // on to a tile that sees a key, or past the part
        while (member >= last_member && at_tile < max(first, low - member * per_head)) {
            --member;
            at_tile = per_head - 1;
        }
    };
    settle_tile();
    const float c = a.scale * kLog2e;

    f32x16 dk[T::kBlocks], dv[T::kBlocks];
#pragma unroll
    for (int b = 0; b < T::kBlocks; ++b) dk[b] = dv[b] = zero16();
    const uint16_t* qb = reinterpret_cast<const uint16_t*>(a.q) + (int64_t)q0 * a.q_stride +
                         kv_head * group * a.head_dim;
    const uint16_t* ob = reinterpret_cast<const uint16_t*>(a.dout) + (int64_t)q0 * a.dout_stride +
                         kv_head * group * a.head_dim;
    const int64_t stat = (int64_t)kv_head * group * a.q_items.start[a.batch] + q0;
    const int64_t past = (int64_t)a.heads * a.q_items.start[a.batch];
    const int64_t q_pitch = a.q_stride * 2, o_pitch = a.dout_stride * 2;
    const bool near = max(q_pitch, o_pitch) <= T::kMaxPitch;
    const uint32_t q_off = T::lane_offset(wave, lane, q_pitch);
    const uint32_t o_off = T::lane_offset(wave, lane, o_pitch);
    const bool on = T::lane_chunk(wave, lane) < chunks;

    // The next tile to load. Tokens past the item's last repeat it and start
    // from the -inf behind the last row's value, so their P is 0.
    auto fetch = [&](int buf) {
        const int token = at_tile * kRows;
        const uint16_t* qm = qb + member * a.head_dim;
        const uint16_t* om = ob + member * a.head_dim;
        uint4* qt = tiles[buf];
        uint4* ot = tiles[buf] + kRows * T::kChunks;
        if (wave < 2) {
            const int t = token + lane;
            const int64_t at = t < nq ? stat + (int64_t)member * a.q_items.start[a.batch] + t
                                      : past;
            dma4((wave ? f.minus_d : f.minus_lse) + at, lds_offset(stats[buf][wave]));
        }
        if (near && token + kRows <= nq) {
            T::template load_rows<kRows, kWaves>(qt, wave, qm + (int64_t)token * a.q_stride,
                                                 q_pitch, q_off, on);
            T::template load_rows<kRows, kWaves>(ot, wave, om + (int64_t)token * a.dout_stride,
                                                 o_pitch, o_off, on);
        } else {
            T::template load<kRows, kWaves>(qt, wave, lane, chunks, [&](int r) {
                return reinterpret_cast<const uint4*>(qm +
                                                      (int64_t)min(token + r, nq - 1) * a.q_stride);
            });
            T::template load<kRows, kWaves>(ot, wave, lane, chunks, [&](int r) {
                return reinterpret_cast<const uint4*>(
                    om + (int64_t)min(token + r, nq - 1) * a.dout_stride);
            });
        }
    };
    // the first tile travels while the keys and values are loaded
    if (member >= last_member) fetch(0);
    bf16x8_t kf[T::kSteps];
    load_query<HD>(kf,
                   reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(a.k) +
                                                  (int64_t)(k0 + (live ? key : 0)) * a.k_stride +
                                                  kv_head * a.head_dim),
                   live, chunks, lane);
    // (keys past the item's last repeat it; their sums are not stored)
    T::template load<kHeld, kWaves>(values, wave, lane, chunks, [&](int r) {
        return reinterpret_cast<const uint4*>(
            reinterpret_cast<const uint16_t*>(a.v) +
            (int64_t)(k0 + min(key0 + r, nk - 1)) * a.v_stride + kv_head * a.head_dim);
    });
    settle(kf);

    // 32 rows of a tile, from row `sub` on. The issue order is the written one:
    // a matrix instruction, the reads of the fragments a few matrix instructions
    // on, and in the first half of the sums the exponentials that the second
    // half needs.
    auto walk = [&](bool masked, int buf, int sub, int row) {
        constexpr int kAhead = 3;
        const uint4* rows = tiles[buf] + sub * T::kChunks;
        const uint32_t at = T::row_base(rows, lane);
        const uint32_t v_at = T::row_base(values + 32 * wave * T::kChunks, lane);
        f32x16 s, dp;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float4 l = *reinterpret_cast<const float4*>(&stats[buf][0][sub + 8 * j + 4 * h]);
            const float4 d = *reinterpret_cast<const float4*>(&stats[buf][1][sub + 8 * j + 4 * h]);
            s[4 * j] = l.x, s[4 * j + 1] = l.y, s[4 * j + 2] = l.z, s[4 * j + 3] = l.w;
            dp[4 * j] = d.x, dp[4 * j + 1] = d.y, dp[4 * j + 2] = d.z, dp[4 * j + 3] = d.w;
        }
        bf16x8_t qf[kAhead], of[kAhead], vf[kAhead];
        auto read = [&](int k) {
            qf[k % kAhead] = T::row_frag(at, 0, k);
            of[k % kAhead] = T::row_frag(at, kRows, k);
            vf[k % kAhead] = T::row_frag(v_at, 0, k);
        };
#pragma unroll
        for (int k = 0; k < kAhead; ++k) read(k);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int k = 0; k < T::kSteps; ++k) {
            s = mfma(qf[k % kAhead], kf[k], s);
            dp = mfma(of[k % kAhead], vf[k % kAhead], dp);
            if (k + kAhead < T::kSteps) read(k + kAhead);
            __builtin_amdgcn_sched_barrier(0);
        }
        if (masked) {
            const int before = from - row - 4 * h;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (acc_row(i, 0) < before) s[i] = -INFINITY;
        }
        const uint32_t tr = T::tr_base(rows, lane);
        constexpr int kSums = 4 * T::kBlocks, kTrAhead = 5;
        bf16x8_t frag[kTrAhead];
        auto read_tr = [&](int i) {          // (t, d, dv or dk)
            const int t = i / (2 * T::kBlocks), d = i / 2 % T::kBlocks;
            frag[i % kTrAhead] = T::tr_frag(tr, (i & 1 ? 0 : kRows) + 16 * t, d);
        };
        bf16x8_t p[2], ds[2];
        auto element = [&](int e) {
            s[e] = __builtin_amdgcn_exp2f(s[e] * c);
            dp[e] *= s[e];
            p[e >> 3][e & 7] = (__bf16)s[e];
            ds[e >> 3][e & 7] = (__bf16)dp[e];
        };
#pragma unroll
        for (int i = 0; i < kTrAhead; ++i) read_tr(i);
#pragma unroll
        for (int e = 0; e < 8; ++e) element(e);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < kSums; ++i) {
            const int t = i / (2 * T::kBlocks), d = i / 2 % T::kBlocks;
            if (i & 1) dk[d] = mfma(frag[i % kTrAhead], ds[t], dk[d]);
            else dv[d] = mfma(frag[i % kTrAhead], p[t], dv[d]);
            if (i + kTrAhead < kSums) read_tr(i + kTrAhead);
            if (t == 0)
#pragma unroll
                for (int e = 8 + 8 * i / (2 * T::kBlocks); e < 8 + 8 * (i + 1) / (2 * T::kBlocks);
                     ++e)
                    element(e);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    int buf = 0;
    while (member >= last_member) {
        const int row = at_tile * kRows;                 // of the tile in `buf`
        tile_barrier();
        --at_tile;
        settle_tile();
        if (member >= last_member) fetch(buf ^ 1);
#pragma unroll 1
        for (int sub = 0; sub < kRows && row + sub < nq; sub += 32)
            walk(row + sub < all_from, buf, sub, row + sub);
        buf ^= 1;
    }

    if (nk == 1)                             // (as in the dq kernel)
#pragma unroll
        for (int b = 0; b < T::kBlocks; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i) dk[b][i] *= 0.f;

    if (f.splits > 1) {
        if (!live) return;
        const int64_t rows = (int64_t)a.k_items.start[a.batch] * a.kv_heads;
        const int64_t at = (part * rows + (int64_t)(k0 + key) * a.kv_heads + kv_head) *
                           a.head_dim;
        store_sums<HD>(dk, f.part + at, a.head_dim, lane);
        store_sums<HD>(dv, f.part2 + at, a.head_dim, lane);
        return;
    }
    tile_barrier();
    uint4* stage = values + wave * 32 * T::kChunks;
    auto to = [&](void* base, int64_t stride) {
        return [=](int r) -> uint4* {
            const int at = key0 + 32 * wave + r;
            if (at >= nk) return nullptr;
            return reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(base) +
                                            (int64_t)(k0 + at) * stride + kv_head * a.head_dim);
        };
    };
    store_rows<HD>(dk, a.scale, stage, chunks, lane, to(a.dk, a.dk_stride));
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    store_rows<HD>(dv, 1.0f, stage, chunks, lane, to(a.dv, a.dv_stride));
}

// What is joined into one result.
struct Joint {
    const float* part;
    float by;
    void* out;
    int64_t stride;
};

// Adds the parts of (token, head) rows in order: 32 lanes per row, two results
// side by side. With `part_d`, also those of D, into minus_d [heads][tokens].
__global__ __launch_bounds__(256) void join_kernel(Joint first, Joint second, int splits,
                                                   int64_t rows, int heads, int hd,
                                                   const float* part_d, float* minus_d) {
    const Joint& j = blockIdx.y ? second : first;
    const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int d = (threadIdx.x & 31) * 4;
    if (row >= rows || d >= hd) return;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int p = 0; p < splits; ++p) {
        const float4 v = *reinterpret_cast<const float4*>(j.part + (p * rows + row) * hd + d);
        s.x += v.x;
        s.y += v.y;
        s.z += v.z;
        s.w += v.w;
    }
    const int64_t token = row / heads;
    const int head = (int)(row - token * heads);
    *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(j.out) + token * j.stride + head * hd +
                              d) =
        make_uint2(pack_bf16x2(s.x * j.by, s.y * j.by), pack_bf16x2(s.z * j.by, s.w * j.by));
    if (part_d && d == 0) {
        float sum = 0.f;
        for (int p = 0; p < splits; ++p) sum += part_d[p * rows + row];
        minus_d[rows / heads * head + token] = -sum;
    }
}

template <int HD>
hipError_t backward_as(BwdArgs& f, const AttnPlan& p, hipStream_t s) {
    const AttnArgs& a = f.a;
    const int64_t q_rows = (int64_t)a.q_items.start[a.batch] * a.heads;
    const int64_t k_rows = (int64_t)a.k_items.start[a.batch] * a.kv_heads;
    hipError_t e;
    if (q_rows > 0) {
        cut_items(a.q_items, a.batch, f.group.size, kHeld, &f.tiles);
        f.splits = p.dq_splits;
        f.part_d = f.part + f.splits * q_rows * a.head_dim;
        dq_kernel<HD><<<dim3((unsigned)f.tiles.start[a.batch] * a.kv_heads, (unsigned)f.splits),
                        dim3(64 * kWaves), 0, s>>>(f);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        if (f.splits > 1) {
            const Joint dq{f.part, a.scale, a.dq, a.dq_stride};
            join_kernel<<<dim3((unsigned)((q_rows + 7) / 8)), dim3(256), 0, s>>>(
                dq, dq, f.splits, q_rows, a.heads, a.head_dim, f.part_d, f.minus_d);
            if ((e = hipGetLastError()) != hipSuccess) return e;
        }
    }
    if (k_rows > 0) {
        cut_items(a.k_items, a.batch, 1, kHeld, &f.tiles);
        f.splits = p.dk_splits;
        f.part2 = f.part + f.splits * k_rows * a.head_dim;
        dkv_kernel<HD><<<dim3((unsigned)(f.tiles.start[a.batch] * a.kv_heads * f.splits)),
                         dim3(64 * kWaves), 0, s>>>(f);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        if (f.splits > 1) {
            const Joint dk{f.part, a.scale, a.dk, a.dk_stride};
            const Joint dv{f.part2, 1.0f, a.dv, a.dv_stride};
            join_kernel<<<dim3((unsigned)((k_rows + 7) / 8), 2), dim3(256), 0, s>>>(
                dk, dv, f.splits, k_rows, a.kv_heads, a.head_dim, nullptr, nullptr);
            return hipGetLastError();
        }
    }
    return hipSuccess;
}

// Parts of a walked axis of `most` entries when `blocks` workgroups hold the
// other.
int parts(int64_t blocks, int64_t most) {
    if (blocks == 0 || blocks >= 4 * kComputeUnits) return 1;
    const bool few = blocks < kComputeUnits;
    const int64_t wanted = ((few ? 2 : 4) * kComputeUnits + blocks - 1) / blocks;
    return (int)std::max<int64_t>(1, std::min<int64_t>(wanted, most / (few ? 256 : 1024)));
}

size_t padded(size_t bytes) { return (bytes + 255) / 256 * 256; }

}  // namespace

void plan_attention_backward(const AttnArgs& a, AttnPlan* p) {
    const Group g = group_of(a);
    ItemTable rt, kt;
    cut_items(a.q_items, a.batch, g.size, kHeld, &rt);
    cut_items(a.k_items, a.batch, 1, kHeld, &kt);
    int64_t most_rows = 0, most_keys = 0;
    for (int b = 0; b < a.batch; ++b) {
        most_rows = std::max<int64_t>(
            most_rows, (int64_t)(a.q_items.start[b + 1] - a.q_items.start[b]) * g.size);
        most_keys = std::max<int64_t>(most_keys, a.k_items.start[b + 1] - a.k_items.start[b]);
    }
    p->dq_splits = parts((int64_t)rt.start[a.batch] * a.kv_heads, most_keys);
    p->dk_splits = parts((int64_t)kt.start[a.batch] * a.kv_heads, most_rows);
    const size_t q_rows = (size_t)a.q_items.start[a.batch] * a.heads;
    const size_t k_rows = (size_t)a.k_items.start[a.batch] * a.kv_heads;
    const size_t dq = p->dq_splits > 1 ? p->dq_splits * q_rows * (a.head_dim + 1) : 0;
    const size_t dk = p->dk_splits > 1 ? 2 * p->dk_splits * k_rows * a.head_dim : 0;
    p->backward_bytes = 256 + 2 * padded((q_rows + 1) * sizeof(float)) +
                        std::max(dq, dk) * sizeof(float);
}

hipError_t launch_attention_backward(const AttnArgs& a, const AttnPlan& p, void* ws,
                                     hipStream_t s) {
    const int64_t q_rows = (int64_t)a.q_items.start[a.batch] * a.heads;
    BwdArgs f{};
    f.a = a;
    f.group = group_of(a);
    char* at = static_cast<char*>(ws);
    f.minus_lse = reinterpret_cast<float*>(at);
    at += padded((q_rows + 1) * sizeof(float));
    f.minus_d = reinterpret_cast<float*>(at);
    at += padded((q_rows + 1) * sizeof(float));
    f.part = reinterpret_cast<float*>(at);
    return a.head_dim <= 64   ? backward_as<64>(f, p, s)
           : a.head_dim <= 96 ? backward_as<96>(f, p, s)
                              : backward_as<128>(f, p, s);
}

}  // namespace p3d
