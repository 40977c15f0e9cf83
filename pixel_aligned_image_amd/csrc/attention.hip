// attention.hip -- p3d_attention (include/p3d_block.h): softmax attention in
// one pass over the keys with a running maximum and sum.
//
// A wave holds 32 query rows as the columns of its products (attn_tile.h): for
// a tile of keys it computes S^T = K Q^T, turns it into P^T = exp(scale (S -
// m)) in registers and adds V^T P^T to O^T, all 32 columns of a lane's query
// in its own registers. The rows of one key head's group of query heads are
// numbered together, so shared heads read their keys once.
//
// The running maximum m is only raised when a tile exceeds it by more than
// 2^8 (in the exponent of the probabilities): until then P is up to 2^8 times
// larger than with the exact maximum, which costs no bits, and the 2^5 or 2^6
// multiplications that a new maximum brings are rarely due.
//
// Where the row tiles do not fill the chip's last round the keys of the last
// ones are cut into parts, each of which leaves (m, l, O) in the workspace,
// joined by combine_kernel. Two cases have kernels of their own: items of few
// rows (single tokens), and items of few keys (global tokens).
//
// Heads of 128 take 0.84 ms for 12,000 tokens of 12 heads (1.06 PFLOP/s) and
// 0.46 ms for 12,289 causal ones (1.0 PFLOP/s of seen pairs; torch's products of
// 8192^3 reach 1.47 here). Bound by the products and the vector instructions of
// the exponentials together: a SIMD's matrix unit is busy 54 % of that time and
// its vector unit 49 (causal 50 and 46), so its two waves mostly take turns, at
// the 1.6-1.8 GHz that the load leaves. Heads of 64 (7000 queries, 2 x 1029
// keys, 16 heads: 47 us and a join of 8, 0.56 PFLOP/s) have half the products
// per exponential: 25 and 46 %, and a last round that is not full.
#include <algorithm>
#include <type_traits>

#include "attn_tile.h"

namespace p3d {

namespace {

using namespace attn;

constexpr int kKeys = 64;                // keys per tile of attention_kernel
constexpr int kWaves = 4;
constexpr int kRows = 32 * kWaves;       // query rows per workgroup
constexpr int kSingleRows = 32;          // query rows of attention_single_kernel
constexpr int kSingleKeys = 32;          // keys per wave tile of attention_single_kernel
constexpr int kMostParts = 64;           // a wave joins them, one lane each

struct FwdArgs {
    AttnArgs a;
    ItemTable tiles;                     // first row tile (single: part) of every item
    Group group;
    int whole, parts;                    // units run whole; parts of every later one
    int share;                           // single: keys of a part
    float* part_o;                       // [slot][rows of a tile][head_dim]
    float2* part_ml;                     // [slot][rows of a tile]
};

// A unit of the launch: one row tile of one key head. Tiles of an item run
// the longest causal ones first and key heads fastest: workgroups go to the
// XCDs in turn, so with 8 (or 16, 24, ...) key heads an XCD's L2 holds the
// same heads throughout.
struct Unit {
    int item, kv_head, q0, nq, k0, nk;
    uint32_t row0, rows;                 // first row of the tile, rows of the item

    __device__ __forceinline__ Unit(const FwdArgs& f, int unit, int per_tile) {
        const int tile = unit / f.a.kv_heads;
        const int it = item_of_tile(f.tiles, f.a.batch, tile);
        const int tiles = f.tiles.start[it + 1] - f.tiles.start[it];
        const int nth = tile - f.tiles.start[it];
        set(f.a, it, unit - tile * f.a.kv_heads, f.group.size,
            (uint32_t)(f.a.causal ? tiles - 1 - nth : nth) * per_tile);
    }
    __device__ __forceinline__ Unit(const AttnArgs& a, int it, int head, int group) {
        set(a, it, head, group, 0);
    }
    __device__ __forceinline__ void set(const AttnArgs& a, int it, int head, int group,
                                        uint32_t first) {
        item = it;
        kv_head = head;
        row0 = first;
        q0 = a.q_items.start[item];
        nq = a.q_items.start[item + 1] - q0;
        k0 = a.k_items.start[item];
        nk = a.k_items.start[item + 1] - k0;
        rows = (uint32_t)nq * group;
    }
};

// The unit of a workgroup, and which part of its keys (-1: all).
__device__ __forceinline__ int unit_of(const FwdArgs& f, int block, int& part) {
    part = -1;
    if (block < f.whole) return block;
    const int u = (block - f.whole) / f.parts;
    part = block - f.whole - u * f.parts;
    return f.whole + u;
}

// One row tile's running softmax: lane l's query is l % 32, and the two
// halves hold different keys (and different columns of O).
template <int HD>
struct Softmax {
    using T = Tile<HD>;
    f32x16 o[T::kBlocks];
    float m, l;                          // l: this half's share

    __device__ __forceinline__ void init() {
#pragma unroll
        for (int b = 0; b < T::kBlocks; ++b) o[b] = zero16();
        m = -INFINITY;
        l = 0.f;
    }

    // S^T of 64 keys (two blocks of 32).
    __device__ __forceinline__ void scores(f32x16 (&s)[2], const bf16x8_t (&q)[T::kSteps],
                                           const uint4* kt, int lane) const {
        const uint32_t at = T::row_base(kt, lane);
        // (ahead of the CU's other waves, whose vector work then fills in)
        __builtin_amdgcn_s_setprio(1);
        s[0] = s[1] = zero16();
#pragma unroll
        for (int k = 0; k < T::kSteps; ++k)
#pragma unroll
            for (int b = 0; b < 2; ++b) s[b] = mfma(T::row_frag(at, 32 * b, k), q[k], s[b]);
        // reads run six matrix instructions ahead
        __builtin_amdgcn_sched_group_barrier(0x100, 6, 0);
#pragma unroll
        for (int i = 0; i < 2 * T::kSteps; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        }
        __builtin_amdgcn_s_setprio(0);
    }

    // Keys at or past `limit` are not seen.
    template <int NB>
    __device__ __forceinline__ void mask(f32x16 (&s)[NB], int key0, int limit, int lane) const {
        const int left = limit - key0 - 4 * (lane >> 5);
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (32 * b + acc_row(i, 0) >= left) s[b][i] = -INFINITY;
    }

    template <int NB>
    __device__ __forceinline__ float top(const f32x16 (&s)[NB]) const {
        float t = s[0][0];
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i) t = fmaxf(t, s[b][i]);
        float own;
        const float other = other_half(t, own);
        return fmaxf(own, other);
    }

    // Whether a query of the wave needs a new maximum.
    template <int NB>
    __device__ __forceinline__ bool exceeds(const f32x16 (&s)[NB], float c) const {
        return __any((top(s) - m) * c > 8.0f);
    }

    // The new maximum.
    template <int NB>
    __device__ __forceinline__ void raise(const f32x16 (&s)[NB], float c) {
        const float raised = fmaxf(m, top(s));
        const float by = raised == -INFINITY ? 0.f : __builtin_amdgcn_exp2f((m - raised) * c);
        m = raised;
        l *= by;
#pragma unroll
        for (int b = 0; b < T::kBlocks; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[b][i] *= by;
    }

    // P^T of 64 keys and its share of l.
    __device__ __forceinline__ void exponentials(const f32x16 (&s)[2], bf16x8_t (&p)[4],
                                                 float c) {
        const float base = m == -INFINITY ? 0.f : m * c;
        float sum = 0.f;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            f32x16 e;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                e[i] = __builtin_amdgcn_exp2f(fmaf(s[b][i], c, -base));
                sum += e[i];
            }
            p[2 * b] = acc_frag(e, 0);
            p[2 * b + 1] = acc_frag(e, 1);
        }
        l += sum;
    }

    // O^T += V^T P^T over 64 keys.
    __device__ __forceinline__ void add(const bf16x8_t (&p)[4], const uint4* vt, int lane) {
        const uint32_t at = T::tr_base(vt, lane);
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int d = 0; d < T::kBlocks; ++d)
                o[d] = mfma(T::tr_frag(at, 16 * t, d), p[t], o[d]);
    }

    // add() of the tile before with `p`, and exponentials() of this one into
    // it: independent of each other, issued in turn.
    __device__ __forceinline__ void exponentials_and_add(const f32x16 (&s)[2], bf16x8_t (&p)[4],
                                                         const uint4* vt, float c, int lane) {
        bf16x8_t next[4];
        add(p, vt, lane);
        exponentials(s, next, c);
        // 8 transposed reads ahead, then per matrix instruction 2 reads and
        // its share of the 112 vector instructions
        __builtin_amdgcn_sched_group_barrier(0x100, 8, 0);
#pragma unroll
        for (int i = 0; i < 4 * T::kBlocks; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
            __builtin_amdgcn_sched_group_barrier(0x002, 28 / T::kBlocks, 0);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = next[i];
    }

    // One block of 32 keys, start to end.
    __device__ __forceinline__ void attend(const bf16x8_t (&q)[T::kSteps], const uint4* kt,
                                           const uint4* vt, int key0, int limit, bool masked,
                                           float c, int lane) {
        const uint32_t k_at = T::row_base(kt, lane), v_at = T::tr_base(vt, lane);
        f32x16 s[1];
        s[0] = zero16();
#pragma unroll
        for (int k = 0; k < T::kSteps; ++k) s[0] = mfma(T::row_frag(k_at, 0, k), q[k], s[0]);
        if (masked) mask(s, key0, limit, lane);
        if (exceeds(s, c)) raise(s, c);
        const float base = m == -INFINITY ? 0.f : m * c;
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            s[0][i] = __builtin_amdgcn_exp2f(fmaf(s[0][i], c, -base));
            sum += s[0][i];
        }
        l += sum;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const bf16x8_t p = acc_frag(s[0], t);
#pragma unroll
            for (int d = 0; d < T::kBlocks; ++d)
                o[d] = mfma(T::tr_frag(v_at, 16 * t, d), p, o[d]);
        }
    }
};

// A part's (m, l, O) to the workspace; `at` counts rows of parts.
template <int HD>
__device__ __forceinline__ void store_part(const FwdArgs& f, const Softmax<HD>& st, int64_t at,
                                           float l, int lane) {
    const int h = lane >> 5, hd = f.a.head_dim;
    if (h == 0) f.part_ml[at] = make_float2(st.m, l);
    float* o = f.part_o + at * hd;
#pragma unroll
    for (int b = 0; b < Tile<HD>::kBlocks; ++b)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int d = 32 * b + 8 * j + 4 * h;
            if (d < hd)
                *reinterpret_cast<float4*>(o + d) =
                    make_float4(st.o[b][4 * j], st.o[b][4 * j + 1], st.o[b][4 * j + 2],
                                st.o[b][4 * j + 3]);
        }
}

template <int HD>
__global__ __launch_bounds__(64 * kWaves, 2) void attention_kernel(FwdArgs f) {
    using T = Tile<HD>;
    __shared__ alignas(kTileAlign) uint4 kt[2][kKeys * T::kChunks];
    __shared__ alignas(kTileAlign) uint4 vt[3][kKeys * T::kChunks];
    const AttnArgs& a = f.a;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int chunks = a.head_dim >> 3;

    int which;
    const int unit = unit_of(f, blockIdx.x, which);
    const Unit u(f, unit, kRows);
    const int kv_head = u.kv_head, q0 = u.q0, nq = u.nq, k0 = u.k0, nk = u.nk;
    const uint32_t row0 = u.row0, rows = u.rows;

    // this lane's query
    const uint32_t row = row0 + 32 * wave + (lane & 31);
    const bool live = row < rows;
    uint32_t token, member;
    f.group.split(live ? row : 0, token, member);
    const int head = kv_head * f.group.size + member;
    // keys of this part, and those this workgroup and this lane see
    const int parts = which < 0 ? 1 : f.parts;
    int share = (nk + parts - 1) / parts;
    share = (share + kKeys - 1) / kKeys * kKeys;
    const int begin = (int)min((int64_t)max(which, 0) * share, (int64_t)nk);
    int end = (int)min((int64_t)begin + share, (int64_t)nk);
    int limit = end;
    if (a.causal) {
        limit = min(end, live ? (int)token + nk - nq + 1 : end);
        uint32_t last, m;
        f.group.split(min(row0 + kRows, rows) - 1, last, m);
        end = min(end, (int)last + nk - nq + 1);
    }
    // the smallest limit of the wave's queries is its first one's
    const int all_see = __builtin_amdgcn_readfirstlane(limit);
    const float c = a.scale * kLog2e;

    Softmax<HD> st;
    st.init();
    if (chunks < T::kChunks) {
        for (int i = 0; i < 2; ++i) T::clear(kt[i], kKeys, 64 * kWaves, threadIdx.x);
        for (int i = 0; i < 3; ++i) T::clear(vt[i], kKeys, 64 * kWaves, threadIdx.x);
        __syncthreads();
    }
    const uint16_t* kb = reinterpret_cast<const uint16_t*>(a.k) + (int64_t)k0 * a.k_stride +
                         kv_head * a.head_dim;
    const uint16_t* vb = reinterpret_cast<const uint16_t*>(a.v) + (int64_t)k0 * a.v_stride +
                         kv_head * a.head_dim;
    const int64_t k_pitch = a.k_stride * 2, v_pitch = a.v_stride * 2;
    const bool near = max(k_pitch, v_pitch) <= T::kMaxPitch;
    const uint32_t k_off = T::lane_offset(wave, lane, k_pitch);
    const uint32_t v_off = T::lane_offset(wave, lane, v_pitch);
    const bool on = T::lane_chunk(wave, lane) < chunks;
    // rows past the item's last key repeat it; their weight is 0
    auto fetch = [&](int key) {
        uint4* kd = kt[key / kKeys & 1];
        uint4* vd = vt[key / kKeys % 3];
        if (near && begin + key + kKeys <= nk) {
            T::template load_rows<kKeys, kWaves>(kd, wave, kb + (int64_t)(begin + key) * a.k_stride,
                                                 k_pitch, k_off, on);
            T::template load_rows<kKeys, kWaves>(vd, wave, vb + (int64_t)(begin + key) * a.v_stride,
                                                 v_pitch, v_off, on);
            return;
        }
        T::template load<kKeys, kWaves>(kd, wave, lane, chunks, [&](int r) {
            return reinterpret_cast<const uint4*>(
                kb + (int64_t)min(begin + key + r, nk - 1) * a.k_stride);
        });
        T::template load<kKeys, kWaves>(vd, wave, lane, chunks, [&](int r) {
            return reinterpret_cast<const uint4*>(
                vb + (int64_t)min(begin + key + r, nk - 1) * a.v_stride);
        });
    };
    const int span = end - begin;
    // the first tile travels while the queries are loaded
    if (span > 0) fetch(0);
    bf16x8_t q[T::kSteps];
    load_query<HD>(q,
                   reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(a.q) +
                                                  (int64_t)(q0 + (int)token) * a.q_stride +
                                                  head * a.head_dim),
                   live, chunks, lane);
    settle(q);

    // Tile by tile (`key` counts from `begin`): the scores of a tile, then
    // the second product of the tile before it in between this tile's
    // exponentials, so that the matrix cores run under them. V therefore
    // stays a tile longer than K (three buffers, two).
    bf16x8_t p[4];
    auto step = [&](auto first, int key) {
        tile_barrier();
        if (key + kKeys < span) fetch(key + kKeys);
        f32x16 sc[2];
        st.scores(sc, q, kt[key / kKeys & 1], lane);
        if (begin + key + kKeys > all_see) st.mask(sc, begin + key, limit, lane);
        const uint4* before = vt[(key / kKeys + 2) % 3];
        if (st.exceeds(sc, c)) {
            if constexpr (!decltype(first)::value) {
                // what the old maximum scaled goes in before the new one does
                st.add(p, before, lane);
#pragma unroll
                for (int i = 0; i < 4; ++i) p[i] = bf16x8_t{};
            }
            st.raise(sc, c);
        }
        if constexpr (decltype(first)::value) st.exponentials(sc, p, c);
        else st.exponentials_and_add(sc, p, before, c, lane);
    };
    if (span > 0) {
        step(std::true_type{}, 0);
        int key = kKeys;
        for (; key < span; key += kKeys) step(std::false_type{}, key);
        st.add(p, vt[(key / kKeys + 2) % 3], lane);
    }

    float own;
    const float other = other_half(st.l, own);
    const float l = own + other;
    const int64_t out_row = (int64_t)(q0 + (int)token) * a.heads + head;
    if (which >= 0) {
        if (live)
            store_part<HD>(f, st,
                           ((int64_t)(unit - f.whole) * f.parts + which) * kRows + row - row0, l,
                           lane);
        return;
    }
    if (a.lse && live && lane < 32)
        a.lse[out_row] = l == 0.f ? -INFINITY : st.m * a.scale + kLn2 * __builtin_amdgcn_logf(l);
    tile_barrier();                          // every wave is done with the tiles
    const float by = l == 0.f ? 0.f : 1.0f / l;
    uint4* stage = wave < 2 ? kt[wave] : vt[wave - 2];
    store_rows<HD>(st.o, by, stage, chunks, lane, [&](int r) -> uint4* {
        const uint32_t at = row0 + 32 * wave + r;
        if (at >= rows) return nullptr;
        uint32_t t, m;
        f.group.split(at, t, m);
        return reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.out) +
                                        (int64_t)(q0 + (int)t) * a.out_stride +
                                        (kv_head * f.group.size + m) * a.head_dim);
    });
}

// Items of at most 32 rows (single tokens with their groups): every wave of
// the workgroup holds the same rows and walks keys of its own, two tiles of 32
// keys in flight each, and the waves' states are joined in LDS. No barrier
// stands in the loop. Bound by K and V, read once: four tokens of 16 heads over
// 40,001 keys of 4 heads take 19 us (4.3 TB/s, of which the launch, the first
// loads and the join are some 5 us) and combine_kernel 4.
template <int HD>
__global__ __launch_bounds__(64 * kWaves, 1) void attention_single_kernel(FwdArgs f) {
    using T = Tile<HD>;
    constexpr int kTile = kSingleKeys * T::kChunks;
    constexpr int kLoads = 2 * kSingleKeys * T::kChunks / 64;
    __shared__ alignas(kTileAlign) uint4 tiles[kWaves][2][2][kTile];  // [wave][buffer][k, v]
    __shared__ float2 ml[kWaves][32];
    const AttnArgs& a = f.a;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int chunks = a.head_dim >> 3;
    // the same number of keys for every workgroup, however long the items are
    const int nth = blockIdx.x / a.kv_heads;
    const int item = item_of_tile(f.tiles, a.batch, nth);
    const int which = nth - f.tiles.start[item];
    const bool split = f.tiles.start[item + 1] - f.tiles.start[item] > 1;
    const Unit u(a, item, blockIdx.x - nth * a.kv_heads, f.group.size);
    const int kv_head = u.kv_head, q0 = u.q0, nq = u.nq, k0 = u.k0, nk = u.nk;
    const uint32_t row = lane & 31, rows = u.rows;
    const bool live = row < rows;
    uint32_t token, member;
    f.group.split(live ? row : 0, token, member);
    const int head = kv_head * f.group.size + member;

    const int begin = (int)min((int64_t)which * f.share, (int64_t)nk);
    const int end = (int)min((int64_t)begin + f.share, (int64_t)nk);
    const int limit = a.causal && live ? min(end, (int)token + nk - nq + 1) : end;
    const int all_see = __builtin_amdgcn_readfirstlane(limit);
    const float c = a.scale * kLog2e;

    Softmax<HD> st;
    st.init();
    if (chunks < T::kChunks) {
        T::clear(tiles[wave][0][0], 4 * kSingleKeys, 64, lane);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
    const uint16_t* kb = reinterpret_cast<const uint16_t*>(a.k) + (int64_t)k0 * a.k_stride +
                         kv_head * a.head_dim;
    const uint16_t* vb = reinterpret_cast<const uint16_t*>(a.v) + (int64_t)k0 * a.v_stride +
                         kv_head * a.head_dim;
    auto fetch = [&](int buf, int key) {
        T::template load<kSingleKeys, 1>(tiles[wave][buf][0], 0, lane, chunks, [&](int r) {
            return reinterpret_cast<const uint4*>(kb + (int64_t)min(key + r, nk - 1) * a.k_stride);
        });
        T::template load<kSingleKeys, 1>(tiles[wave][buf][1], 0, lane, chunks, [&](int r) {
            return reinterpret_cast<const uint4*>(vb + (int64_t)min(key + r, nk - 1) * a.v_stride);
        });
    };
    const int first = begin + wave * kSingleKeys;
    constexpr int kStep = kWaves * kSingleKeys;
    if (first < end) fetch(0, first);        // (ahead of the queries)
    bf16x8_t q[T::kSteps];
    load_query<HD>(q,
                   reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(a.q) +
                                                  (int64_t)(q0 + (int)token) * a.q_stride +
                                                  head * a.head_dim),
                   live, chunks, lane);
    settle(q);
    int buf = 0;
    for (int key = first; key < end; key += kStep, buf ^= 1) {
        // the wave's reads of the other buffer are done before it is filled
        if (key + kStep < end) {
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            fetch(buf ^ 1, key + kStep);
            wave_wait<kLoads>();
        } else {
            wave_wait<0>();
        }
        st.attend(q, tiles[wave][buf][0], tiles[wave][buf][1], key, limit,
                  key + kSingleKeys > all_see, c, lane);
    }

    // Join the waves: each scales its state to the common maximum; wave 0
    // adds the others' O from LDS.
    float own;
    const float other = other_half(st.l, own);
    float l = own + other;
    if (lane < 32) ml[wave][lane] = make_float2(st.m, l);
    __syncthreads();
    float m = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) m = fmaxf(m, ml[w][row].x);
    const float by = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f((st.m - m) * c);
    l = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        const float2 v = ml[w][row];
        // (no maximum: the sums are 0, or NaN where the scores were)
        l += m == -INFINITY ? v.y : v.y * __builtin_amdgcn_exp2f((v.x - m) * c);
    }
    // [wave][register][lane]; the tiles are no longer read
    float* joint = reinterpret_cast<float*>(&tiles[0][0][0][0]);
    static_assert((kWaves - 1) * 16 * T::kBlocks * 64 * 4 <= kWaves * 4 * kTile * 16, "joint");
    if (wave) {
#pragma unroll
        for (int b = 0; b < T::kBlocks; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                joint[(((wave - 1) * T::kBlocks + b) * 16 + i) * 64 + lane] = st.o[b][i] * by;
    }
    __syncthreads();
    if (wave) return;
#pragma unroll
    for (int b = 0; b < T::kBlocks; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float s = st.o[b][i] * by;
#pragma unroll
            for (int w = 0; w < kWaves - 1; ++w)
                s += joint[((w * T::kBlocks + b) * 16 + i) * 64 + lane];
            st.o[b][i] = s;
        }
    st.m = m;
    const int64_t out_row = (int64_t)(q0 + (int)token) * a.heads + head;
    if (!live) return;
    if (split) {
        store_part<HD>(f, st, (int64_t)blockIdx.x * kSingleRows + row, l, lane);
        return;
    }
    if (a.lse && lane < 32)
        a.lse[out_row] = l == 0.f ? -INFINITY : m * a.scale + kLn2 * __builtin_amdgcn_logf(l);
    const float inv = l == 0.f ? 0.f : 1.0f / l;
    uint16_t* o = reinterpret_cast<uint16_t*>(a.out) + (int64_t)(q0 + (int)token) * a.out_stride +
                  head * a.head_dim;
    const int h = lane >> 5;
#pragma unroll
    for (int b = 0; b < T::kBlocks; ++b)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int d = 32 * b + 8 * j + 4 * h;
            if (d < a.head_dim)
                *reinterpret_cast<uint2*>(o + d) =
                    make_uint2(pack_bf16x2(st.o[b][4 * j] * inv, st.o[b][4 * j + 1] * inv),
                               pack_bf16x2(st.o[b][4 * j + 2] * inv, st.o[b][4 * j + 3] * inv));
        }
}

// Items of at most 32 NB keys (global tokens): no loop at all. Bound by q in
// and out out, which both go through the wave's LDS tile in whole rows: with 16
// bytes of every row per instruction, as the operands lie, the lines of 32 rows
// do not survive in L1 (100,000 tokens of 12 heads over 5 keys: 156 us, and 118
// through LDS, 5.2 TB/s). Several row tiles per wave, the next one's queries
// loaded under one, were slower (129 us with 3, 144 with 6) than more
// workgroups.
template <int HD, int NB>
__global__ __launch_bounds__(64 * kWaves, NB == 1 ? 3 : 2) void attention_few_kernel(FwdArgs f,
                                                                                     bool nt) {
    using T = Tile<HD>;
    __shared__ alignas(kTileAlign) uint4 kt[32 * NB * T::kChunks];
    __shared__ alignas(kTileAlign) uint4 vt[32 * NB * T::kChunks];
    __shared__ alignas(kTileAlign) uint4 rows_lds[kWaves][32 * T::kChunks];
    const AttnArgs& a = f.a;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int chunks = a.head_dim >> 3;
    const Unit u(f, blockIdx.x, kRows);
    const int kv_head = u.kv_head, q0 = u.q0, nq = u.nq, k0 = u.k0, nk = u.nk;
    const int head0 = kv_head * (int)f.group.size;

    if (chunks < T::kChunks || nk == 0) {    // (without keys, zeros stand for them)
        T::clear(kt, 32 * NB, 64 * kWaves, threadIdx.x);
        T::clear(vt, 32 * NB, 64 * kWaves, threadIdx.x);
        T::clear(rows_lds[0], 32 * kWaves, 64 * kWaves, threadIdx.x);
        __syncthreads();
    }
    const uint16_t* kb = reinterpret_cast<const uint16_t*>(a.k) + (int64_t)k0 * a.k_stride +
                         kv_head * a.head_dim;
    const uint16_t* vb = reinterpret_cast<const uint16_t*>(a.v) + (int64_t)k0 * a.v_stride +
                         kv_head * a.head_dim;
    if (nk > 0) {
        T::template load<32 * NB, kWaves>(kt, wave, lane, chunks, [&](int r) {
            return reinterpret_cast<const uint4*>(kb + (int64_t)min(r, nk - 1) * a.k_stride);
        });
        T::template load<32 * NB, kWaves>(vt, wave, lane, chunks, [&](int r) {
            return reinterpret_cast<const uint4*>(vb + (int64_t)min(r, nk - 1) * a.v_stride);
        });
    }
    const float c = a.scale * kLog2e;
    // an element's place in q or out by its row
    auto place = [&](uint32_t row, int64_t stride) {
        uint32_t token, member;
        f.group.split(row, token, member);
        return (int64_t)(q0 + (int)token) * stride + (head0 + (int)member) * a.head_dim;
    };
    const uint32_t row0 = u.row0 + 32 * wave;
    uint4* tile = rows_lds[wave];
    if (row0 < u.rows)                       // rows past the last repeat it
        T::template load<32, 1>(tile, 0, lane, chunks, [&](int r) {
            return reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(a.q) +
                                                  place(min(row0 + r, u.rows - 1), a.q_stride));
        });
    tile_barrier();
    if (row0 >= u.rows) return;
    const uint32_t q_at = T::row_base(tile, lane);
    bf16x8_t q[T::kSteps];
#pragma unroll
    for (int k = 0; k < T::kSteps; ++k) q[k] = T::row_frag(q_at, 0, k);
    const uint32_t row = row0 + (lane & 31);
    const bool live = row < u.rows;
    uint32_t token, member;
    f.group.split(live ? row : 0, token, member);
    const int limit = a.causal && live ? min(nk, (int)token + nk - nq + 1) : nk;

    const uint32_t k_at = T::row_base(kt, lane);
    f32x16 s[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) s[b] = zero16();
#pragma unroll
    for (int k = 0; k < T::kSteps; ++k)
#pragma unroll
        for (int b = 0; b < NB; ++b) s[b] = mfma(T::row_frag(k_at, 32 * b, k), q[k], s[b]);
    Softmax<HD> st;
    st.init();
    st.mask(s, 0, limit, lane);
    const float top = st.top(s);
    const float base = top == -INFINITY ? 0.f : top * c;
    bf16x8_t p[2 * NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            s[b][i] = __builtin_amdgcn_exp2f(fmaf(s[b][i], c, -base));
            st.l += s[b][i];
        }
        p[2 * b] = acc_frag(s[b], 0);
        p[2 * b + 1] = acc_frag(s[b], 1);
    }
    const uint32_t v_at = T::tr_base(vt, lane);
#pragma unroll
    for (int t = 0; t < 2 * NB; ++t)
#pragma unroll
        for (int d = 0; d < T::kBlocks; ++d)
            st.o[d] = mfma(T::tr_frag(v_at, 16 * t, d), p[t], st.o[d]);
    float own;
    const float other = other_half(st.l, own);
    const float l = own + other;
    stage_rows<HD>(st.o, l == 0.f ? 0.f : 1.0f / l, tile, chunks, lane);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    if (a.lse && live && lane < 32)
        a.lse[(int64_t)(q0 + (int)token) * a.heads + head0 + member] =
            l == 0.f ? -INFINITY : top * a.scale + kLn2 * __builtin_amdgcn_logf(l);
    write_rows<HD>(tile, chunks, lane, [&](int r) -> uint4* {
        if (row0 + r >= u.rows) return nullptr;
        return reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.out) +
                                        place(row0 + r, a.out_stride));
    }, nt);
}

// Joins the parts of a row, one wave per row: lane p weighs part p, then each
// half adds every other part, 4 columns a lane.
__global__ __launch_bounds__(256) void combine_kernel(FwdArgs f, int per_tile, bool single) {
    const AttnArgs& a = f.a;
    const int lane = threadIdx.x & 63, h = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int tail = blockIdx.x * 4 / per_tile;
    const int r = (blockIdx.x * 4 + wave) % per_tile;
    const Unit u = single ? Unit(a, tail / a.kv_heads, tail % a.kv_heads, f.group.size)
                          : Unit(f, f.whole + tail, per_tile);
    const uint32_t row = u.row0 + r;
    if (row >= u.rows) return;
    const float c = a.scale * kLog2e;
    // a part's slot: the parts of a unit in turn, or (single) of the key heads
    const int before = f.tiles.start[u.item];
    const int parts = single ? f.tiles.start[u.item + 1] - before : f.parts;
    if (single && parts == 1) return;
    const int64_t slot = single ? (int64_t)before * a.kv_heads + u.kv_head
                                : (int64_t)tail * f.parts;
    const int64_t first = slot * per_tile + r, step = (single ? a.kv_heads : 1) * per_tile;
    const float2 ml = lane < parts ? f.part_ml[first + lane * step]
                                   : make_float2(-INFINITY, 0.f);
    const float m = lane_max(ml.x);
    const float weight = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f((ml.x - m) * c);
    const float l = lane_sum<64>(ml.y * weight);
    const int d = (lane & 31) * 4;
    const float* from = f.part_o + first * a.head_dim + (d < a.head_dim ? d : 0);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int p = 0; p < parts; p += 8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {            // (four loads in flight)
            const int mine = p + 2 * i + h, there = min(mine, parts - 1);
            const float other = __shfl(weight, there);
            const float w = mine < parts ? other : 0.f;
            const float4 v = *reinterpret_cast<const float4*>(from + there * step * a.head_dim);
            o.x += v.x * w;
            o.y += v.y * w;
            o.z += v.z * w;
            o.w += v.w * w;
        }
    }
    float own;
    o.x = other_half(o.x, own) + own;
    o.y = other_half(o.y, own) + own;
    o.z = other_half(o.z, own) + own;
    o.w = other_half(o.w, own) + own;
    const float inv = l == 0.f ? 0.f : 1.0f / l;
    uint32_t token, member;
    f.group.split(row, token, member);
    const int head = u.kv_head * f.group.size + member;
    const int64_t at = u.q0 + (int)token;
    if (h == 0 && d < a.head_dim)
        *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.out) + at * a.out_stride +
                                  head * a.head_dim + d) =
            make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
    if (a.lse && lane == 0)
        a.lse[at * a.heads + head] =
            l == 0.f ? -INFINITY : m * a.scale + kLn2 * __builtin_amdgcn_logf(l);
}

template <int HD>
hipError_t forward_as(const FwdArgs& f, const AttnPlan& p, int blocks, hipStream_t s) {
    const dim3 grid((unsigned)blocks), threads(64 * kWaves);
    // where q and out do not fit the last-level cache anyway, out goes past it
    const int64_t moved = (int64_t)f.a.q_items.start[f.a.batch] * f.a.heads * f.a.head_dim * 4;
    const bool nt = moved > (int64_t(256) << 20);
    if (p.single)
        attention_single_kernel<HD><<<grid, threads, 0, s>>>(f);
    else if (p.few == 1)
        attention_few_kernel<HD, 1><<<grid, threads, 0, s>>>(f, nt);
    else if (p.few == 2)
        attention_few_kernel<HD, 2><<<grid, threads, 0, s>>>(f, nt);
    else
        attention_kernel<HD><<<grid, threads, 0, s>>>(f);
    return hipGetLastError();
}

// Parts of the single-token kernel, of `share` keys each: one per CU where the
// keys are long enough (its tiles fill a CU's LDS), at least 256 keys.
int single_parts(const AttnArgs& a, int64_t share, ItemTable* start) {
    int64_t at = 0;
    for (int b = 0; b < a.batch; ++b) {
        start->start[b] = (int32_t)at;
        const int64_t keys = a.k_items.start[b + 1] - a.k_items.start[b];
        const bool rows = a.q_items.start[b + 1] > a.q_items.start[b];
        at += rows ? std::max<int64_t>(1, (keys + share - 1) / share) : 0;
    }
    for (int b = a.batch; b <= P3D_MAX_BATCH; ++b) start->start[b] = (int32_t)at;
    return (int)at;
}

}  // namespace

// The units of a launch fill the chip in rounds of `slots` workgroups. The
// units past the last full round are cut along the keys into as many parts as
// fit one round (at least 256 keys each), so that a last round of a few long
// units does not run on a few CUs alone. Causal launches of more than a round
// end on their shortest tiles and are left whole.
AttnPlan attention_plan(const AttnArgs& a) {
    AttnPlan p{};
    const int group = a.heads / a.kv_heads;
    int64_t most_rows = 0, most_keys = 0;
    for (int32_t b = 0; b < a.batch; ++b) {
        most_rows = std::max<int64_t>(
            most_rows, (int64_t)(a.q_items.start[b + 1] - a.q_items.start[b]) * group);
        most_keys = std::max<int64_t>(most_keys, a.k_items.start[b + 1] - a.k_items.start[b]);
    }
    const size_t row_bytes = a.head_dim * sizeof(float) + sizeof(float2);
    ItemTable tiles;
    p.single = most_rows <= kSingleRows;
    p.per_tile = p.single ? kSingleRows : kRows;
    p.parts = 1;
    p.forward_bytes = 256;
    if (p.single) {
        cut_items(a.q_items, a.batch, group, p.per_tile, &tiles);
        p.units = tiles.start[a.batch] * a.kv_heads;
        int64_t share = std::max<int64_t>(
            256, ((int64_t)a.k_items.start[a.batch] * a.kv_heads / kComputeUnits + 127) / 128 * 128);
        share = std::max(share, (most_keys / kMostParts + 128) / 128 * 128);
        // uncut, short items need no second launch (one token of 8 heads on 4:
        // 12.7 us against 15.3 with 512 keys, 16.6 against 15.5 with 1024)
        if (most_keys <= 512) share = std::max<int64_t>(share, 512);
        while (single_parts(a, share, &tiles) * a.kv_heads > std::max(p.units, kComputeUnits))
            share += (share / 16 + 127) / 128 * 128;
        p.share = (int32_t)share;
        const int parts = single_parts(a, share, &tiles) * a.kv_heads;
        p.whole = parts == p.units ? p.units : 0;
        if (p.whole == 0) p.forward_bytes += (size_t)parts * p.per_tile * row_bytes;
    } else {
        cut_items(a.q_items, a.batch, group, p.per_tile, &tiles);
        p.few = most_keys <= 32 ? 1 : most_keys <= 64 ? 2 : 0;
        p.units = tiles.start[a.batch] * a.kv_heads;
        // workgroups a CU holds, by LDS and registers
        const int slots = kComputeUnits * (a.head_dim <= 64 ? 3 : 2);
        p.whole = p.few || (a.causal && p.units >= slots) ? p.units : p.units / slots * slots;
        if (p.whole < p.units)
            p.parts = (int32_t)std::min<int64_t>(
                {slots / (p.units - p.whole), most_keys / 256, kMostParts});
        if (p.parts <= 1) {
            p.whole = p.units;
            p.parts = 1;
        }
        p.forward_bytes += (size_t)(p.units - p.whole) * p.parts * p.per_tile * row_bytes;
    }
    plan_attention_backward(a, &p);
    return p;
}

hipError_t launch_attention(const AttnArgs& a, const AttnPlan& p, void* ws, hipStream_t s) {
    if (p.units == 0) return hipSuccess;
    FwdArgs f;
    f.a = a;
    f.group = group_of(a);
    f.whole = p.whole;
    f.parts = p.parts;
    f.share = p.share;
    const int tail = p.units - p.whole;
    int slots = tail * p.parts;
    if (p.single) slots = single_parts(a, p.share, &f.tiles) * a.kv_heads;
    else cut_items(a.q_items, a.batch, f.group.size, p.per_tile, &f.tiles);
    f.part_o = static_cast<float*>(ws);
    f.part_ml = reinterpret_cast<float2*>(f.part_o + (int64_t)slots * p.per_tile * a.head_dim);
    const int blocks = p.single ? slots : p.whole + slots;
    const hipError_t e = a.head_dim <= 64   ? forward_as<64>(f, p, blocks, s)
                         : a.head_dim <= 96 ? forward_as<96>(f, p, blocks, s)
                                            : forward_as<128>(f, p, blocks, s);
    if (e != hipSuccess || tail == 0) return e;
    const int joined = p.single ? a.batch * a.kv_heads : tail;
    combine_kernel<<<dim3((unsigned)(joined * (p.per_tile / 4))), dim3(256), 0, s>>>(
        f, p.per_tile, p.single);
    return hipGetLastError();
}

}  // namespace p3d
