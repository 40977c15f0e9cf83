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
// With few rows and many keys the keys are cut into `splits` parts, each of
// which leaves (m, l, O) in the workspace, joined by combine_kernel.
#include <algorithm>

#include "attn_tile.h"

namespace p3d {

namespace {

using namespace attn;

constexpr int kKeys = 64;                // keys per tile of attention_kernel
constexpr int kWaves = 4;
constexpr int kRows = 32 * kWaves;       // query rows per workgroup
constexpr int kSingleKeys = 32;          // keys per wave tile of attention_single_kernel

struct FwdArgs {
    AttnArgs a;
    ItemTable tiles;                     // first row tile of every item
    Group group;
    int splits;
    float* part_o;                       // [splits][nq * heads][head_dim]
    float2* part_ml;                     // [splits][nq * heads]
};

// One row tile's running softmax: lane l's query is l % 32, and the two
// halves hold different keys (and different columns of O).
template <int HD>
struct Softmax {
    f32x16 o[Tile<HD>::kBlocks];
    float m, l;                          // l: this half's share

    __device__ __forceinline__ void init() {
#pragma unroll
        for (int b = 0; b < Tile<HD>::kBlocks; ++b) o[b] = zero16();
        m = -INFINITY;
        l = 0.f;
    }

    // Keys key0 .. key0 + 32 NB - 1 in the tiles' rows 0 ..; those at or past
    // `limit` are not seen. c = scale log2(e).
    template <int NB>
    __device__ __forceinline__ void attend(const bf16x8_t (&q)[Tile<HD>::kSteps], const uint4* kt,
                                           const uint4* vt, int key0, int limit, bool masked,
                                           float c, int lane) {
        using T = Tile<HD>;
        const int h = lane >> 5;
        f32x16 s[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            s[b] = zero16();
#pragma unroll
            for (int k = 0; k < T::kSteps; ++k)
                s[b] = mfma(T::row_frag(kt, 32 * b, lane, k), q[k], s[b]);
        }
        if (masked) {
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (key0 + 32 * b + acc_row(i, h) >= limit) s[b][i] = -INFINITY;
        }
        float top = -INFINITY;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i) top = fmaxf(top, s[b][i]);
        float own;
        const float other = other_half(top, own);
        top = fmaxf(own, other);
        if (__any((top - m) * c > 8.0f || (m == -INFINITY && top > m))) {
            const float raised = fmaxf(m, top);
            const float by = raised == -INFINITY ? 0.f
                                                 : __builtin_amdgcn_exp2f((m - raised) * c);
            m = raised;
            l *= by;
#pragma unroll
            for (int b = 0; b < T::kBlocks; ++b)
#pragma unroll
                for (int i = 0; i < 16; ++i) o[b][i] *= by;
        }
        const float base = m == -INFINITY ? 0.f : m * c;
        float sum = 0.f;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                s[b][i] = __builtin_amdgcn_exp2f(s[b][i] * c - base);
                sum += s[b][i];
            }
        l += sum;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const bf16x8_t p = acc_frag(s[b], t);
#pragma unroll
                for (int d = 0; d < T::kBlocks; ++d)
                    o[d] = mfma(T::tr_frag(vt, 32 * b + 16 * t, lane, d), p, o[d]);
            }
    }
};

// A part's (m, l, O) to the workspace; `row` is token * heads + head.
template <int HD>
__device__ __forceinline__ void store_part(const FwdArgs& f, const Softmax<HD>& st, int part,
                                           int64_t row, int64_t rows, float l, int lane) {
    const int h = lane >> 5, hd = f.a.head_dim;
    const int64_t at = part * rows + row;
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
    __shared__ uint4 kt[2][kKeys * T::kChunks];
    __shared__ uint4 vt[2][kKeys * T::kChunks];
    const AttnArgs& a = f.a;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int chunks = a.head_dim >> 3;

    // Row tiles of an item, the longest causal ones first, key heads fastest:
    // workgroups go to the XCDs in turn, so with 8 (or 16, 24, ...) key heads
    // an XCD's L2 holds the same heads throughout.
    const int tile = blockIdx.x / a.kv_heads, kv_head = blockIdx.x - tile * a.kv_heads;
    const int item = item_of_tile(f.tiles, a.batch, tile);
    const int tiles = f.tiles.start[item + 1] - f.tiles.start[item];
    const int nth = tile - f.tiles.start[item];
    const uint32_t row0 = (uint32_t)(a.causal ? tiles - 1 - nth : nth) * kRows;
    const int q0 = a.q_items.start[item], nq = a.q_items.start[item + 1] - q0;
    const int k0 = a.k_items.start[item], nk = a.k_items.start[item + 1] - k0;
    const uint32_t rows = (uint32_t)nq * f.group.size;

    // this lane's query
    const uint32_t row = row0 + 32 * wave + (lane & 31);
    const bool live = row < rows;
    uint32_t token, member;
    f.group.split(live ? row : 0, token, member);
    const int head = kv_head * f.group.size + member;
    bf16x8_t q[T::kSteps];
    load_query<HD>(q,
                   reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(a.q) +
                                                  (int64_t)(q0 + (int)token) * a.q_stride +
                                                  head * a.head_dim),
                   live, chunks, lane);

    // keys of this part, and those this workgroup and this lane see
    int part = (nk + f.splits - 1) / f.splits;
    part = (part + kKeys - 1) / kKeys * kKeys;
    const int begin = (int)min((int64_t)blockIdx.y * part, (int64_t)nk);
    int end = (int)min((int64_t)begin + part, (int64_t)nk);
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
        for (int i = 0; i < 2; ++i) {
            T::clear(kt[i], kKeys, 64 * kWaves, threadIdx.x);
            T::clear(vt[i], kKeys, 64 * kWaves, threadIdx.x);
        }
        __syncthreads();
    }
    const uint16_t* kb = reinterpret_cast<const uint16_t*>(a.k) + (int64_t)k0 * a.k_stride +
                         kv_head * a.head_dim;
    const uint16_t* vb = reinterpret_cast<const uint16_t*>(a.v) + (int64_t)k0 * a.v_stride +
                         kv_head * a.head_dim;
    // rows past the item's last key repeat it; their weight is 0
    auto fetch = [&](int buf, int key) {
        T::template load<kKeys, kWaves>(kt[buf], wave, lane, chunks, [&](int r) {
            return reinterpret_cast<const uint4*>(kb + (int64_t)min(key + r, nk - 1) * a.k_stride);
        });
        T::template load<kKeys, kWaves>(vt[buf], wave, lane, chunks, [&](int r) {
            return reinterpret_cast<const uint4*>(vb + (int64_t)min(key + r, nk - 1) * a.v_stride);
        });
    };
    if (begin < end) fetch(0, begin);
    int buf = 0;
    for (int key = begin; key < end; key += kKeys, buf ^= 1) {
        tile_barrier();
        if (key + kKeys < end) fetch(buf ^ 1, key + kKeys);
        st.template attend<2>(q, kt[buf], vt[buf], key, limit, key + kKeys > all_see, c, lane);
    }

    float own;
    const float other = other_half(st.l, own);
    const float l = own + other;
    const int64_t out_row = (int64_t)(q0 + (int)token) * a.heads + head;
    if (f.splits > 1) {
        if (live)
            store_part<HD>(f, st, blockIdx.y, out_row,
                           (int64_t)a.q_items.start[a.batch] * a.heads, l, lane);
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
// stands in the loop.
template <int HD>
__global__ __launch_bounds__(64 * kWaves, 1) void attention_single_kernel(FwdArgs f) {
    using T = Tile<HD>;
    constexpr int kTile = kSingleKeys * T::kChunks;
    constexpr int kLoads = 2 * kSingleKeys * T::kChunks / 64;
    __shared__ uint4 tiles[kWaves][2][2][kTile];         // [wave][buffer][k, v]
    __shared__ float2 ml[kWaves][32];
    const AttnArgs& a = f.a;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int chunks = a.head_dim >> 3;
    const int item = blockIdx.x / a.kv_heads, kv_head = blockIdx.x - item * a.kv_heads;
    const int q0 = a.q_items.start[item], nq = a.q_items.start[item + 1] - q0;
    const int k0 = a.k_items.start[item], nk = a.k_items.start[item + 1] - k0;
    const uint32_t rows = (uint32_t)nq * f.group.size;
    if (rows == 0) return;
    const uint32_t row = lane & 31;
    const bool live = row < rows;
    uint32_t token, member;
    f.group.split(live ? row : 0, token, member);
    const int head = kv_head * f.group.size + member;

    bf16x8_t q[T::kSteps];
    load_query<HD>(q,
                   reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(a.q) +
                                                  (int64_t)(q0 + (int)token) * a.q_stride +
                                                  head * a.head_dim),
                   live, chunks, lane);
    int part = (nk + f.splits - 1) / f.splits;
    part = (part + kSingleKeys - 1) / kSingleKeys * kSingleKeys;
    const int begin = (int)min((int64_t)blockIdx.y * part, (int64_t)nk);
    const int end = (int)min((int64_t)begin + part, (int64_t)nk);
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
    if (first < end) fetch(0, first);
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
        st.template attend<1>(q, tiles[wave][buf][0], tiles[wave][buf][1], key, limit,
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
        l += m == -INFINITY ? 0.f : v.y * __builtin_amdgcn_exp2f((v.x - m) * c);
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
    if (f.splits > 1) {
        store_part<HD>(f, st, blockIdx.y, out_row, (int64_t)a.q_items.start[a.batch] * a.heads, l,
                       lane);
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

// Joins the parts of a row, 32 lanes per row, 4 columns a lane.
__global__ __launch_bounds__(256) void combine_kernel(FwdArgs f, int64_t rows) {
    const AttnArgs& a = f.a;
    const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int d = (threadIdx.x & 31) * 4;
    if (row >= rows) return;
    const float c = a.scale * kLog2e;
    float m = -INFINITY;
    for (int s = 0; s < f.splits; ++s) m = fmaxf(m, f.part_ml[s * rows + row].x);
    float l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    if (m != -INFINITY) {
        for (int s = 0; s < f.splits; ++s) {
            const float2 v = f.part_ml[s * rows + row];
            const float by = __builtin_amdgcn_exp2f((v.x - m) * c);
            l += v.y * by;
            if (d < a.head_dim) {
                const float4 p = *reinterpret_cast<const float4*>(
                    f.part_o + (s * rows + row) * a.head_dim + d);
                o.x += p.x * by;
                o.y += p.y * by;
                o.z += p.z * by;
                o.w += p.w * by;
            }
        }
    }
    const float inv = l == 0.f ? 0.f : 1.0f / l;
    const int64_t token = row / a.heads;
    const int head = (int)(row - token * a.heads);
    if (d < a.head_dim)
        *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.out) + token * a.out_stride +
                                  head * a.head_dim + d) =
            make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
    if (a.lse && d == 0)
        a.lse[row] = l == 0.f ? -INFINITY : m * a.scale + kLn2 * __builtin_amdgcn_logf(l);
}

template <int HD>
hipError_t forward_as(const FwdArgs& f, const AttnPlan& p, int tiles, hipStream_t s) {
    if (p.single)
        attention_single_kernel<HD><<<dim3((unsigned)(f.a.batch * f.a.kv_heads), (unsigned)f.splits),
                                      dim3(64 * kWaves), 0, s>>>(f);
    else
        attention_kernel<HD><<<dim3((unsigned)tiles * f.a.kv_heads, (unsigned)f.splits),
                               dim3(64 * kWaves), 0, s>>>(f);
    return hipGetLastError();
}

}  // namespace

AttnPlan attention_plan(const AttnArgs& a) {
    AttnPlan p{};
    const int group = a.heads / a.kv_heads;
    int64_t most_rows = 0, most_keys = 0;
    for (int32_t b = 0; b < a.batch; ++b) {
        most_rows = std::max<int64_t>(
            most_rows, (int64_t)(a.q_items.start[b + 1] - a.q_items.start[b]) * group);
        most_keys = std::max<int64_t>(most_keys, a.k_items.start[b + 1] - a.k_items.start[b]);
    }
    p.single = most_rows <= 32;
    ItemTable tiles;
    cut_items(a.q_items, a.batch, group, kRows, &tiles);
    // Workgroups before a split. Fewer than the CUs: parts of at least 256
    // keys, about two workgroups per CU (one of the single-token kernel,
    // whose tiles fill a CU's LDS).
    const int64_t blocks = (int64_t)(p.single ? a.batch : tiles.start[a.batch]) * a.kv_heads;
    p.splits = 1;
    if (blocks > 0 && blocks < kComputeUnits) {
        const int64_t wanted = ((p.single ? 1 : 2) * kComputeUnits + blocks - 1) / blocks;
        p.splits = (int32_t)std::max<int64_t>(1, std::min<int64_t>(wanted, most_keys / 256));
    }
    const int64_t rows = (int64_t)a.q_items.start[a.batch] * a.heads;
    p.forward_bytes = 256;
    if (p.splits > 1)
        p.forward_bytes += (size_t)p.splits * rows * (a.head_dim * sizeof(float) + sizeof(float2));
    plan_attention_backward(a, &p);
    return p;
}

hipError_t launch_attention(const AttnArgs& a, const AttnPlan& p, void* ws, hipStream_t s) {
    const int64_t rows = (int64_t)a.q_items.start[a.batch] * a.heads;
    if (rows == 0) return hipSuccess;
    FwdArgs f;
    f.a = a;
    f.group = group_of(a);
    cut_items(a.q_items, a.batch, f.group.size, kRows, &f.tiles);
    f.splits = p.splits;
    f.part_o = static_cast<float*>(ws);
    f.part_ml = reinterpret_cast<float2*>(static_cast<float*>(ws) +
                                          (int64_t)p.splits * rows * a.head_dim);
    const int tiles = f.tiles.start[a.batch];
    hipError_t e = a.head_dim <= 64   ? forward_as<64>(f, p, tiles, s)
                   : a.head_dim <= 96 ? forward_as<96>(f, p, tiles, s)
                                      : forward_as<128>(f, p, tiles, s);
    if (e != hipSuccess || p.splits == 1) return e;
    combine_kernel<<<dim3((unsigned)((rows + 7) / 8)), dim3(256), 0, s>>>(f, rows);
    return hipGetLastError();
}

}  // namespace p3d
