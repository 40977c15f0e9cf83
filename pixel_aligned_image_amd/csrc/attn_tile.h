// attn_tile.h -- tiles of the attention kernels: the LDS layout, the
// direct-to-LDS loads and the matrix-core fragments shared by the forward and
// backward kernels. Device code only.
//
// All products run as v_mfma_f32_32x32x16_bf16. Operand A holds 32 rows, B 32
// columns; lane l holds row (or column) l % 32 and, of the 16 contraction
// indices, the 8 of half h = l / 32. The result has column l % 32 in lane l
// and row 8 (r / 4) + 4 h + r % 4 in register r.
//
// A softmax tile is computed transposed (keys as rows, queries as columns), so
// a lane holds one query: its row maximum and sum are sums over registers and
// one exchange of the halves. Registers 8 t .. 8 t + 7 of that result are then
// the B fragment of the 16 contraction indices 16 t + 8 (j / 4) + 4 h + j % 4
// (j = 0..7) as they stand: the order of a contraction is free, and the other
// operand is read in the same order (tr_frag). No value crosses lanes between
// the two products.
#pragma once

#include "block_internal.h"

namespace p3d {
namespace attn {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ f32x16 mfma(bf16x8_t a, bf16x8_t b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ f32x16 zero16() {
    f32x16 z;
#pragma unroll
    for (int i = 0; i < 16; ++i) z[i] = 0.f;
    return z;
}

// Row r of a 32-row result that register i of half h holds.
__device__ __forceinline__ constexpr int acc_row(int i, int h) {
    return 8 * (i >> 2) + 4 * h + (i & 3);
}

// Loads queued for LDS or registers are done, LDS reads are done, then the
// workgroup meets: what the DMA brought is there for every wave, and every
// wave has left what the next DMA overwrites.
__device__ __forceinline__ void tile_barrier() {
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// This wave's queued loads, all but the newest N, are done, and so are its
// LDS reads.
template <int N>
__device__ __forceinline__ void wave_wait() {
    static_assert(N >= 0 && N < 64, "vmcnt");
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
}

// 64 lanes x 16 bytes from global memory into 1 KB of LDS at the uniform byte
// offset `lds`, lane l at 16 l; lanes that are switched off write nothing. The
// instruction is written out so that the compiler does not wait for it at the
// next LDS read: the waits above are the only ones that cover it. The LDS
// offset goes in m0, an operand, so the compiler writes it. (A write of m0
// needs one wait state before a load to LDS.)
__device__ __forceinline__ void dma16(const void* src, uint32_t lds) {
    asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
                 :
                 : "{m0}"(__builtin_amdgcn_readfirstlane(lds)), "v"(src)
                 : "memory");
}

// 64 lanes x 4 bytes into 256 bytes of LDS, lane l at 4 l.
__device__ __forceinline__ void dma4(const void* src, uint32_t lds) {
    asm volatile("s_nop 0\n\tglobal_load_lds_dword %1, off"
                 :
                 : "{m0}"(__builtin_amdgcn_readfirstlane(lds)), "v"(src)
                 : "memory");
}

// dma16 from a uniform base and a 32-bit offset per lane.
__device__ __forceinline__ void dma16_from(const void* from, uint32_t offset, uint32_t lds) {
    const uint64_t at = (uint64_t)(uintptr_t)from;
    const uint64_t base = ((uint64_t)__builtin_amdgcn_readfirstlane((uint32_t)(at >> 32)) << 32) |
                          (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)at);
    asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                 :
                 : "{m0}"(__builtin_amdgcn_readfirstlane(lds)), "v"(offset), "s"(base)
                 : "memory");
}

__device__ __forceinline__ uint32_t lds_offset(const void* p) {
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)p;
}

// An LDS tile of rows of Chunks 16-byte chunks (8: heads up to 64 wide, 16:
// up to 128). Chunk c of row r sits at slot c ^ swizzle(r). Two kinds of read
// have to spread over the banks (a 256-byte window): 16 consecutive rows at
// one chunk (row fragments), and 4 consecutive rows at 4 neighbouring chunks
// (transposed fragments); the swizzle separates both. A fragment's chunk is an
// exclusive or on a byte address, so a tile starts on a whole row: its array is
// declared with alignas(kTileAlign), and tiles inside it are whole rows apart.
constexpr int kTileAlign = 256;

template <int HD>
struct Tile {
    static constexpr int kChunks = HD <= 64 ? 8 : 16;
    static constexpr int kSteps = HD / 16;          // contraction steps over the head
    static constexpr int kBlocks = HD / 32;         // 32-wide blocks of the head

    static __device__ __forceinline__ int swizzle(int row) {
        if constexpr (kChunks == 16) return ((row & 3) << 2) | ((row >> 2) & 3);
        else return ((row & 2) << 1) | ((row >> 2) & 3);
    }

    // Rows [0, Rows) into `tile`, by waves wave, wave + Waves, ...; `src(row)`
    // is the address of a row's first chunk. Chunks from `chunks` on stay as
    // they are in LDS.
    template <int Rows, int Waves, typename Src>
    static __device__ __forceinline__ void load(uint4* tile, int wave, int lane, int chunks,
                                                Src src) {
        constexpr int kPer = 64 / kChunks;          // rows of one instruction
        static_assert(Rows % (kPer * Waves) == 0, "rows per wave");
        const uint32_t at = lds_offset(tile);
        const int sub = lane / kChunks, c = lane % kChunks;
#pragma unroll
        for (int i = 0; i < Rows / (kPer * Waves); ++i) {
            const int row0 = (i * Waves + wave) * kPer;
            const int row = row0 + sub;
            const int chunk = c ^ swizzle(row);
            if (chunk < chunks) dma16(src(row) + chunk, at + row0 * kChunks * 16);
        }
    }

    // The same for rows a fixed `pitch` of bytes apart, from `first` on, none of
    // them past the end: a scalar base per instruction and one 32-bit offset
    // per lane, which `lane_offset` makes once (pitch at most kMaxPitch).
    static constexpr int64_t kMaxPitch = int64_t(1) << 28;
    static __device__ __forceinline__ int lane_chunk(int wave, int lane) {
        // (a row's swizzle is the same for all of the lane's rows)
        return (lane % kChunks) ^ swizzle(wave * (64 / kChunks) + lane / kChunks);
    }
    static __device__ __forceinline__ uint32_t lane_offset(int wave, int lane, int64_t pitch) {
        return (uint32_t)(lane / kChunks * pitch) + lane_chunk(wave, lane) * 16;
    }
    template <int Rows, int Waves>
    static __device__ __forceinline__ void load_rows(uint4* tile, int wave, const void* first,
                                                     int64_t pitch, uint32_t lane_off, bool on) {
        constexpr int kPer = 64 / kChunks;
        static_assert(Rows % (kPer * Waves) == 0 && (Waves * kPer) % 16 == 0, "rows per wave");
        const uint32_t at = lds_offset(tile);
#pragma unroll
        for (int i = 0; i < Rows / (kPer * Waves); ++i) {
            const int row0 = (i * Waves + wave) * kPer;
            if (on)
                dma16_from(static_cast<const char*>(first) + row0 * pitch, lane_off,
                           at + row0 * kChunks * 16);
        }
    }

    // Zeros in the chunks of a tile's rows that load() leaves as they are.
    static __device__ __forceinline__ void clear(uint4* tile, int rows, int threads, int tid) {
        for (int i = tid; i < rows * kChunks; i += threads) tile[i] = make_uint4(0, 0, 0, 0);
    }

    // LDS byte addresses that a lane's fragments of a tile start from: one
    // register each per tile. The chunk of a contraction step or of a block of
    // columns is an exclusive or on it and rows are immediate offsets. The
    // value is opaque to the compiler, which would otherwise keep an address
    // per fragment (32 registers and as many additions per tile).
    static __device__ __forceinline__ uint32_t row_base(const uint4* tile, int lane) {
        const int r = lane & 31;
        uint32_t at = lds_offset(tile) + (r * kChunks + ((lane >> 5) ^ swizzle(r))) * 16;
        asm volatile("" : "+v"(at));
        return at;
    }
    static __device__ __forceinline__ uint32_t tr_base(const uint4* tile, int lane) {
        const int i2 = (lane >> 2) & 3, h = lane >> 5;
        const int f = kChunks == 16 ? i2 << 2 : (i2 & 2) << 1;
        const int chunk = ((((lane >> 4) & 1) << 1) | ((lane >> 1) & 1)) ^ f ^ h;
        uint32_t at = lds_offset(tile) + ((4 * h + i2) * kChunks + chunk) * 16 + (lane & 1) * 8;
        asm volatile("" : "+v"(at));
        return at;
    }

    typedef const __attribute__((address_space(3))) char lds_char;

    // Rows row0 .. row0 + 31 (a multiple of 32) as operand A, contraction
    // step s of the head.
    static __device__ __forceinline__ bf16x8_t row_frag(uint32_t base, int row0, int s) {
        lds_char* p = (lds_char*)(uintptr_t)(base ^ (32 * s));
        return *(const __attribute__((address_space(3))) bf16x8_t*)(p + row0 * kChunks * 16);
    }

    // Columns 32 db .. 32 db + 31 of the head as the rows of operand A, the
    // contraction over the tile's rows row0 + 8 (j / 4) + 4 h + j % 4: two
    // transposing reads of 4 rows each. In a transposing read the 16 lanes of
    // a group address 4 rows x 16 columns, 4 columns a lane, and each gets
    // one column's 4 values.
    static __device__ __forceinline__ bf16x8_t tr_frag(uint32_t base, int row0, int db) {
        s16x8 v;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            lds_char* p = (lds_char*)(uintptr_t)(base ^ (64 * db) ^ (32 * e));
            const s16x4 q = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (__attribute__((address_space(3))) s16x4*)(p + (row0 + 8 * e) * kChunks * 16));
#pragma unroll
            for (int j = 0; j < 4; ++j) v[4 * e + j] = q[j];
        }
        return __builtin_bit_cast(bf16x8_t, v);
    }
};

// Registers 8 t .. 8 t + 7 of a result as the B fragment of its rows.
__device__ __forceinline__ bf16x8_t acc_frag(const f32x16& p, int t) {
    bf16x8_t f;
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = (__bf16)p[8 * t + j];
    return f;
}

// Query rows of one key head, numbered token * group + member: a row's token
// and member without a division by a variable. `inverse` is floor(2^32 /
// group) + 1 (group > 1): the high half of row * inverse is the quotient or
// one more.
struct Group {
    uint32_t size, inverse;
    __device__ __forceinline__ void split(uint32_t row, uint32_t& token, uint32_t& member) const {
        if (size == 1) {
            token = row;
            member = 0;
            return;
        }
        uint32_t q = __umulhi(row, inverse);
        if (q * size > row) --q;
        token = q;
        member = row - q * size;
    }
};

// Item of a tile number: the last one that starts at or before it.
__device__ __forceinline__ int item_of_tile(const ItemTable& t, int batch, int tile) {
    int lo = 0, hi = batch;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (t.start[mid] <= tile) lo = mid; else hi = mid;
    }
    return lo;
}

// The head's columns of one query row as operand B.
template <int HD>
__device__ __forceinline__ void load_query(bf16x8_t (&q)[Tile<HD>::kSteps], const uint4* row,
                                           bool live, int chunks, int lane) {
#pragma unroll
    for (int k = 0; k < Tile<HD>::kSteps; ++k) {
        const int chunk = 2 * k + (lane >> 5);
        const uint4 v = live && chunk < chunks ? row[chunk] : make_uint4(0, 0, 0, 0);
        q[k] = __builtin_bit_cast(bf16x8_t, v);
    }
}

// The values are there: the compiler's wait for their loads stands here and
// not at their first use inside a loop, where it would also wait for the tile
// loads in flight, which it does not know of.
template <int N>
__device__ __forceinline__ void settle(bf16x8_t (&q)[N]) {
#pragma unroll
    for (int k = 0; k < N; ++k) asm volatile("" : "+v"(q[k]));
}

// A finished tile's rows go out through LDS (32 rows of the tile layout) so
// that whole rows leave in 16-byte pieces: into LDS, and from there, row r to
// dst(r) where that is not null (`nt`: past the caches).
template <int HD>
__device__ __forceinline__ void stage_rows(const f32x16 (&o)[Tile<HD>::kBlocks], float by,
                                           uint4* stage, int chunks, int lane) {
    using T = Tile<HD>;
    const int r = lane & 31, h = lane >> 5;
    uint2* stage2 = reinterpret_cast<uint2*>(stage);
#pragma unroll
    for (int b = 0; b < T::kBlocks; ++b)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (4 * b + j >= chunks) continue;
            uint2 v;
            v.x = pack_bf16x2(o[b][4 * j] * by, o[b][4 * j + 1] * by);
            v.y = pack_bf16x2(o[b][4 * j + 2] * by, o[b][4 * j + 3] * by);
            stage2[(r * T::kChunks + ((4 * b + j) ^ T::swizzle(r))) * 2 + h] = v;
        }
}

template <int HD, typename Dst>
__device__ __forceinline__ void write_rows(const uint4* stage, int chunks, int lane, Dst dst,
                                           bool nt = false) {
    using T = Tile<HD>;
#pragma unroll
    for (int i = 0; i < 32 * T::kChunks / 64; ++i) {
        const int at = i * 64 + lane;
        const int row = at / T::kChunks, c = at % T::kChunks;
        uint4* p = dst(row);
        if (p && c < chunks) {
            const uint4 v = stage[row * T::kChunks + (c ^ T::swizzle(row))];
            if (nt) store_nt16(p + c, v);
            else p[c] = v;
        }
    }
}

template <int HD, typename Dst>
__device__ __forceinline__ void store_rows(const f32x16 (&o)[Tile<HD>::kBlocks], float by,
                                           uint4* stage, int chunks, int lane, Dst dst) {
    stage_rows<HD>(o, by, stage, chunks, lane);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    write_rows<HD>(stage, chunks, lane, dst);
}

// The group of query heads that share a key head.
inline Group group_of(const AttnArgs& a) {
    Group g;
    g.size = (uint32_t)(a.heads / a.kv_heads);
    g.inverse = g.size > 1 ? (uint32_t)((uint64_t(1) << 32) / g.size + 1) : 0;
    return g;
}

// Tiles of `per_tile` rows of every item, an item having `each` rows per entry.
inline void cut_items(const ItemTable& items, int batch, int64_t each, int per_tile,
                      ItemTable* tiles) {
    int32_t at = 0;
    for (int b = 0; b < batch; ++b) {
        tiles->start[b] = at;
        const int64_t rows = (items.start[b + 1] - items.start[b]) * each;
        at += (int32_t)((rows + per_tile - 1) / per_tile);
    }
    for (int b = batch; b <= P3D_MAX_BATCH; ++b) tiles->start[b] = at;
}

}  // namespace attn
}  // namespace p3d
