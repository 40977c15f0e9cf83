// group_norm.hip -- p3d_group_norm and its gradient over channels-last rows.
//
//   x^ = (x - mean) rstd,  u = x^ w + b,  out = act(u)
//   du = dout act'(u),  dbias = sum du,  dweight = sum du x^
//   dx = rstd (w du - A - x^ B),  A, B = avg(w du), avg(w du x^) of the group
//
// Both directions are memory bound: statistics over a whole map stand between
// the first and the last use of a row, so x (and dout) is read twice, from the
// caches where it fits: 3 (5) times the map's bytes in all, and 265 us where x has
// 537 MB, 6.1 TB/s of them, a large copy's rate. A small map takes as long as its
// launches do (12 to 18 us).
//
// A call is cut into chunks of rows and slices of whole groups; a thread owns
// 16-byte vectors of channels and walks the chunk's rows, so per-channel factors
// stay in registers. Chunk results go to the workspace and are joined in a fixed
// order.
#include <algorithm>

#include "model_internal.h"

namespace p3d {

namespace {

constexpr int kThreads = 256;

// How a workgroup's threads lie over the vectors of its slice of channels, and
// over rows.
struct Lay {
    int nv, tx, ty;             // vectors of the slice; threads along it, rows at a time
    __host__ __device__ explicit Lay(int vectors)
        : nv(vectors), tx(vectors < kThreads ? vectors : kThreads), ty(kThreads / tx) {}
};

// The last item or chunk range that starts at or before `at`.
__device__ __forceinline__ int range_of(const ItemTable& t, int batch, int at) {
    int lo = 0, hi = batch;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (t.start[mid] <= at) lo = mid; else hi = mid;
    }
    return lo;
}

// Rows that thread row `ty` of `step` takes of `rows`.
__device__ __forceinline__ int rows_of(int rows, int ty, int step) {
    return ty < rows ? (rows - ty + step - 1) / step : 0;
}

// A chunk: of its item's blocks of `ty` rows every `of`-th from the `at`-th on, so
// that the workgroups that run side by side read side by side: 263 us where 264,000
// rows have 1024 channels, and 361 with chunks of neighbouring rows, 516 KB of
// them, that meet in one memory channel.
struct Chunk {
    int item, at, of, rows, ty;
    int64_t row0;               // of the item
    __device__ __forceinline__ Chunk(const ItemTable& items, const ItemTable& chunk, int batch,
                                     int number, int ty_)
        : item(range_of(chunk, batch, number)), at(number - chunk.start[item]),
          of(chunk.start[item + 1] - chunk.start[item]),
          rows(items.start[item + 1] - items.start[item]), ty(ty_), row0(items.start[item]) {}
    // of thread row y: its first row, how many, and how far apart
    __device__ __forceinline__ int64_t first(int y) const { return row0 + (int64_t)at * ty + y; }
    __device__ __forceinline__ int count(int y) const { return rows_of(rows, at * ty + y, of * ty); }
    __device__ __forceinline__ int64_t step() const { return (int64_t)of * ty; }
};

template <typename T>
__device__ __forceinline__ const uint4* vectors(const void* base, int64_t row, int64_t stride) {
    return reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(base) +
                                          row * stride * (16 / Vec<T>::N));
}

// One vector of a per-channel parameter, `other` where it is absent.
template <typename T>
__device__ __forceinline__ void param(const void* base, int v, float other,
                                      float (&f)[Vec<T>::N]) {
    if (base) {
        Vec<T>::widen(reinterpret_cast<const uint4*>(base)[v], f);
    } else {
#pragma unroll
        for (int e = 0; e < Vec<T>::N; ++e) f[e] = other;
    }
}

// Lanes for each of `groups` in a workgroup.
__device__ __forceinline__ int lanes_of(int groups) {
    int lanes = 64;
    while (lanes > 1 && lanes * groups > kThreads) lanes >>= 1;
    return lanes;
}

// One channel's weight.
template <typename T>
__device__ __forceinline__ float weight_of(const void* weight, int channel) {
    if (!weight) return 1.f;
    if constexpr (sizeof(T) == 4) return reinterpret_cast<const float*>(weight)[channel];
    else return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(weight)[channel] << 16);
}

// ------------------------------------------------------------- statistics ---
// Count, mean and sum of squared deviations of a set of numbers, and the same
// of two sets together: no sum of squares is ever taken about another point
// than the set's own mean, so a mean far from 0 costs no more than its own last
// place: a variance is off by 2^-48 of the mean's square or so, and by nothing
// where all values are alike.
struct Moments {
    float n, mean, m2;
    __device__ __forceinline__ void join(float bn, float bmean, float bm2) {
        if (bn == 0.f) return;
        const float all = n + bn, d = bmean - mean;
        const float w = n == 0.f ? 1.f : bn * __builtin_amdgcn_rcpf(all);
        mean += d * w;
        m2 += bm2 + d * d * n * w;
        n = all;
    }
};

// `n` numbers' mean and squared deviations, from a point near the mean, the squared
// deviations from it and their sum.
__device__ __forceinline__ void centre(float& point, float& d2, float sum, int n) {
    const float off = sum * (1.f / (float)n);
    point += off;
    d2 -= sum * off;
}

// The chunk's moments of every group. Where a vector's channels are of one
// group (Whole), a thread keeps one pair for it, else a pair per channel.
// One batch of 8 (4) rows is centred on its own mean in registers and then joined
// to the thread's: 4 operations a value in all, below the 13 that a bf16 stream at
// the memory's rate leaves. That mean is a rounded sum. In binary32 its error, several
// last places where all values are alike, is the mean of the deviations from it, which
// are exact then, and comes off again: a fifth operation (rows that are 12,345.678
// throughout had deviations of 0.002 otherwise, and results off by 0.8). 64 bf16
// numbers of a kind have an exact sum.
template <typename T, bool Whole>
__global__ __launch_bounds__(kThreads, 4) void group_stats_kernel(
    GroupArgs a, ItemTable chunk, float2* __restrict__ partial) {
    constexpr int N = Vec<T>::N, K = Whole ? 1 : N, PerUnit = Whole ? N : 1;
    constexpr int kBatch = Whole ? 8 : 4;   // rows that a thread loads before it uses them
    constexpr bool kCentre = sizeof(T) == 4;
    __shared__ float2 unit[(Whole ? 1 : N) * 4096 / N];
    const Lay lay(a.channels / N / gridDim.y);
    const int v0 = blockIdx.y * lay.nv, groups = a.groups / gridDim.y, group0 = blockIdx.y * groups;
    const Chunk c(a.items, chunk, a.batch, blockIdx.x, lay.ty);
    const int tx = threadIdx.x % lay.tx, ty = threadIdx.x / lay.tx;
    const int mine = ty < lay.ty ? c.count(ty) : 0;
    const int64_t step = a.x_stride * (16 / N) * c.step();      // bytes
    for (int v = tx; v < lay.nv && ty < lay.ty; v += lay.tx) {
        const char* p =
            reinterpret_cast<const char*>(vectors<T>(a.x, c.first(ty), a.x_stride) + v0 + v);
        float mean[K], m2[K];
#pragma unroll
        for (int k = 0; k < K; ++k) mean[k] = m2[k] = 0.f;
        int r = 0;
        for (; r + kBatch <= mine; r += kBatch) {
            uint4 q[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                q[i] = *reinterpret_cast<const uint4*>(p);
                p += step;
            }
            float s[K], off[K], d2[K];
#pragma unroll
            for (int k = 0; k < K; ++k) s[k] = off[k] = d2[k] = 0.f;
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                float f[N];
                Vec<T>::widen(q[i], f);
#pragma unroll
                for (int e = 0; e < N; ++e) s[Whole ? 0 : e] += f[e];
            }
#pragma unroll
            for (int k = 0; k < K; ++k) s[k] *= 1.f / (kBatch * PerUnit);
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                float f[N];
                Vec<T>::widen(q[i], f);
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    const float d = f[e] - s[Whole ? 0 : e];
                    if constexpr (kCentre) off[Whole ? 0 : e] += d;
                    d2[Whole ? 0 : e] += d * d;
                }
            }
#pragma unroll
            for (int k = 0; k < K; ++k)
                if constexpr (kCentre) centre(s[k], d2[k], off[k], kBatch * PerUnit);
            // rows before, and this batch's share of all
            const float w = kBatch * __builtin_amdgcn_rcpf((float)(r + kBatch));
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const float d = s[k] - mean[k];
                mean[k] += d * w;
                m2[k] += d2[k] + d * d * ((float)r * w * PerUnit);
            }
        }
        for (; r < mine; ++r) {
            float f[N];
            Vec<T>::widen(*reinterpret_cast<const uint4*>(p), f);
            p += step;
            const float w = __builtin_amdgcn_rcpf((float)(r + 1));
            float s[K], d2[K];
#pragma unroll
            for (int k = 0; k < K; ++k) s[k] = d2[k] = 0.f;
#pragma unroll
            for (int e = 0; e < N; ++e) s[Whole ? 0 : e] += f[e];
            if constexpr (Whole) {
                s[0] *= 1.f / N;
                float off = 0.f;
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    const float d = f[e] - s[0];
                    if constexpr (kCentre) off += d;
                    d2[0] += d * d;
                }
                if constexpr (kCentre) centre(s[0], d2[0], off, N);
            }
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const float d = s[k] - mean[k];
                mean[k] += d * w;
                m2[k] += d2[k] + d * d * ((float)r * w * PerUnit);
            }
        }
#pragma unroll
        for (int k = 0; k < K; ++k) unit[(ty * lay.nv + v) * K + k] = make_float2(mean[k], m2[k]);
    }
    __syncthreads();
    // a group's units, K a vector, of every thread row: by `lanes` lanes
    const int per = Whole ? a.channels / a.groups / N : a.channels / a.groups;
    const int width = lay.nv * K;
    const int lanes = lanes_of(groups), lane = threadIdx.x & (lanes - 1);
    for (int g0 = 0; g0 < groups; g0 += kThreads / lanes) {
        const int g = g0 + threadIdx.x / lanes;
        Moments m{0.f, 0.f, 0.f};
        if (g < groups) {
            for (int e = lane; e < per * lay.ty; e += lanes) {
                const int y = e / per;
                const int n = c.count(y);
                const float2 u = unit[y * width + g * per + (e - y * per)];
                m.join((float)(n * PerUnit), u.x, u.y);
            }
        }
        for (int off = 1; off < lanes; off <<= 1) {
            const float n = __shfl_xor(m.n, off), mean = __shfl_xor(m.mean, off),
                        m2 = __shfl_xor(m.m2, off);
            m.join(n, mean, m2);
        }
        if (g < groups && lane == 0)
            partial[(int64_t)(group0 + g) * gridDim.x + blockIdx.x] = make_float2(m.mean, m.m2);
    }
}

// Mean and variance of an item's group from the moments of its `n` chunks, in
// binary64, by `lanes` neighbouring lanes (a power of two, 64 at most). The
// chunks' counts are known, so the mean comes first and the deviations are about
// it: no division a chunk. The chunks were written by other dies, so a load
// takes a microsecond: `Held` of a lane are on their way at once.
struct Joined {
    double mean, var;
};

__device__ __forceinline__ double over_lanes(double v, int lanes) {
    for (int off = 1; off < lanes; off <<= 1) v += __shfl_xor(v, off);
    return v;
}

template <int Held>
__device__ __forceinline__ Joined join_chunks(const float2* __restrict__ p, int n, int lane,
                                              int lanes, int rows, int ty, int per) {
    Joined j{0., 0.};
    if (n == 0) return j;
    // `whole` blocks of ty rows a chunk, one more in the first `more` chunks, and
    // the last block, in chunk `last`, short of `miss` rows. (The quotient is made
    // while the loads are on their way.)
    const int blocks = (rows + ty - 1) / ty, whole = blocks / n, more = blocks - whole * n;
    const int last = (blocks - 1) % n;
    const double block = (double)ty * per, miss = ((double)blocks * ty - rows) * per;
    const double base = block * whole, count = 1. / ((double)rows * per);
    float2 u[Held];
    double sum[4] = {0., 0., 0., 0.}, first = 0.;
    float m2[4] = {0.f, 0.f, 0.f, 0.f}, d2[4] = {0.f, 0.f, 0.f, 0.f}, e2 = 0.f;
    const auto load = [&](int from) {
#pragma unroll
        for (int k = 0; k < Held; ++k) {
            const int c = from + k * lanes + lane;
            u[k] = c < n ? p[c] : make_float2(0.f, 0.f);
        }
    };
    const float xl = p[last].x;
    for (int from = 0; from < n; from += Held * lanes) {
        load(from);
#pragma unroll
        for (int k = 0; k < Held; ++k) {
            sum[k & 3] += (double)u[k].x;
            if (from + k * lanes + lane < more) first += (double)u[k].x;
            m2[k & 3] += u[k].y;
        }
    }
    const double all = over_lanes((sum[0] + sum[1]) + (sum[2] + sum[3]), lanes);
    if (more) first = over_lanes(first, lanes);
    j.mean = (base * all + block * first - miss * (double)xl) * count;
    // deviations of the chunks' means: the difference is taken in two parts, so
    // binary32 holds it
    const float hi = (float)j.mean, lo = (float)(j.mean - (double)hi);
    for (int from = 0; from < n; from += Held * lanes) {
        if (n > Held * lanes) load(from);
#pragma unroll
        for (int k = 0; k < Held; ++k) {
            const int c = from + k * lanes + lane;
            float d = c < n ? (u[k].x - hi) - lo : 0.f;
            d *= d;
            d2[k & 3] += d;
            if (c < more) e2 += d;
        }
    }
    const double dl = (double)((xl - hi) - lo);
    const double within = over_lanes((double)((m2[0] + m2[1]) + (m2[2] + m2[3])), lanes);
    const double between = over_lanes(
        base * (double)((d2[0] + d2[1]) + (d2[2] + d2[3])) + block * (double)e2, lanes);
    j.var = (within + between - miss * (dl * dl)) * count;
    if (j.var < 0.) j.var = 0.;
    return j;
}

// The mean in two binary32 parts (so that subtracting it from x loses nothing)
// and rstd.
__device__ __forceinline__ float4 stat_of(const Joined& j, float eps) {
    const float hi = (float)j.mean;
    return make_float4(hi, (float)(j.mean - (double)hi),
                       1.f / sqrtf((float)(j.var + (double)eps)), 0.f);
}

// A wave joins the chunks of a group of an item (16 a lane: a large map's 1023 at once).
__global__ __launch_bounds__(kThreads) void group_join_kernel(GroupArgs a, ItemTable chunk,
                                                              int ty,
                                                              const float2* __restrict__ partial,
                                                              float4* __restrict__ stat) {
    const int64_t at = (int64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6);
    if (at >= (int64_t)a.batch * a.groups) return;
    const int b = (int)(at / a.groups), g = (int)(at % a.groups), lane = threadIdx.x & 63;
    const int first = chunk.start[b];
    const Joined j = join_chunks<16>(partial + (int64_t)g * chunk.start[a.batch] + first,
                                 chunk.start[b + 1] - first, lane, 64,
                                 a.items.start[b + 1] - a.items.start[b], ty,
                                 a.channels / a.groups);
    if (lane) return;
    const float4 s = stat_of(j, a.eps);
    stat[at] = s;
    if (a.mean) a.mean[at] = s.x;
    if (a.rstd) a.rstd[at] = s.z;
}

// The same by a workgroup for `groups` groups of item b from group0 on, into LDS;
// `write` as well into mean and rstd.
__device__ __forceinline__ void join_here(const GroupArgs& a, const ItemTable& chunk, int ty,
                                          const float2* __restrict__ partial, int b, int group0,
                                          int groups, bool write, float4* __restrict__ stat) {
    const int lanes = lanes_of(groups), lane = threadIdx.x & (lanes - 1);
    const int first = chunk.start[b], n = chunk.start[b + 1] - first;
    for (int g0 = 0; g0 < groups; g0 += kThreads / lanes) {
        const int g = g0 + threadIdx.x / lanes;
        const bool on = g < groups;
        // (12: with 16 the apply kernel spills registers)
        const Joined j = join_chunks<12>(
            partial + (int64_t)(group0 + (on ? g : 0)) * chunk.start[a.batch] + first, n, lane,
            lanes, a.items.start[b + 1] - a.items.start[b], ty, a.channels / a.groups);
        if (on && lane == 0) {
            const float4 s = stat_of(j, a.eps);
            stat[g] = s;
            if (write && a.mean) a.mean[(int64_t)b * a.groups + group0 + g] = s.x;
            if (write && a.rstd) a.rstd[(int64_t)b * a.groups + group0 + g] = s.z;
        }
    }
    __syncthreads();
}

// ------------------------------------------------------------------ apply ---
template <bool Past>
__device__ __forceinline__ uint4 load16(const char* p) {
    if constexpr (Past)
        return __builtin_bit_cast(uint4,
                                  __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(p)));
    else
        return *reinterpret_cast<const uint4*>(p);
}

// out = act((x - hi) k + o) with k = rstd w and o = b - lo k. Rows run last to
// first: what the statistics read last is still in the caches. `Past`:
// a map larger than those is loaded past them here, so that what was just read
// does not drive out what was read before and is wanted next (265 us with it and
// 286 without where x has 537 MB; 161 and 156, the gradient after it, where x has
// 102 MB).
// `Here`: the workgroup joins its item's chunks itself.
template <typename T, int Act, bool Whole, bool Past, bool Here>
__global__ __launch_bounds__(kThreads, 4) void group_apply_kernel(
    GroupArgs a, ItemTable chunk, const float2* __restrict__ partial,
    const float4* __restrict__ stats) {
    constexpr int N = Vec<T>::N, K = Whole ? 1 : N, U = Whole ? 4 : 2;
    extern __shared__ float4 joined[];              // Here: [groups]
    const Lay lay(a.channels / N / gridDim.y);
    const int v0 = blockIdx.y * lay.nv, groups = a.groups / gridDim.y, group0 = blockIdx.y * groups;
    const int at = blockIdx.x;
    const Chunk c(a.items, chunk, a.batch, at, lay.ty);
    const int tx = threadIdx.x % lay.tx, ty = threadIdx.x / lay.tx;
    const int mine = ty < lay.ty ? c.count(ty) : 0;
    const int64_t step = -a.x_stride * (16 / N) * c.step(),
                  ostep = -a.out_stride * (16 / N) * c.step();
    const int64_t row = c.first(ty) + (mine - 1) * c.step();        // the last, and on to the first
    const int per = a.channels / a.groups;
    // The first rows are on their way before the statistics are there.
    uint4 q[U];
    const auto load = [&](const char* p, int rows) {
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (i < rows) q[i] = load16<Past>(p + i * step);
    };
    const char* x0 = reinterpret_cast<const char*>(vectors<T>(a.x, row, a.x_stride) + v0);
    char* o0 = const_cast<char*>(
        reinterpret_cast<const char*>(vectors<T>(a.out, row, a.out_stride) + v0));
    load(x0 + tx * 16, mine);
    const float4* stat = joined;
    if constexpr (Here)
        join_here(a, chunk, lay.ty, partial, c.item, group0, groups, at == chunk.start[c.item],
                  joined);
    else
        stat = stats + (int64_t)c.item * a.groups + group0;
    if (mine == 0) return;
    for (int v = tx; v < lay.nv; v += lay.tx) {
        const char* p = x0 + v * 16;
        char* o = o0 + v * 16;
        if (v != tx) load(p, mine);
        float hi[K], by[N], off[N];
        param<T>(a.weight, v0 + v, 1.f, by);
        param<T>(a.bias, v0 + v, 0.f, off);
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const float4 s = stat[(v * N + (Whole ? 0 : e)) / per];
            hi[Whole ? 0 : e] = s.x;
            by[e] *= s.z;
            off[e] -= s.y * by[e];
        }
        const auto one = [&](uint4 x) {
            float f[N];
            Vec<T>::widen(x, f);
#pragma unroll
            for (int e = 0; e < N; ++e)
                f[e] = activate<Act>((f[e] - hi[Whole ? 0 : e]) * by[e] + off[e]);
            return Vec<T>::narrow(f);
        };
        int r = 0;
        for (; r + U <= mine; r += U) {
#pragma unroll
            for (int i = 0; i < U; ++i) store_nt16(o + i * ostep, one(q[i]));
            p += U * step;
            o += U * ostep;
            load(p, mine - r - U);
        }
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (r + i < mine) store_nt16(o + i * ostep, one(q[i]));
    }
}

// --------------------------------------------------------------- gradient ---
// What the gradient's kernels know of a vector of channels.
template <typename T, bool Whole>
struct Channels {
    static constexpr int N = Vec<T>::N, K = Whole ? 1 : N;
    float mean[K], rstd[K], w[N], b[N];

    __device__ __forceinline__ void load(const GroupArgs& a, int item, int v) {
        const int per = a.channels / a.groups;
        param<T>(a.weight, v, 1.f, w);
        param<T>(a.bias, v, 0.f, b);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int64_t at = (int64_t)item * a.groups + (v * N + k) / per;
            mean[k] = a.mean_in[at];
            rstd[k] = a.rstd_in[at];
        }
    }
    // x^ and du of element e
    template <int Act>
    __device__ __forceinline__ void at(int e, float x, float d, float& xn, float& du) const {
        xn = (x - mean[Whole ? 0 : e]) * rstd[Whole ? 0 : e];
        du = d * slope<Act>(xn * w[e] + b[e]);
    }
};

// Sums of du and of du x^ of every channel over the chunk: [2][channels].
template <typename T, int Act, bool Whole>
__global__ __launch_bounds__(kThreads, 4) void group_sums_kernel(GroupArgs a, ItemTable chunk,
                                                                 float* __restrict__ partial) {
    constexpr int N = Vec<T>::N, U = Whole ? 4 : 2;
    __shared__ float sums[2 * kThreads * N];
    const Lay lay(a.channels / N / gridDim.y);
    const int v0 = blockIdx.y * lay.nv, width = lay.nv * N;
    const Chunk c(a.items, chunk, a.batch, blockIdx.x, lay.ty);
    const int tx = threadIdx.x % lay.tx, ty = threadIdx.x / lay.tx;
    const int mine = ty < lay.ty ? c.count(ty) : 0;
    const int64_t step = a.x_stride * (16 / N) * c.step(),
                  dstep = a.dout_stride * (16 / N) * c.step();
    float* to = partial + (int64_t)blockIdx.x * 2 * a.channels + v0 * N;
    for (int v = tx; v < lay.nv && ty < lay.ty; v += lay.tx) {
        const char* p =
            reinterpret_cast<const char*>(vectors<T>(a.x, c.first(ty), a.x_stride) + v0 + v);
        const char* d = reinterpret_cast<const char*>(
            vectors<T>(a.dout, c.first(ty), a.dout_stride) + v0 + v);
        Channels<T, Whole> ch;
        ch.load(a, c.item, v0 + v);
        float s1[N], s2[N];
#pragma unroll
        for (int e = 0; e < N; ++e) s1[e] = s2[e] = 0.f;
        const auto add = [&](uint4 qx, uint4 qd) {
            float fx[N], fd[N];
            Vec<T>::widen(qx, fx);
            Vec<T>::widen(qd, fd);
#pragma unroll
            for (int e = 0; e < N; ++e) {
                float xn, du;
                ch.template at<Act>(e, fx[e], fd[e], xn, du);
                s1[e] += du;
                s2[e] += du * xn;
            }
        };
        int r = 0;
        for (; r + U <= mine; r += U) {
            uint4 qx[U], qd[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                qx[i] = *reinterpret_cast<const uint4*>(p + i * step);
                qd[i] = *reinterpret_cast<const uint4*>(d + i * dstep);
            }
#pragma unroll
            for (int i = 0; i < U; ++i) add(qx[i], qd[i]);
            p += U * step;
            d += U * dstep;
        }
        for (; r < mine; ++r, p += step, d += dstep)
            add(*reinterpret_cast<const uint4*>(p), *reinterpret_cast<const uint4*>(d));
        if (lay.ty == 1) {
#pragma unroll
            for (int e = 0; e < N; ++e) {
                to[v * N + e] = s1[e];
                to[a.channels + v * N + e] = s2[e];
            }
        } else {
            // (then tx covers the row: one vector a thread)
#pragma unroll
            for (int e = 0; e < N; ++e) {
                sums[ty * width + v * N + e] = s1[e];
                sums[kThreads * N + ty * width + v * N + e] = s2[e];
            }
        }
    }
    if (lay.ty == 1) return;
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * width; i += kThreads) {
        const int half = i >= width, col = i - half * width;
        const float* from = sums + half * kThreads * N + col;
        float s = 0.f;
        for (int y = 0; y < lay.ty; ++y) s += from[y * width];
        to[half * a.channels + col] = s;
    }
}

// The items' sums [batch][2][channels] of the chunks': 32 columns and 32 lanes
// over the chunks.
constexpr int kTotalCols = 32, kTotalLanes = 32;

__global__ __launch_bounds__(kTotalCols * kTotalLanes) void group_totals_kernel(
    int columns, ItemTable chunk, const float* __restrict__ partial, float* __restrict__ total) {
    __shared__ double part[kTotalLanes][kTotalCols + 1];
    const int x = threadIdx.x % kTotalCols, y = threadIdx.x / kTotalCols;
    const int col = blockIdx.x * kTotalCols + x, b = blockIdx.y;
    double s = 0.;
    if (col < columns) {
        const float* p = partial + col;
#pragma unroll 8
        for (int c = chunk.start[b] + y; c < chunk.start[b + 1]; c += kTotalLanes)
            s += p[(int64_t)c * columns];
    }
    part[y][x] = s;
    __syncthreads();
    if (y == 0 && col < columns) {
        for (int i = 1; i < kTotalLanes; ++i) s += part[i][x];
        total[(int64_t)b * columns + col] = (float)s;
    }
}

// Sums over chunks [first, last) of `count` neighbouring columns from p on, rows
// `pitch` apart, into LDS, by the whole workgroup: sum[count] at its start. The
// chunks were written by other dies: 8 loads of a thread are on their way at once.
__device__ __forceinline__ void sum_chunks(const float* __restrict__ p, int64_t pitch, int count,
                                           int first, int last, double* part, float* sum) {
    const int across = count < kThreads ? count : kThreads, down = kThreads / across;
    const int x = threadIdx.x % across, y = threadIdx.x / across;
    for (int c0 = 0; c0 < count; c0 += across) {
        const bool on = c0 + x < count && y < down;
        double s = 0.;
        if (on) {
            const float* q = p + c0 + x;
#pragma unroll 8
            for (int c = first + y; c < last; c += down) s += q[(int64_t)c * pitch];
        }
        __syncthreads();
        part[threadIdx.x] = s;
        __syncthreads();
        if (on && y == 0) {
            for (int k = 1; k < down; ++k) s += part[k * across + x];
            sum[c0 + x] = (float)s;
        }
    }
    __syncthreads();
}

// dx; and, by the workgroups behind the chunks', dweight and dbias, of kThreads
// channels each from the items' sums, or (`Here`: the workgroups join the chunks
// themselves) of kHereCols from the chunks'.
constexpr int kHereCols = 32;

template <typename T, int Act, bool Whole, bool Here>
__global__ __launch_bounds__(kThreads, 4) void group_dx_kernel(GroupArgs a, ItemTable chunk,
                                                               int chunks,
                                                               const float* __restrict__ partial,
                                                               const float* __restrict__ total) {
    constexpr int N = Vec<T>::N, U = Whole ? 4 : 2;
    // [groups]: A and B of the item, with -1 / count; Here: then the sums of the
    // slice's channels
    extern __shared__ float2 avg[];
    __shared__ double part[Here ? kThreads : 1];
    if ((int)blockIdx.x >= chunks) {
        if (blockIdx.y) return;
        const int block = (int)blockIdx.x - chunks;
        if constexpr (Here) {
            float* sum = reinterpret_cast<float*>(avg);
            const int col = block * kHereCols, count = min(kHereCols, a.channels - col);
            for (int half = 0; half < 2; ++half) {
                sum_chunks(partial + half * a.channels + col, 2 * a.channels, count, 0,
                           chunk.start[a.batch], part, sum);
                float* to = half ? a.dweight : a.dbias;
                if (to && (int)threadIdx.x < count) to[col + threadIdx.x] = sum[threadIdx.x];
                __syncthreads();
            }
            return;
        }
        const int col = block * kThreads + threadIdx.x;
        if (col >= a.channels) return;
        double s1 = 0., s2 = 0.;
#pragma unroll 8
        for (int b = 0; b < a.batch; ++b) {
            const float* t = total + (int64_t)b * 2 * a.channels + col;
            s1 += t[0];
            s2 += t[a.channels];
        }
        if (a.dbias) a.dbias[col] = (float)s1;
        if (a.dweight) a.dweight[col] = (float)s2;
        return;
    }
    const Lay lay(a.channels / N / gridDim.y);
    const int v0 = blockIdx.y * lay.nv, groups = a.groups / gridDim.y, width = lay.nv * N;
    const Chunk c(a.items, chunk, a.batch, (int)blockIdx.x, lay.ty);
    const int per = a.channels / a.groups;
    {
        // the item's sums of the slice's channels: du's, and du x^'s `apart` on
        const float* t = total + (int64_t)c.item * 2 * a.channels + v0 * N;
        int apart = a.channels;
        if constexpr (Here) {
            float* sum = reinterpret_cast<float*>(avg + groups);
            for (int half = 0; half < 2; ++half)
                sum_chunks(partial + half * a.channels + v0 * N, 2 * a.channels, width,
                           chunk.start[c.item], chunk.start[c.item + 1], part, sum + half * width);
            t = sum;
            apart = width;
        }
        const int64_t count = (int64_t)(a.items.start[c.item + 1] - a.items.start[c.item]) * per;
        const float by = (float)(-1. / (double)count);
        const int lanes = lanes_of(groups), lane = threadIdx.x & (lanes - 1);
        for (int g0 = 0; g0 < groups; g0 += kThreads / lanes) {
            const int g = g0 + threadIdx.x / lanes;
            float s1 = 0.f, s2 = 0.f;
            if (g < groups) {
                for (int e = lane; e < per; e += lanes) {
                    const int col = g * per + e;
                    const float w = weight_of<T>(a.weight, v0 * N + col);
                    s1 += w * t[col];
                    s2 += w * t[apart + col];
                }
            }
            for (int off = 1; off < lanes; off <<= 1) {
                s1 += __shfl_xor(s1, off);
                s2 += __shfl_xor(s2, off);
            }
            if (g < groups && lane == 0) avg[g] = make_float2(s1 * by, s2 * by);
        }
    }
    __syncthreads();
    const int tx = threadIdx.x % lay.tx, ty = threadIdx.x / lay.tx;
    if (ty >= lay.ty) return;
    const int mine = c.count(ty);
    const int64_t step = -a.x_stride * (16 / N) * c.step(),
                  dstep = -a.dout_stride * (16 / N) * c.step(),
                  ostep = -a.out_stride * (16 / N) * c.step();
    const int64_t row = c.first(ty) + (mine - 1) * c.step();        // the last, and on to the first
    for (int v = tx; v < lay.nv; v += lay.tx) {
        const char* p = reinterpret_cast<const char*>(vectors<T>(a.x, row, a.x_stride) + v0 + v);
        const char* d =
            reinterpret_cast<const char*>(vectors<T>(a.dout, row, a.dout_stride) + v0 + v);
        char* o = const_cast<char*>(
            reinterpret_cast<const char*>(vectors<T>(a.dx, row, a.out_stride) + v0 + v));
        Channels<T, Whole> ch;
        ch.load(a, c.item, v0 + v);
        constexpr int K = Channels<T, Whole>::K;
        float2 m[K];
#pragma unroll
        for (int k = 0; k < K; ++k) m[k] = avg[(v * N + k) / per];
        const auto one = [&](uint4 qx, uint4 qd) {
            float fx[N], fd[N];
            Vec<T>::widen(qx, fx);
            Vec<T>::widen(qd, fd);
#pragma unroll
            for (int e = 0; e < N; ++e) {
                float xn, du;
                ch.template at<Act>(e, fx[e], fd[e], xn, du);
                const int k = Whole ? 0 : e;
                fx[e] = ch.rstd[k] * (du * ch.w[e] + (m[k].x + xn * m[k].y));
            }
            return Vec<T>::narrow(fx);
        };
        int r = 0;
        for (; r + U <= mine; r += U) {
            uint4 qx[U], qd[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                qx[i] = *reinterpret_cast<const uint4*>(p + i * step);
                qd[i] = *reinterpret_cast<const uint4*>(d + i * dstep);
            }
#pragma unroll
            for (int i = 0; i < U; ++i) store_nt16(o + i * ostep, one(qx[i], qd[i]));
            p += U * step;
            d += U * dstep;
            o += U * ostep;
        }
        for (; r < mine; ++r, p += step, d += dstep, o += ostep)
            store_nt16(o, one(*reinterpret_cast<const uint4*>(p),
                              *reinterpret_cast<const uint4*>(d)));
    }
}

// ------------------------------------------------------------- small items ---
// Items whose slice of channels fits a workgroup's registers take one launch: a
// workgroup holds the slice of all of an item's rows between the sums and their
// use, so the data is read once and the statistics are about the exact mean.
// What it saves is a launch or two. Here and in the chunks' kernels, us, bf16 with 32
// groups: the forward call 10 and 14 (64 rows of 1024 in one item, 1024 in 16 items),
// 12 and 17 (64 items of 64 rows of 1024), 19 and 23 (256 of 64 of 512); the gradient
// 11.8 and 15.4, 15.8 and 16.0, 18.5 and 18.8 (binary32: 22 and 20), and 35 and 24 for
// the last of these, whose workgroups, a whole item each, hold all that they can. With
// more than a workgroup a CU it is the slower: 14 us, not 12, and the gradient 24, not
// 18.5, for those 64 items in 8 slices each.
constexpr int kSmallThreads = 1024;

// Vectors that a thread holds: 32 elements.
template <typename T>
constexpr int kHold = 32 / Vec<T>::N;

struct SmallLay {
    int nv, ty;                 // vectors of the slice, each a thread's; rows at a time
    __host__ __device__ explicit SmallLay(int vectors) : nv(vectors), ty(kSmallThreads / vectors) {}
};

// Lanes for each of `sums` in such a workgroup.
__device__ __forceinline__ int small_lanes(int sums) {
    int lanes = 64;
    while (lanes > 1 && lanes * sums > kSmallThreads) lanes >>= 1;
    return lanes;
}

// Sums over a group's vectors and thread rows of each thread's value: sums[g] of
// the slice's groups, in every thread's sight on return.
__device__ __forceinline__ void sum_groups(float v, const SmallLay& lay, bool on, int groups,
                                           float* units, float* sums) {
    const int per = lay.nv / groups;
    __syncthreads();                        // (the sums before are read by now)
    if (on) units[threadIdx.x] = v;
    __syncthreads();
    const int lanes = small_lanes(groups), lane = threadIdx.x & (lanes - 1);
    for (int g0 = 0; g0 < groups; g0 += kSmallThreads / lanes) {
        const int g = g0 + threadIdx.x / lanes;
        float s = 0.f;
        if (g < groups) {
            for (int e = lane; e < per * lay.ty; e += lanes) {
                const int y = e / per;
                s += units[y * lay.nv + g * per + (e - y * per)];
            }
        }
        for (int off = 1; off < lanes; off <<= 1) s += __shfl_xor(s, off);
        if (g < groups && lane == 0) sums[g] = s;
    }
    __syncthreads();
}

// (A vector's channels are of one group: plans see to it.)
template <typename T, int Act>
__global__ __launch_bounds__(kSmallThreads) void group_small_kernel(GroupArgs a) {
    constexpr int N = Vec<T>::N, H = kHold<T>;
    extern __shared__ float lds_small[];
    const SmallLay lay(a.channels / N / gridDim.x);
    const int v0 = blockIdx.x * lay.nv;
    const int groups = a.groups / gridDim.x, group0 = blockIdx.x * groups;
    const int per = a.channels / a.groups, item = blockIdx.y;
    const int64_t row0 = a.items.start[item];
    const int rows = (int)(a.items.start[item + 1] - row0);
    const int tx = threadIdx.x % lay.nv, ty = threadIdx.x / lay.nv;
    const bool on = ty < lay.ty;
    const int mine = on ? rows_of(rows, ty, lay.ty) : 0;
    float* units = lds_small;
    float* sum = units + kSmallThreads;
    float* sum2 = sum + groups;
    uint4 q[H];
#pragma unroll
    for (int i = 0; i < H; ++i)
        q[i] = i < mine ? vectors<T>(a.x, row0 + ty + (int64_t)i * lay.ty, a.x_stride)[v0 + tx]
                        : make_uint4(0, 0, 0, 0);
    float by[N], off[N];
    param<T>(a.weight, v0 + tx, 1.f, by);
    param<T>(a.bias, v0 + tx, 0.f, off);
    float s = 0.f, s2 = 0.f;
#pragma unroll
    for (int i = 0; i < H; ++i) {
        float f[N];
        Vec<T>::widen(q[i], f);
#pragma unroll
        for (int e = 0; e < N; ++e) s += f[e];
    }
    sum_groups(s, lay, on, groups, units, sum);
    // deviations about the mean as binary32 has it; their own mean is what it is
    // off by
    const int g = tx * N / per;
    const float inv = rows > 0 ? 1.f / ((float)rows * (float)per) : 0.f;
    const float mean = sum[g] * inv;
    s = 0.f;
#pragma unroll
    for (int i = 0; i < H; ++i) {
        if (i >= mine) continue;
        float f[N];
        Vec<T>::widen(q[i], f);
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const float d = f[e] - mean;
            s += d;
            s2 += d * d;
        }
    }
    sum_groups(s2, lay, on, groups, units, sum2);
    sum_groups(s, lay, on, groups, units, sum);
    const float lo = sum[g] * inv;
    float var = sum2[g] * inv - lo * lo;
    if (var < 0.f) var = 0.f;               // (and a NaN stays one)
    const float rstd = 1.f / sqrtf(var + a.eps);
    if (threadIdx.x < lay.nv && tx * N % per == 0) {    // a group's first vector writes for it
        const int64_t at = (int64_t)item * a.groups + group0 + g;
        if (a.mean) a.mean[at] = mean + lo;
        if (a.rstd) a.rstd[at] = rstd;
    }
#pragma unroll
    for (int e = 0; e < N; ++e) {
        by[e] *= rstd;
        off[e] -= lo * by[e];
    }
#pragma unroll
    for (int i = 0; i < H; ++i) {
        if (i >= mine) continue;
        float f[N];
        Vec<T>::widen(q[i], f);
#pragma unroll
        for (int e = 0; e < N; ++e) f[e] = activate<Act>((f[e] - mean) * by[e] + off[e]);
        const_cast<uint4*>(vectors<T>(a.out, row0 + ty + (int64_t)i * lay.ty,
                                      a.out_stride))[v0 + tx] = Vec<T>::narrow(f);
    }
}

// The gradient of small items in one launch; of several, whose parameter
// gradients are summed up after it, their sums go to `total` [batch][2][channels].
template <typename T, int Act>
__global__ __launch_bounds__(kSmallThreads) void group_small_backward_kernel(
    GroupArgs a, float* __restrict__ total) {
    constexpr int N = Vec<T>::N, H = kHold<T>;
    extern __shared__ float lds_small[];
    const SmallLay lay(a.channels / N / gridDim.x);
    const int v0 = blockIdx.x * lay.nv, width = lay.nv * N;
    const int groups = a.groups / gridDim.x, per = a.channels / a.groups;
    const int item = blockIdx.y;
    const int64_t row0 = a.items.start[item];
    const int rows = (int)(a.items.start[item + 1] - row0);
    const int tx = threadIdx.x % lay.nv, ty = threadIdx.x / lay.nv;
    const bool on = ty < lay.ty;
    const int mine = on ? rows_of(rows, ty, lay.ty) : 0;
    float* parts = lds_small;               // [2][ty][width], then the columns' sums [2][width]
    float* columns = parts + 2 * kSmallThreads * N;
    float2* avg = reinterpret_cast<float2*>(columns + 2 * width);
    uint4 qx[H], qd[H];
#pragma unroll
    for (int i = 0; i < H; ++i) {
        const int64_t row = row0 + ty + (int64_t)i * lay.ty;
        qx[i] = i < mine ? vectors<T>(a.x, row, a.x_stride)[v0 + tx] : make_uint4(0, 0, 0, 0);
        qd[i] = i < mine ? vectors<T>(a.dout, row, a.dout_stride)[v0 + tx] : make_uint4(0, 0, 0, 0);
    }
    Channels<T, true> ch;
    ch.load(a, item, v0 + tx);
    float s1[N], s2[N];
#pragma unroll
    for (int e = 0; e < N; ++e) s1[e] = s2[e] = 0.f;
#pragma unroll
    for (int i = 0; i < H; ++i) {
        if (i >= mine) continue;
        float fx[N], fd[N];
        Vec<T>::widen(qx[i], fx);
        Vec<T>::widen(qd[i], fd);
#pragma unroll
        for (int e = 0; e < N; ++e) {
            float xn, du;
            ch.template at<Act>(e, fx[e], fd[e], xn, du);
            s1[e] += du;
            s2[e] += du * xn;
        }
    }
    if (on)
#pragma unroll
        for (int e = 0; e < N; ++e) {
            parts[ty * width + tx * N + e] = s1[e];
            parts[kSmallThreads * N + ty * width + tx * N + e] = s2[e];
        }
    __syncthreads();
    // a column by neighbouring lanes, as many as there are for it
    int lanes = small_lanes(2 * width);
    for (int c0 = 0; c0 < 2 * width; c0 += kSmallThreads / lanes) {
        const int c = c0 + threadIdx.x / lanes, half = c >= width, col = c - half * width;
        float s = 0.f;
        if (c < 2 * width)
            for (int y = threadIdx.x & (lanes - 1); y < lay.ty; y += lanes)
                s += parts[half * kSmallThreads * N + y * width + col];
        for (int off = 1; off < lanes; off <<= 1) s += __shfl_xor(s, off);
        if (c < 2 * width && (threadIdx.x & (lanes - 1)) == 0) {
            columns[c] = s;
            const int channel = v0 * N + col;
            if (a.batch > 1) {
                total[((int64_t)item * 2 + half) * a.channels + channel] = s;
            } else {
                float* to = half ? a.dweight : a.dbias;
                if (to) to[channel] = s;
            }
        }
    }
    __syncthreads();
    lanes = small_lanes(groups);
    const float by = rows > 0 ? -1.f / ((float)rows * (float)per) : 0.f;
    for (int g0 = 0; g0 < groups; g0 += kSmallThreads / lanes) {
        const int g = g0 + threadIdx.x / lanes;
        float t1 = 0.f, t2 = 0.f;
        if (g < groups)
            for (int e = threadIdx.x & (lanes - 1); e < per; e += lanes) {
                const int col = g * per + e;
                const float w = weight_of<T>(a.weight, v0 * N + col);
                t1 += w * columns[col];
                t2 += w * columns[width + col];
            }
        for (int off = 1; off < lanes; off <<= 1) {
            t1 += __shfl_xor(t1, off);
            t2 += __shfl_xor(t2, off);
        }
        if (g < groups && (threadIdx.x & (lanes - 1)) == 0) avg[g] = make_float2(t1 * by, t2 * by);
    }
    __syncthreads();
    const float2 m = avg[tx * N / per];
#pragma unroll
    for (int i = 0; i < H; ++i) {
        if (i >= mine) continue;
        float fx[N], fd[N];
        Vec<T>::widen(qx[i], fx);
        Vec<T>::widen(qd[i], fd);
#pragma unroll
        for (int e = 0; e < N; ++e) {
            float xn, du;
            ch.template at<Act>(e, fx[e], fd[e], xn, du);
            fx[e] = ch.rstd[0] * (du * ch.w[e] + (m.x + xn * m.y));
        }
        const_cast<uint4*>(vectors<T>(a.dx, row0 + ty + (int64_t)i * lay.ty,
                                      a.out_stride))[v0 + tx] = Vec<T>::narrow(fx);
    }
}

// ----------------------------------------------------------------- launch ---
// Whether the second kernel's workgroups join their item's chunks, of `bytes`
// each, themselves: what they read for it, all together, against a launch of 4 us.
// Here and with a launch of its own, us: the forward call 27.7 and 29.4 (40,000 rows
// of 512 in 2 groups, 16 MB), 104.0 and 105.5 (90,000 of 1024 in 16 items, 16 MB),
// 30.0 and 29.2 (20,000 of 1024 in one group, 8 MB); the gradient 17.6 and 19.0 (4096
// of 512, 4 MB), 19.5 and 21.3 (10,000 in 2 items, 12 MB), 19.9 and 19.0 (7000, 12 MB),
// 21.2 and 18.9 (4096 of 1024, 8 MB). The bound is on the sum, so a map of all of 1023
// chunks passes where it has 2 groups or fewer.
bool join_in_apply(const GroupArgs& a, const GroupPlan& p, size_t bytes) {
    int64_t pairs = 0;
    for (int b = 0; b < a.batch; ++b) {
        const int64_t n = p.chunk.start[b + 1] - p.chunk.start[b];
        if (n == 0) return false;                   // (nothing would write its mean and rstd)
        pairs += n * n;
    }
    return pairs * (int64_t)bytes <= (int64_t(16) << 20);
}

// Whether x is so large that its second pass loads it past the caches.
bool is_past(const GroupArgs& a, int unit) {
    return (int64_t)a.items.start[a.batch] * a.channels * (16 / unit) > int64_t(200) << 20;
}

template <typename T, bool Whole>
hipError_t forward_of(const GroupArgs& a, const GroupPlan& p, float2* partial, float4* stat,
                      hipStream_t s) {
    const auto with_act = [&](auto run) {
        if (a.act == P3D_ACT_SILU) run(std::integral_constant<int, P3D_ACT_SILU>());
        else if (a.act == P3D_ACT_GELU) run(std::integral_constant<int, P3D_ACT_GELU>());
        else run(std::integral_constant<int, P3D_ACT_NONE>());
        return hipGetLastError();
    };
    if (p.small) {
        const size_t lds = (kSmallThreads + 2 * a.groups / p.small) * sizeof(float);
        return with_act([&](auto act) {
            group_small_kernel<T, decltype(act)::value>
                <<<dim3(p.small, a.batch), kSmallThreads, lds, s>>>(a);
        });
    }
    const int chunks = p.chunk.start[a.batch];
    if (chunks) {
        group_stats_kernel<T, Whole><<<dim3(chunks, p.slices), kThreads, 0, s>>>(a, p.chunk, partial);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    // (A map loaded past the caches has its chunks joined before: of 262,144 rows of
    // 1024 channels in one group 264 us, 286 where the workgroups joined them and loaded
    // through the caches.)
    const bool past = is_past(a, Vec<T>::N);
    const bool here = !past && join_in_apply(a, p, a.groups * sizeof(float2));
    if (!here) {
        const int64_t waves = (int64_t)a.batch * a.groups;
        group_join_kernel<<<(unsigned)((waves + 3) / 4), kThreads, 0, s>>>(a, p.chunk, p.ty,
                                                                           partial, stat);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess || !chunks) return e;
    }
    return with_act([&](auto act) {
        constexpr int A = decltype(act)::value;
        const size_t lds = here ? a.groups / p.slices * sizeof(float4) : 0;
        const dim3 grid(chunks, p.slices);
        if (here)
            group_apply_kernel<T, A, Whole, false, true>
                <<<grid, kThreads, lds, s>>>(a, p.chunk, partial, stat);
        else if (past)
            group_apply_kernel<T, A, Whole, true, false>
                <<<grid, kThreads, 0, s>>>(a, p.chunk, partial, stat);
        else
            group_apply_kernel<T, A, Whole, false, false>
                <<<grid, kThreads, 0, s>>>(a, p.chunk, partial, stat);
    });
}

template <typename T, int Act, bool Whole>
hipError_t backward_act(const GroupArgs& a, const GroupPlan& p, float* partial, float* total,
                        hipStream_t s) {
    const int more = a.dweight || a.dbias ? (a.channels + kThreads - 1) / kThreads : 0;
    if (p.small) {
        const int width = a.channels / p.small, groups = a.groups / p.small;
        const size_t lds = (2 * kSmallThreads * Vec<T>::N + 2 * width + 2 * groups) * sizeof(float);
        group_small_backward_kernel<T, Act>
            <<<dim3(p.small, a.batch), kSmallThreads, lds, s>>>(a, total);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess || a.batch == 1 || more == 0) return e;
        group_dx_kernel<T, Act, Whole, false>
            <<<more, kThreads, 0, s>>>(a, p.chunk, 0, nullptr, total);
        return hipGetLastError();
    }
    const int chunks = p.chunk.start[a.batch];
    if (chunks) {
        group_sums_kernel<T, Act, Whole>
            <<<dim3(chunks, p.slices), kThreads, 0, s>>>(a, p.chunk, partial);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const size_t lds = a.groups / p.slices * sizeof(float2);
    if (join_in_apply(a, p, 2 * a.channels * sizeof(float))) {
        const int here = more ? (a.channels + kHereCols - 1) / kHereCols : 0;
        group_dx_kernel<T, Act, Whole, true>
            <<<dim3(chunks + here, p.slices), kThreads,
               std::max(lds + 2 * a.channels / p.slices * sizeof(float), kHereCols * sizeof(float)),
               s>>>(a, p.chunk, chunks, partial, total);
        return hipGetLastError();
    }
    const dim3 grid((unsigned)((2 * a.channels + kTotalCols - 1) / kTotalCols), (unsigned)a.batch);
    group_totals_kernel<<<grid, kTotalCols * kTotalLanes, 0, s>>>(2 * a.channels, p.chunk, partial,
                                                                  total);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (chunks + more == 0) return hipSuccess;
    group_dx_kernel<T, Act, Whole, false>
        <<<dim3(chunks + more, p.slices), kThreads, lds, s>>>(a, p.chunk, chunks, partial,
                                                              total);
    return hipGetLastError();
}

template <typename T, bool Whole>
hipError_t backward_of(const GroupArgs& a, const GroupPlan& p, float* partial, float* total,
                       hipStream_t s) {
    if (a.act == P3D_ACT_SILU)
        return backward_act<T, P3D_ACT_SILU, Whole>(a, p, partial, total, s);
    if (a.act == P3D_ACT_GELU)
        return backward_act<T, P3D_ACT_GELU, Whole>(a, p, partial, total, s);
    return backward_act<T, P3D_ACT_NONE, Whole>(a, p, partial, total, s);
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

// Chunks of at least 4 rows a thread, for at most 4 workgroups a CU, all of them
// running at once. A map that does not fill those is cut into slices of whole
// groups, the narrowest of whole cache lines (8 vectors), so that it has fewer
// chunks to join: 15.9 us and the gradient 17.9, in whole rows 16.4 and 20.5, where
// 4096 rows have 512 channels of bf16. One that the caches hold is cut as far as 512
// bytes a row: 24 and 31 us, in whole rows 24 and 42.5, where 8192 rows have 2048. A
// larger one is read in whole rows: 265 us where 262,144 rows have 1024, 283 so cut
// and 319 in the narrowest slices.
GroupPlan group_norm_plan(const GroupArgs& a, p3d_dtype dt) {
    GroupPlan p;
    const int unit = dt == P3D_BF16 ? 8 : 4;
    const int64_t most = 4 * kComputeUnits;
    const int64_t n = a.items.start[a.batch];
    const int narrow = n < most * 4 * Lay(a.channels / unit).ty ? 8
                       : is_past(a, unit)                       ? a.channels
                                                                : 32;
    p.slices = 1;
    for (int d = 2; d <= a.groups; ++d)
        if (a.groups % d == 0 && a.channels / d % unit == 0 && a.channels / d / unit >= narrow)
            p.slices = d;
    // The small items' kernels: a workgroup a CU at most, slices as above, every
    // item's rows in the threads' registers.
    p.small = 0;
    int64_t longest = 0;
    for (int b = 0; b < a.batch; ++b)
        longest = std::max<int64_t>(longest, a.items.start[b + 1] - a.items.start[b]);
    if (a.channels / a.groups % unit == 0)
        for (int d = 1; d <= a.groups && d * a.batch <= kComputeUnits; ++d) {
            if (a.groups % d || (d > 1 && a.channels / d / unit < 8)) continue;
            if (longest <= (int64_t)32 / unit * SmallLay(a.channels / d / unit).ty) p.small = d;
        }
    const Lay lay(a.channels / unit / p.slices);
    const int64_t rows = std::max<int64_t>((n * p.slices + most - 1) / most, 4 * lay.ty);
    p.ty = lay.ty;
    // (Odd numbers of chunks: workgroups go round 8 dies, and of an even number a
    // die would come back to the same memory channels in every round: 320 us, not
    // 263, where 262,144 rows have 1024 channels.)
    int32_t at = 0;
    for (int b = 0; b < a.batch; ++b) {
        p.chunk.start[b] = at;
        const int32_t of = (int32_t)((a.items.start[b + 1] - a.items.start[b] + rows - 1) / rows);
        at += of > 0 ? (of - 1) | 1 : 0;
    }
    for (int b = a.batch; b <= P3D_MAX_BATCH; ++b) p.chunk.start[b] = at;
    const size_t chunks = at, batch = a.batch;
    const size_t forward = round256(chunks * a.groups * sizeof(float2)) +
                           batch * a.groups * sizeof(float4);
    const size_t backward = round256(chunks * 2 * a.channels * sizeof(float)) +
                            batch * 2 * a.channels * sizeof(float);
    p.bytes = round256(std::max(forward, backward));
    return p;
}

hipError_t launch_group_norm(const GroupArgs& a, const GroupPlan& p, p3d_dtype dt, void* ws,
                             hipStream_t s) {
    float2* partial = static_cast<float2*>(ws);
    float4* stat = reinterpret_cast<float4*>(
        static_cast<char*>(ws) +
        round256((size_t)p.chunk.start[a.batch] * a.groups * sizeof(float2)));
    const int per = a.channels / a.groups;
    if (dt == P3D_BF16)
        return per % 8 ? forward_of<Bf16, false>(a, p, partial, stat, s)
                       : forward_of<Bf16, true>(a, p, partial, stat, s);
    return per % 4 ? forward_of<float, false>(a, p, partial, stat, s)
                   : forward_of<float, true>(a, p, partial, stat, s);
}

hipError_t launch_group_norm_backward(const GroupArgs& a, const GroupPlan& p, p3d_dtype dt,
                                      void* ws, hipStream_t s) {
    float* partial = static_cast<float*>(ws);
    float* total = reinterpret_cast<float*>(
        static_cast<char*>(ws) +
        round256((size_t)p.chunk.start[a.batch] * 2 * a.channels * sizeof(float)));
    const int per = a.channels / a.groups;
    if (dt == P3D_BF16)
        return per % 8 ? backward_of<Bf16, false>(a, p, partial, total, s)
                       : backward_of<Bf16, true>(a, p, partial, total, s);
    return per % 4 ? backward_of<float, false>(a, p, partial, total, s)
                   : backward_of<float, true>(a, p, partial, total, s);
}

}  // namespace p3d
