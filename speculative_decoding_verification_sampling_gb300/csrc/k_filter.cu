// k_filter.cu -- rows of logits under temperature, top-k, top-p and min-p:
// drawing from them, and the verification rule between them.
//
// The rule is the library's (nextadmin.net lesson "Speculative Decoding", § Core
// algorithm; aiengineeringfromscratch.com Phase 10 lesson 25, § The exact rule)
// with q and p the filtered distributions; sv_filter.cuh states the filters and
// the arithmetic.
//
// A cluster of CTAs takes a row (filter_rows): each CTA copies its part to
// shared memory, and everything else works on that copy, so HBM is read once.
//   - The row's maximum, by one exchange.
//   - T = 0: its first index.
//   - top-k, k up to a few hundred: a threshold that at least k logits reach
//     comes from the threads' own maxima (a histogram of one value per thread);
//     what reaches it, a little more than k tokens, goes to the first CTA's
//     list, which is ranked there, cut and drawn from.
//   - otherwise the cut is found by histograms of counts (top-k) or of weights
//     (top-p) over the whole row: the tokens of the bin that holds the cut are
//     ranked, or where they are too many (equal logits), sorted into finer bins
//     of (logit, index) again.
// Exchanges go through shared memory of the cluster: each CTA publishes, all
// read after one cluster barrier, all come to the same answer.
//
// The verification (filter_decide) reads the rows' records, walks the positions
// of a sequence in one warp, and draws from (q_j - p_j)+ over the tokens that
// the target row keeps: from its list, or else over the vocabulary.
#include <atomic>
#include <cooperative_groups.h>
#include <cstdint>
#include <cuda_runtime.h>

#include "sv_cluster.cuh"
#include "sv_filter.cuh"
#include "sv_launch.h"

namespace sv {
namespace {

namespace cg = cooperative_groups;

constexpr int FT = 256, FW = FT / 32;   // threads and warps of a CTA
constexpr int MAX_C = 16;               // CTAs of a cluster
constexpr int BINS = 2048, BIN_EACH = BINS / FT;
constexpr int COARSE = 256;             // bins of the threads' maxima, a thread each
constexpr float RANGE = 64.0f;          // what the bins span: weights to 2^-64 of the largest
constexpr int ST_INVALID = 1;

__device__ const FilterTable kFilterTable = filter_table();

struct Vec16 {
    static __device__ __forceinline__ uint4 load(const void *p)
    {
        uint4 v;
        asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                     : "l"(p));
        return v;
    }
};
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Elements of a row, N to a 16-byte vector.
struct RowF32 {
    static constexpr int N = 4, ES = 4;
    static constexpr uint32_t NONE = 0xff800000u;   // words of minus infinity
    static __device__ __forceinline__ float get(const uint4 &v, int k)
    {
        return __uint_as_float(k == 0 ? v.x : k == 1 ? v.y : k == 2 ? v.z : v.w);
    }
    static __device__ __forceinline__ float one(const void *p, size_t i) { return __ldg(static_cast<const float *>(p) + i); }
    static __device__ __forceinline__ uint4 pack(const float (&x)[N])
    {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
    static __device__ __forceinline__ float largest(const uint4 &v)
    {
        return max_nan(max_nan(get(v, 0), get(v, 1)), max_nan(get(v, 2), get(v, 3)));
    }
};
struct RowBF16 {
    static constexpr int N = 8, ES = 2;
    static constexpr uint32_t NONE = 0xff80ff80u;
    static __device__ __forceinline__ float get(const uint4 &v, int k)
    {
        const uint32_t w = k < 2 ? v.x : k < 4 ? v.y : k < 6 ? v.z : v.w;
        return __uint_as_float(k & 1 ? w & 0xffff0000u : w << 16);
    }
    static __device__ __forceinline__ float one(const void *p, size_t i)
    {
        return __uint_as_float((uint32_t)__ldg(static_cast<const uint16_t *>(p) + i) << 16);
    }
    static __device__ __forceinline__ uint4 pack(const float (&x)[N])
    {
        uint32_t w[4];
        for (int k = 0; k < 4; ++k)
            w[k] = (__float_as_uint(x[2 * k]) >> 16) | (__float_as_uint(x[2 * k + 1]) & 0xffff0000u);
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b)
    {
        uint32_t r;
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    static __device__ __forceinline__ float largest(const uint4 &v)
    {
        const uint32_t w = max2(max2(v.x, v.y), max2(v.z, v.w));
        return max_nan(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
};

struct RowShared {
    u64 slot[2][4][FW];   // published, by round parity: up to four numbers per warp
    u64 sums[FW], sums2[FW];
    float2 table[64];
    uint32_t hist[BINS], hist_hi[BINS];   // counts, or sums in two words
    u64 key[FILTER_CAP];  // the list: (logit, order) keys,
    u64 w[FILTER_CAP];    // weights,
    int32_t x[FILTER_CAP];   // tokens
    u64 cut, base;
    double least;         // T ln(min_p)
    float c_hi, c_lo, cut_x;
    int lo, hi, cut_token;
};
constexpr size_t ROW_HDR = (sizeof(RowShared) + 127) & ~(size_t)127;

// ------------------------------------------------------------------ sums
__device__ __forceinline__ u64 shfl_up64(u64 v, int o)
{
    return __shfl_up_sync(0xffffffffu, v, o);
}
__device__ __forceinline__ u64 warp_sum64(u64 v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ u64 warp_scan64(u64 v, int lane)   // inclusive
{
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 y = shfl_up64(v, o);
        v += lane >= o ? y : 0;
    }
    return v;
}
// Sum of the threads ahead of this one; `total` of all.
__device__ __forceinline__ u64 block_scan64(u64 v, u64 *sums, u64 &total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const u64 in = warp_scan64(v, lane);
    __syncthreads();   // the last call's reads
    if (lane == 31)
        sums[warp] = in;
    __syncthreads();
    u64 before = 0;
    total = 0;
#pragma unroll
    for (int k = 0; k < FW; ++k) {
        before += k < warp ? sums[k] : 0;
        total += sums[k];
    }
    return before + in - v;
}

// ------------------------------------------------------------------ one row
template <class T>
struct Row {
    RowShared &S;
    cg::cluster_group cl;
    const uint4 *data;      // this CTA's part
    int C, rank, lane, warp;
    int v0, seg0, seg1;     // vectors: of the part, of this warp's segment
    int off, V;             // tokens ahead of the row in its first vector
    int len;                // vectors of a segment
    uint32_t round = 0;

    __device__ __forceinline__ Row(RowShared &s, const uint4 *d, int nv, int o, int vocab)
        : S(s), cl(cg::this_cluster()), data(d), C((int)cl_size()), rank((int)cl_rank()), lane(threadIdx.x & 31),
          warp(threadIdx.x >> 5), off(o), V(vocab)
    {
        len = ((nv + C * FW - 1) / (C * FW) + 31) & ~31;
        v0 = min(rank * FW * len, nv);
        seg0 = min((rank * FW + warp) * len, nv);
        seg1 = min(seg0 + len, nv);
    }
    __device__ __forceinline__ int segment() const { return rank * FW + warp; }
    // f(logit, token) for every token of this warp's segment, in any order
    template <class F>
    __device__ __forceinline__ void each(F f) const
    {
        for (int v = seg0 + lane; v < seg1; v += 32) {
            const uint4 q = data[v - v0];
#pragma unroll
            for (int k = 0; k < T::N; ++k)
                f(T::get(q, k), v * T::N + k - off);
        }
    }
    // Publishes n numbers per warp (the same in every lane) and returns where warp w of CTA r has them.
    struct Board {
        u64 *at;
        cg::cluster_group cl;
        __device__ __forceinline__ u64 get(int i, int segment) const
        {
            return *cl.map_shared_rank(at + i * FW + segment % FW, segment / FW);
        }
    };
    template <int N>
    __device__ __forceinline__ Board publish(const u64 (&x)[N])
    {
        u64 *at = &S.slot[round & 1][0][0];
        ++round;
        if (lane == 0)
#pragma unroll
            for (int i = 0; i < N; ++i)
                at[i * FW + warp] = x[i];
        cl_sync();
        return Board{at, cl};
    }
    // A number per warp: their sum ahead of this warp's, and in all
    __device__ __forceinline__ u64 ahead(const Board &b, int i, u64 &total) const
    {
        u64 all = 0, mine = 0;
        for (int s = lane; s < C * FW; s += 32) {
            const u64 x = b.get(i, s);
            all += x;
            mine += s < segment() ? x : 0;
        }
        total = warp_sum64(all);
        return warp_sum64(mine);
    }
    __device__ __forceinline__ u64 sum(const Board &b, int i) const
    {
        u64 total;
        ahead(b, i, total);
        return total;
    }
    template <class F>
    __device__ __forceinline__ u64 fold(const Board &b, int i, u64 start, F f) const
    {
        u64 x = start;
        for (int s = lane; s < C * FW; s += 32)
            x = f(x, b.get(i, s));
#pragma unroll
        for (int o = 16; o; o >>= 1)
            x = f(x, (u64)__shfl_xor_sync(0xffffffffu, x, o));
        return x;
    }

    static __device__ __forceinline__ u64 key_of(float x, int token)
    {
        return (u64)filter_key(x) << 32 | (0xffffffffu - (uint32_t)token);
    }

    // The tokens for which keep(x, token) holds, `n` in all and `before` of them ahead of this warp, go to
    // the first CTA's list in ascending order.  by_place: the key's low word tells the place in the list.
    template <class F>
    __device__ __forceinline__ void collect(F keep, int before, bool by_place)
    {
        u64 *key = cl.map_shared_rank(S.key, 0);
        int32_t *tok = cl.map_shared_rank(S.x, 0);
        for (int v = seg0; v < seg1; v += 32) {
            uint32_t mine = 0;
            uint4 q = make_uint4(0, 0, 0, 0);
            if (v + lane < seg1) {
                q = data[v + lane - v0];
#pragma unroll
                for (int k = 0; k < T::N; ++k)
                    mine |= (keep(T::get(q, k), (v + lane) * T::N + k - off) ? 1u : 0u) << k;
            }
            if (!__any_sync(0xffffffffu, mine))
                continue;
            int cnt = __popc(mine), in = cnt;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, in, o);
                in += lane >= o ? y : 0;
            }
            int at = before + in - cnt;
            before += __shfl_sync(0xffffffffu, in, 31);
#pragma unroll
            for (int k = 0; k < T::N; ++k)
                if ((mine >> k & 1) && at < FILTER_CAP) {
                    const int token = (v + lane) * T::N + k - off;
                    key[at] = by_place ? (u64)filter_key(T::get(q, k)) << 32 | (0xffffffffu - (uint32_t)at)
                                       : key_of(T::get(q, k), token);
                    tok[at] = token;
                    ++at;
                }
        }
        cl_sync();
    }

    // The first CTA sorts the n keys of its list, largest first.
    __device__ __forceinline__ void sort(int n)
    {
        int size = 32;
        while (size < n)
            size *= 2;
        for (int i = n + threadIdx.x; i < size; i += FT)
            S.key[i] = 0;
        for (int a = 2; a <= size; a *= 2)
            for (int b = a / 2; b; b /= 2) {
                __syncthreads();
                for (int i = threadIdx.x; i < size / 2; i += FT) {
                    const int lo = 2 * i - (i & (b - 1)), hi = lo + b;
                    const u64 x = S.key[lo], y = S.key[hi];
                    if ((x < y) == ((lo & a) == 0)) {
                        S.key[lo] = y;
                        S.key[hi] = x;
                    }
                }
            }
        __syncthreads();
    }

    // The cut by a count (the first `share` tokens) or by a sum (the tokens ahead of which less than `share` of
    // the whole lies), among the tokens with keys from `floor` on: the key of the last token that stays.
    template <bool SUM>
    __device__ u64 cut(const FilterWeight &W, double share, u64 floor)
    {
        u64 from = 0, to = ~0ull, base = 0, target = SUM ? 0 : (u64)share;   // keys in question; what lies ahead of them
        int shift = 0;
        const float step = W.c_hi * ((float)BINS / RANGE);
#pragma unroll 1
        for (int level = 0; level < 10; ++level) {
            for (int i = threadIdx.x; i < BINS; i += FT)
                S.hist[i] = S.hist_hi[i] = 0;
            if (threadIdx.x == 0)
                S.lo = -1;
            __syncthreads();
            auto bin_of = [&](float x, int token) {
                if (!(x > -F_INF))
                    return -1;
                const u64 k = key_of(x, token);
                if (k < floor || k < from || k > to)
                    return -1;
                return level ? (int)((to - k) >> shift) : min(BINS - 1, (int)((W.m - x) * step));
            };
            each([&](float x, int token) {
                const int b = bin_of(x, token);
                if (b < 0)
                    return;
                if constexpr (SUM) {
                    const u64 w = W(x);
                    if (w == 0)
                        return;
                    const uint32_t lo = (uint32_t)w;
                    const uint32_t hi = (uint32_t)(w >> 32) + (atomicAdd(&S.hist[b], lo) > ~lo);
                    if (hi)
                        atomicAdd(&S.hist_hi[b], hi);
                } else {
                    atomicAdd(&S.hist[b], 1u);
                }
            });
            __syncthreads();
            cl_sync();
            // all CTAs' bins, a thread's in a row
            u64 bins[BIN_EACH], mine = 0, all;
#pragma unroll
            for (int k = 0; k < BIN_EACH; ++k)
                bins[k] = 0;
            for (int r = 0; r < C; ++r) {
                const uint32_t *lo = cl.map_shared_rank(S.hist, r) + threadIdx.x * BIN_EACH;
                const uint32_t *hi = cl.map_shared_rank(S.hist_hi, r) + threadIdx.x * BIN_EACH;
#pragma unroll
                for (int k = 0; k < BIN_EACH; ++k)
                    bins[k] += lo[k] | (SUM ? (u64)hi[k] << 32 : 0);
            }
#pragma unroll
            for (int k = 0; k < BIN_EACH; ++k)
                mine += bins[k];
            u64 at = base + block_scan64(mine, S.sums, all);
            if (SUM && level == 0)
                target = max((u64)ceil(share * (double)all), 1ull);   // less than it: the same as less than the share
            if (at < target && at + mine >= target) {
#pragma unroll
                for (int k = 0; k < BIN_EACH; ++k) {
                    if (at < target && at + bins[k] >= target) {
                        S.lo = threadIdx.x * BIN_EACH + k;
                        S.base = at;
                    }
                    at += bins[k];
                }
            }
            __syncthreads();
            const int bin = S.lo;
            if (bin < 0) {
                cl_sync();      // the others may still read this CTA's bins
                return floor;   // there are no more
            }
            base = S.base;
            u64 n = 0, least = ~0ull, most = 0;
            each([&](float x, int token) {
                if (bin_of(x, token) == bin) {
                    const u64 k = key_of(x, token);
                    ++n;
                    least = k < least ? k : least;
                    most = k > most ? k : most;
                }
            });
            n = warp_sum64(n);
#pragma unroll
            for (int o = 16; o; o >>= 1) {
                const u64 a = __shfl_xor_sync(0xffffffffu, least, o), b = __shfl_xor_sync(0xffffffffu, most, o);
                least = a < least ? a : least;
                most = b > most ? b : most;
            }
            const u64 told[3] = {n, least, most};
            const Board board = publish(told);
            u64 total;
            const int before = (int)ahead(board, 0, total);
            from = fold(board, 1, ~0ull, [](u64 a, u64 b) { return a < b ? a : b; });
            to = fold(board, 2, 0, [](u64 a, u64 b) { return a > b ? a : b; });
            if (total <= FILTER_CAP) {
                collect([&](float x, int token) {
                    const u64 k = key_of(x, token);
                    return x > -F_INF && k >= from && k <= to;
                }, before, false);
                if (rank == 0) {
                    const int count = (int)total;
                    sort(count);
                    if constexpr (SUM) {
                        constexpr int E = FILTER_CAP / FT;
                        u64 w[E], s = 0;
#pragma unroll
                        for (int k = 0; k < E; ++k) {
                            const int i = threadIdx.x * E + k;
                            w[k] = i < count ? W(filter_value((uint32_t)(S.key[i] >> 32))) : 0;
                            s += w[k];
                        }
                        at = base + block_scan64(s, S.sums, all);
                        // the token whose weight reaches the target is the last
#pragma unroll
                        for (int k = 0; k < E; ++k) {
                            if (at < target && at + w[k] >= target)
                                S.cut = S.key[threadIdx.x * E + k];
                            at += w[k];
                        }
                    } else if (threadIdx.x == 0) {
                        S.cut = S.key[min((int)(target - base), count) - 1];
                    }
                }
                cl_sync();
                return *cl.map_shared_rank(&S.cut, 0);
            }
            const u64 span = to - from;
            shift = max(0, 64 - __clzll((long long)span) - 11);
        }
        return from;
    }

    // The sum of the weights from `cut` on.
    __device__ __forceinline__ u64 mass(const FilterWeight &W, u64 cut) const
    {
        const float x0 = filter_value((uint32_t)(cut >> 32));
        const uint32_t last = 0xffffffffu - (uint32_t)cut;
        u64 s = 0;
        each([&](float x, int token) {
            if (cut == 0 || x > x0 || (x == x0 && (uint32_t)token <= last))
                s += W(x);
        });
        return warp_sum64(s);
    }
};

// Copies this CTA's part of a row to shared memory: 16 bytes at a time, the vectors at the row's ends element
// by element (what is not the row's becomes minus infinity).  Returns the thread's largest logit (NaN if any is).
template <class T>
__device__ __forceinline__ float load_part(const Row<T> &R, const void *row, uint4 *data, int nv)
{
    const uint8_t *base = reinterpret_cast<const uint8_t *>(row) - R.off * T::ES;   // a 16-byte boundary
    float top = -F_INF;
    auto edge = [&](int v) {
        float x[T::N];
#pragma unroll
        for (int k = 0; k < T::N; ++k) {
            const int i = v * T::N + k - R.off;
            x[k] = i >= 0 && i < R.V ? T::one(row, i) : -F_INF;
        }
        return T::pack(x);
    };
    constexpr int FLY = 8;
    const bool ragged = R.off != 0 || (R.off + R.V) % T::N != 0;
    for (int v = R.seg0 + R.lane; v < R.seg1; v += 32 * FLY) {
        uint4 q[FLY];
#pragma unroll
        for (int u = 0; u < FLY; ++u) {
            const int at = v + 32 * u;
            q[u] = make_uint4(T::NONE, T::NONE, T::NONE, T::NONE);
            if (at < R.seg1)
                q[u] = ragged && (at == 0 || at == nv - 1) ? edge(at) : Vec16::load(base + (size_t)at * 16);
        }
#pragma unroll
        for (int u = 0; u < FLY; ++u) {
            if (v + 32 * u < R.seg1)
                data[v + 32 * u - R.v0] = q[u];
            top = max_nan(top, T::largest(q[u]));
        }
    }
    return top;
}

template <class T, bool VERIFY>
__global__ void __launch_bounds__(FT) filter_rows(const __grid_constant__ FilterParams P)
{
    extern __shared__ __align__(128) uint8_t smem[];
    RowShared &S = *reinterpret_cast<RowShared *>(smem);
    uint4 *data = reinterpret_cast<uint4 *>(smem + ROW_HDR);
    const int row = (int)cl_id(), V = P.V, tid = threadIdx.x;
    const int per = VERIFY ? 2 * P.K + 1 : P.K;
    const int b = row / per, i = row - b * per;
    const bool draft = VERIFY && i > P.K;
    const FilterSet &F = draft ? P.df : P.f;
    const uint8_t *src = static_cast<const uint8_t *>(draft ? P.draft : P.logits) +
                         (size_t)(VERIFY ? draft ? b * P.K + i - P.K - 1 : b * (P.K + 1) + i : row) * V * T::ES;
    const int off = (int)((reinterpret_cast<uintptr_t>(src) & 15) / T::ES);
    const int nv = (off + V + T::N - 1) / T::N;
    Row<T> R(S, data, nv, off, V);
    const int rank = R.rank;

    const float temp = F.T ? __ldg(F.T + b) : 1.0f, p = F.p ? __ldg(F.p + b) : 1.0f;
    const float least = F.least ? __ldg(F.least + b) : 0.0f;
    int k = F.k ? __ldg(F.k + b) : 0;
    k = k <= 0 || k > V ? V : k;
    float u = 0.0f;
    if (!VERIFY)
        u = __ldg(P.uniforms + row);
    int code = !(temp >= 0.0f && temp < F_INF) || p != p || !(least <= 1.0f) || !(u >= 0.0f && u < 1.0f) ? ST_INVALID : 0;

    if (tid < 64)
        S.table[tid] = kFilterTable.t[tid];
    if (tid == FT - 32) {
        // temperatures beyond 2^-100 and 2^100 count as these
        const double t = fmin(fmax((double)temp, 0x1p-100), 0x1p100), c = 1.4426950408889634 / t;
        S.c_hi = temp > 0.0f ? (float)c : 0.0f;
        S.c_lo = temp > 0.0f ? (float)(c - (double)S.c_hi) : 0.0f;
        S.least = least > 0.0f ? t * log((double)least) : 0.0;
    }
    const float mine = load_part<T>(R, src, data, nv);
    float m = mine;
#pragma unroll
    for (int o = 16; o; o >>= 1)
        m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    {
        __syncthreads();
        const u64 x[1] = {__float_as_uint(m)};
        const auto board = R.publish(x);
        m = __uint_as_float((uint32_t)R.fold(board, 0, 0xff800000u, [](u64 a, u64 b) {
            return (u64)__float_as_uint(max_nan(__uint_as_float((uint32_t)a), __uint_as_float((uint32_t)b)));
        }));
    }
    if (code == 0 && !(m > -F_INF && m < F_INF))
        code = ST_NONFINITE;
    FilterRow rec{};
    rec.n = -1;
    rec.code = code;
    // what a row comes to: its record, or a token and its probability
    auto finish = [&](int token, float prob) {
        if (VERIFY) {
            P.rows[row] = rec;
        } else {
            P.out_tokens[row] = code ? -1 : token;
            if (P.out_prob)
                P.out_prob[row] = code ? __int_as_float(0x7fc00000) : prob;
            if (code && P.status)
                atomicCAS(P.status, 0, code);
        }
    };
    if (code) {
        if (rank == 0 && tid == 0)
            finish(-1, 0.0f);
        cl_sync();
        return;
    }
    const FilterWeight W(m, S.c_hi, S.c_lo, S.table);
    rec.m = m;
    rec.c_hi = S.c_hi;
    rec.c_lo = S.c_lo;

    if (temp == 0.0f) {
        u64 first = ~0ull;
        R.each([&](float x, int token) {
            if (x == m && (u64)token < first)
                first = (u64)token;
        });
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            const u64 a = __shfl_xor_sync(0xffffffffu, first, o);
            first = a < first ? a : first;
        }
        const u64 x[1] = {first};
        const auto board = R.publish(x);
        first = R.fold(board, 0, ~0ull, [](u64 a, u64 b) { return a < b ? a : b; });
        rec.cut = m;
        rec.last = (uint32_t)first;
        rec.Z = 1ull << 43;
        if (rank == 0 && tid == 0)
            finish((int)first, 1.0f);
        cl_sync();
        return;
    }

    const float xmin = least > 0.0f ? __double2float_ru((double)m + S.least) : -F_INF;
    // ---- a threshold that what is kept reaches, for lists
    const bool few = k <= FILTER_CAP / 4 && k <= 32 * R.C;   // there are 256 C threads' maxima
    bool listed = V <= FILTER_CAP;
    float t0 = p < 1.0f ? -F_INF : xmin;   // top-p's total counts what min-p drops
    if (!listed && few) {
        S.hist[tid] = 0;
        __syncthreads();
        if (mine > -F_INF)
            atomicAdd(&S.hist[min(COARSE - 1, (int)((m - mine) * (W.c_hi * (COARSE / RANGE))))], 1u);
        if (tid == 0)
            S.lo = COARSE - 1;
        __syncthreads();
        cl_sync();
        u64 n = 0, all;
        for (int r = 0; r < R.C; ++r)
            n += R.cl.map_shared_rank(S.hist, r)[tid];
        const u64 before = block_scan64(n, S.sums, all);
        if (before < (u64)k && before + n >= (u64)k)
            S.lo = tid;
        __syncthreads();
        const int lo = S.lo;
        // the bin's lower end, and what it may be off by
        if (lo < COARSE - 1)
            t0 = fmaxf(t0, m - (float)(lo + 1) * (RANGE / COARSE / W.c_hi) * 1.000001f - fabsf(m) * 0x1p-21f);
        listed = true;
    } else if (!listed && p >= 1.0f && least > 0.0f) {
        listed = true;
    }
    if (listed) {
        auto keep = [&](float x, int) { return x >= t0 && x > -F_INF; };
        u64 n = 0;
        R.each([&](float x, int token) { n += keep(x, token); });
        const u64 x[1] = {warp_sum64(n)};
        const auto board = R.publish(x);
        u64 total;
        const int before = (int)R.ahead(board, 0, total);
        if (total > FILTER_CAP) {
            listed = false;
        } else {
            R.collect(keep, before, true);
            if (rank != 0)
                return;   // nothing of this CTA is read any more
            const int count = (int)total;
            R.sort(count);
            constexpr int E = FILTER_CAP / FT;
            u64 w[E], s = 0, ones;
            int place[E];
            float xs[E];
            for (int e = 0; e < E; ++e) {
                const int r = tid * E + e;
                const u64 key = r < count ? S.key[r] : 0;
                xs[e] = filter_value((uint32_t)(key >> 32));
                place[e] = (int)(0xffffffffu - (uint32_t)key);
                w[e] = r < count && r < k ? W(xs[e]) : 0;
                s += w[e];
            }
            u64 at = block_scan64(s, S.sums, ones);
            // less than p of the total: the same as less than the next whole number
            const u64 target = p >= 1.0f ? ~0ull : (u64)ceil((double)fmaxf(p, 0.0f) * (double)ones);
            int stay = 0;
            bool kept[E];
            for (int e = 0; e < E; ++e) {
                const int r = tid * E + e;
                kept[e] = r < count && (r == 0 || (r < k && at < target && xs[e] >= xmin));
                at += w[e];
                stay += kept[e];
            }
            for (int e = 0; e < E; ++e)
                if (tid * E + e < count)
                    S.w[place[e]] = kept[e] ? w[e] : 0;
            // the last kept key's token is the cut
            const int last = (int)block_scan64(stay, S.sums2, ones) + stay;
            if (stay > 0 && last == (int)ones)
                for (int e = 0; e < E; ++e)
                    if (kept[e] && (e == E - 1 || !kept[e + 1])) {
                        S.cut_x = xs[e];
                        S.cut_token = S.x[place[e]];
                    }
            __syncthreads();
            s = 0;
            for (int e = 0; e < E; ++e) {
                w[e] = tid * E + e < count ? S.w[tid * E + e] : 0;
                s += w[e];
            }
            u64 Z;
            u64 upto = block_scan64(s, S.sums, Z);
            if (VERIFY) {
                rec.cut = S.cut_x;
                rec.last = (uint32_t)S.cut_token;
                rec.Z = Z;
                rec.n = draft ? -1 : 0;
                if (!draft) {
                    // tokens of no weight need not be listed
                    int c = 0;
                    for (int e = 0; e < E; ++e)
                        c += w[e] != 0;
                    u64 kept_all;
                    int to = (int)block_scan64(c, S.sums2, kept_all);
                    const size_t list = (size_t)(b * (P.K + 1) + i) * FILTER_CAP;
                    for (int e = 0; e < E; ++e)
                        if (w[e]) {
                            P.list_x[list + to] = S.x[tid * E + e];
                            P.list_w[list + to++] = w[e];
                        }
                    rec.n = (int)kept_all;
                }
                if (tid == 0)
                    finish(-1, 0.0f);
            } else {
                const u64 v = (u64)((double)u * (double)Z);
                for (int e = 0; e < E; ++e) {
                    if (w[e] && upto <= v && upto + w[e] > v)
                        finish(S.x[tid * E + e], (float)((double)w[e] / (double)Z));
                    upto += w[e];
                }
            }
            return;
        }
    }

    // ---- the cut by histograms over the row
    u64 cut = 0;
    if (k < V)
        cut = R.template cut<false>(W, (double)k, 0);
    if (p < 1.0f)
        cut = R.template cut<true>(W, (double)fmaxf(p, 0.0f), cut);
    if (least > 0.0f) {
        const u64 c = (u64)filter_key(xmin) << 32;
        cut = c > cut ? c : cut;
    }
    const u64 x[1] = {R.mass(W, cut)};
    const auto board = R.publish(x);
    u64 Z;
    const u64 before = R.ahead(board, 0, Z);
    rec.cut = cut ? filter_value((uint32_t)(cut >> 32)) : -F_INF;
    rec.last = 0xffffffffu - (uint32_t)cut;
    rec.Z = Z;
    if (VERIFY) {
        if (rank == 0 && tid == 0)
            finish(-1, 0.0f);
    } else {
        // the segment on which the uniform falls, then the vector, by its whole CTA
        const u64 v = (u64)((double)u * (double)Z);
        if (tid == 0)
            S.hi = 0;
        __syncthreads();
        if (R.lane == 0 && before <= v && before + x[0] > v) {
            S.hi = 1;
            S.lo = R.warp;
            S.cut = before;
        }
        __syncthreads();
        if (S.hi) {
            const int a0 = min((rank * FW + S.lo) * R.len, nv), a1 = min(a0 + R.len, nv);
            u64 at = S.cut;
            for (int a = a0; a < a1; a += FT) {
                u64 w[T::N], s = 0;
                const bool in = a + tid < a1;
                const uint4 q = in ? data[a + tid - R.v0] : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int e = 0; e < T::N; ++e) {
                    const float y = T::get(q, e);
                    const int token = (a + tid) * T::N + e - off;
                    w[e] = in && (y > rec.cut || (y == rec.cut && (uint32_t)token <= rec.last)) ? W(y) : 0;
                    s += w[e];
                }
                u64 all;
                u64 upto = at + block_scan64(s, S.sums, all);
#pragma unroll
                for (int e = 0; e < T::N; ++e) {
                    if (w[e] && upto <= v && upto + w[e] > v)
                        finish((a + tid) * T::N + e - off, (float)((double)w[e] / (double)Z));
                    upto += w[e];
                }
                at += all;
            }
        }
    }
    cl_sync();
}

// ------------------------------------------------------------------ the rule
struct DecideShared {
    u64 slot[2][2][FW];
    u64 sums[FW];
    float2 table[64];
    int j, code, seg;
    u64 before;
};

template <class T>
__global__ void __launch_bounds__(FT) filter_decide(const __grid_constant__ FilterParams P)
{
    __shared__ DecideShared S;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b = (int)cl_id(), rank = (int)cl_rank(), C = (int)cl_size(), K = P.K, V = P.V;
    const auto cl = cg::this_cluster();
    if (tid < 64)
        S.table[tid] = kFilterTable.t[tid];
    __syncthreads();
    pdl_wait();
    const FilterRow *rows = P.rows + (size_t)b * (2 * K + 1);
    const uint8_t *tgt = static_cast<const uint8_t *>(P.logits) + (size_t)b * (K + 1) * V * T::ES;
    const uint8_t *drf = static_cast<const uint8_t *>(P.draft) + (size_t)b * K * V * T::ES;
    auto of = [&](const FilterRow &r) { return FilterWeight(r.m, r.c_hi, r.c_lo, S.table); };
    auto weight = [](const FilterRow &r, const FilterWeight &W, float x, int token) -> u64 {
        return x > r.cut || (x == r.cut && (uint32_t)token <= r.last) ? W(x) : 0;
    };
    if (warp == 0) {
        // a position per lane
        bool go = false;
        int code = 0;
        if (lane <= K) {
            const FilterRow q = rows[lane];
            const float u = __ldg(P.uniforms + ((size_t)b * (K + 1) + lane) * 2);
            const float v = __ldg(P.uniforms + ((size_t)b * (K + 1) + lane) * 2 + 1);
            const bool fine = (lane == K || (u >= 0.0f && u < 1.0f)) && v >= 0.0f && v < 1.0f;
            code = fine ? q.code : ST_INVALID;
            if (lane < K) {
                const FilterRow p = rows[K + 1 + lane];
                const int d = __ldg(P.tokens + (size_t)b * K + lane);
                if (code != ST_INVALID && p.code == ST_INVALID)
                    code = ST_INVALID;
                if (code != ST_INVALID && (d < 0 || d >= V))
                    code = ST_TOKEN;
                if (code == 0)
                    code = p.code;
                if (code == 0) {
                    const double wq = (double)weight(q, of(q), T::one(tgt, (size_t)lane * V + d), d);
                    const double wp = (double)weight(p, of(p), T::one(drf, (size_t)lane * V + d), d);
                    // u p < q
                    go = (double)u * wp * (double)q.Z < wq * (double)p.Z;
                }
            }
        }
        const int j = __ffs(~__ballot_sync(0xffffffffu, go)) - 1;
        code = __shfl_sync(0xffffffffu, code, j);
        if (lane == 0) {
            S.j = j;
            S.code = code;
        }
        if (rank == 0 && lane <= K) {
            P.out_tokens[(size_t)b * (K + 1) + lane] = code == 0 && lane < j ? __ldg(P.tokens + (size_t)b * K + lane) : -1;
            if (lane == 0) {
                P.out_len[b] = code ? -code : j;
                if (code && P.status)
                    atomicCAS(P.status, 0, code);
            }
        }
    }
    __syncthreads();
    const int j = S.j;
    if (S.code)
        return;   // every CTA of the cluster
    const FilterRow q = rows[j];
    FilterRow p{};
    const bool bonus = j == K;
    if (!bonus)
        p = rows[K + 1 + j];
    const FilterWeight Wq = of(q), Wp = of(p);
    const double iq = 1.0 / (double)q.Z, ip = bonus ? 0.0 : 1.0 / (double)p.Z;
    const double v = (double)__ldg(P.uniforms + ((size_t)b * (K + 1) + j) * 2 + 1);
    const size_t row_q = (size_t)j * V;
    // (q - p)+ in units of 2^-62; nothing for equal ones, so the products are not to be fused with the difference
    auto left = [&](u64 wq, u64 wp) -> u64 {
        const double r = __dsub_rn(__dmul_rn((double)wq, iq), __dmul_rn((double)wp, ip));
        return r > 0.0 ? (u64)__double2ll_rn(r * 0x1p62) : 0;
    };
    int32_t *out = P.out_tokens + (size_t)b * (K + 1) + j;
    if (q.n >= 0) {
        if (rank != 0)
            return;
        constexpr int E = FILTER_CAP / FT;
        const size_t list = ((size_t)b * (K + 1) + j) * FILTER_CAP;
        u64 wq[E], r[E], s = 0, sq = 0;
        int x[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int i = tid * E + e;
            wq[e] = r[e] = 0;
            x[e] = 0;
            if (i < q.n) {
                x[e] = P.list_x[list + i];
                wq[e] = P.list_w[list + i];
                r[e] = bonus ? wq[e] : left(wq[e], weight(p, Wp, T::one(drf, row_q + x[e]), x[e]));
            }
            s += r[e];
            sq += wq[e];
        }
        u64 all, all_q;
        u64 upto = block_scan64(s, S.sums, all);
        const u64 upto_q = block_scan64(sq, S.sums, all_q);
        if (all == 0) {
            // nothing is left of the target beside the draft: from the target itself
            upto = upto_q;
            all = all_q;
#pragma unroll
            for (int e = 0; e < E; ++e)
                r[e] = wq[e];
        }
        const u64 at = (u64)(v * (double)all);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            if (r[e] && upto <= at && upto + r[e] > at)
                *out = x[e];
            upto += r[e];
        }
        return;
    }
    // over the vocabulary: a segment per warp, then the segment on which the uniform falls
    const int each = (V + C * FW - 1) / (C * FW);
    const int me = rank * FW + warp, e0 = min(me * each, V), e1 = min(e0 + each, V);
    auto rest = [&](int token, u64 &wq) -> u64 {
        wq = weight(q, Wq, T::one(tgt, row_q + token), token);
        return bonus || wq == 0 ? wq : left(wq, weight(p, Wp, T::one(drf, row_q + token), token));
    };
    u64 s = 0, sq = 0;
    for (int x = e0 + lane; x < e1; x += 32) {
        u64 wq;
        s += rest(x, wq);
        sq += wq;
    }
    s = warp_sum64(s);
    sq = warp_sum64(sq);
    if (lane == 0) {
        S.slot[0][0][warp] = s;
        S.slot[0][1][warp] = sq;
    }
    if (tid == 0)
        S.seg = -1;
    cl_sync();
    u64 all = 0, all_q = 0, before = 0, before_q = 0;
    for (int g = lane; g < C * FW; g += 32) {
        const u64 a = *cl.map_shared_rank(&S.slot[0][0][g % FW], g / FW), c = *cl.map_shared_rank(&S.slot[0][1][g % FW], g / FW);
        all += a;
        all_q += c;
        before += g < me ? a : 0;
        before_q += g < me ? c : 0;
    }
    all = warp_sum64(all);
    all_q = warp_sum64(all_q);
    before = warp_sum64(before);
    before_q = warp_sum64(before_q);
    const bool whole = all == 0;
    if (whole) {
        all = all_q;
        before = before_q;
        s = sq;
    }
    const u64 at = (u64)(v * (double)all);
    if (lane == 0 && before <= at && before + s > at) {
        S.seg = warp;
        S.before = before;
    }
    __syncthreads();
    if (S.seg >= 0) {
        const int a0 = min((rank * FW + S.seg) * each, V), a1 = min(a0 + each, V);
        u64 upto = S.before;
        for (int a = a0; a < a1; a += FT) {
            u64 r = 0, wq, sum;
            if (a + tid < a1) {
                r = rest(a + tid, wq);
                r = whole ? wq : r;
            }
            const u64 mine = upto + block_scan64(r, S.sums, sum);
            if (r && mine <= at && mine + r > at)
                *out = a + tid;
            upto += sum;
        }
    }
    cl_sync();
}

// ------------------------------------------------------------------ host
template <class Kern, class Par>
cudaError_t launch_clusters(Kern kern, long long clusters, int csize, size_t smem, bool after, cudaStream_t stream,
                            const Par &P)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(clusters * csize));
    cfg.blockDim = dim3(FT);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim = {(unsigned)csize, 1, 1};
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = after ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, P);
}

template <class T, bool VERIFY>
cudaError_t rows(const FilterParams &P, int sms, cudaStream_t stream)
{
    const long long n = (long long)P.B * (VERIFY ? 2 * P.K + 1 : P.K);
    const long long bytes = ((long long)P.V + T::N) * T::ES;
    // parts of 48 KB at most, so that several CTAs share an SM; smaller ones where there are few rows
    int C = 1;
    while (C < MAX_C && (bytes / C > 48 * 1024 || (n * C < 2 * sms && bytes / C > 4096)))
        C *= 2;
    const long long nv = (P.V + T::N - 1) / T::N + 1;
    const long long part = ((nv + (long long)C * FW - 1) / ((long long)C * FW) + 31) / 32 * 32 * FW;
    const size_t smem = ROW_HDR + (size_t)part * 16;
    static std::atomic<uint64_t> raised{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(raised.load(std::memory_order_relaxed) & bit)) {
        e = cudaFuncSetAttribute(filter_rows<T, VERIFY>, cudaFuncAttributeMaxDynamicSharedMemorySize, 232448);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(filter_rows<T, VERIFY>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess)
            return e;
        raised.fetch_or(bit, std::memory_order_relaxed);
    }
    return launch_clusters(filter_rows<T, VERIFY>, n, C, smem, false, stream, P);
}

}  // namespace

int filter_max_v() { return FILTER_MAX_V; }

size_t filter_workspace(int B, int K)
{
    return (size_t)B * ((2 * K + 1) * sizeof(FilterRow) + (size_t)(K + 1) * FILTER_CAP * 12);
}

void filter_place(FilterParams &P, void *workspace)
{
    char *w = static_cast<char *>(workspace);
    P.rows = reinterpret_cast<FilterRow *>(w);
    w += (size_t)P.B * (2 * P.K + 1) * sizeof(FilterRow);
    P.list_w = reinterpret_cast<u64 *>(w);
    w += (size_t)P.B * (P.K + 1) * FILTER_CAP * 8;
    P.list_x = reinterpret_cast<int32_t *>(w);
}

cudaError_t launch_filter_sample(const FilterParams &P, int tdt, int sms, cudaStream_t stream, int *launches)
{
    *launches = 0;
    cudaError_t e = P.status ? cudaMemsetAsync(P.status, 0, sizeof(int32_t), stream) : cudaSuccess;
    if (e == cudaSuccess)
        e = tdt ? rows<RowBF16, false>(P, sms, stream) : rows<RowF32, false>(P, sms, stream);
    if (e == cudaSuccess)
        ++*launches;
    return e;
}

cudaError_t launch_filter_verify(const FilterParams &P, int tdt, int sms, cudaStream_t stream, int *launches)
{
    *launches = 0;
    cudaError_t e = P.status ? cudaMemsetAsync(P.status, 0, sizeof(int32_t), stream) : cudaSuccess;
    if (e == cudaSuccess)
        e = tdt ? rows<RowBF16, true>(P, sms, stream) : rows<RowF32, true>(P, sms, stream);
    if (e != cudaSuccess)
        return e;
    ++*launches;
    const int C = 8;
    e = tdt ? launch_clusters(filter_decide<RowBF16>, P.B, C, 0, true, stream, P)
            : launch_clusters(filter_decide<RowF32>, P.B, C, 0, true, stream, P);
    if (e == cudaSuccess)
        ++*launches;
    return e;
}

}  // namespace sv
