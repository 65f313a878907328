// k_filter.cu -- rows of logits under temperature, top-k, top-p and min-p:
// drawing from them, and the verification rule between them.
//
// The rule is the library's (nextadmin.net lesson "Speculative Decoding", § Core
// algorithm; aiengineeringfromscratch.com Phase 10 lesson 25, § The exact rule)
// with q and p the filtered distributions; sv_filter.cuh states the filters and
// the arithmetic.
//
// A cluster of CTAs takes a row (filter_rows).  The row is read from HBM once,
// for its maximum; what else is read of it comes from L2, which holds the rows in
// flight (kept in shared memory, there was room for three CTAs to an SM, each
// waiting for the others of its cluster most of the time: 256 rows of 128256, 242
// us, where they took 717 us so).
//   - T = 0: the maximum's first index.
//   - top-k, k up to 128, and min-p: a threshold that what is kept reaches, for
//     top-k from the threads' own maxima (a histogram of one value per thread: at
//     least k logits reach the k-th of them); what reaches it, a few more tokens
//     than are kept, goes to lists, which the first CTA gathers, ranks, cuts and
//     draws from.
//   - larger k and top-p alone, rows of 8192 16-bit logits or more: how often each value occurs, in
//     counts of 32 bits; a value's weight is computed once.  Counts and weights
//     give the cut and every CTA's share of what is kept, and only the CTA on which
//     the uniform falls looks at its tokens once more.
//   - the same, other rows: a histogram of the weights, in bins of 1/64 octave of the
//     weight.  A bin holds the sum of 1 + q, the weights' ratios to the bin's own,
//     in fixed point: two additions of 32 bits per token, in any order.  The tokens
//     of the bin with the cut go to lists and are ranked; meanwhile each warp sums
//     up the weights of its segment above that bin, for the draw.
//   - bins of more than 256 tokens, as under equal logits: the cut by histograms of
//     (logit, index) in finer and finer parts, over the CTAs' lists.
// Exchanges: each warp writes its numbers to every CTA of the cluster, all read
// behind one cluster barrier, all come to the same answer.  A barrier of its own
// lies ahead of the first one: no CTA writes to one that has not begun.
//
// Measured (one GB300, calls back to back, captured): one row of 128256 bfloat16
// logits, top-k 20 and top-p 0.8: 10.3 us, of which the launch and the first pass
// are 4 us and each exchange 1 us; top-p 0.9 alone: 25 us (ten exchanges, and 64
// tokens to a thread).  256 such rows: 26 us (2.5 TB/s: two waves of CTAs, each a
// first pass and then a second one) and 104 us (the instructions of the count, 14 a token,
// and of the values' weights, and the exchanges, 42 % of the issue slots taken).
// 256 rows without filters: 71 us (a weight a token, 45 instructions).
//
// The verification (filter_decide) reads the rows' records, walks the positions
// of a sequence in one warp, and draws from (q_j - p_j)+ over the tokens that
// the target row keeps: from its list, or else over the vocabulary, where a
// cluster shares it.  256 sequences, K = 4, 128256, top-k 20 to 50: 190 us, of which
// it takes 20 us; 3.1 TB/s.
#include <algorithm>
#include <atomic>
#include <cooperative_groups.h>
#include <cstdint>
#include <cuda_runtime.h>
#include <type_traits>

#include "sv_cluster.cuh"
#include "sv_filter.cuh"
#include "sv_launch.h"

namespace sv {
namespace {

namespace cg = cooperative_groups;

constexpr int FT = 256, FW = FT / 32;   // threads and warps of a CTA
constexpr int MAX_C = 16;               // CTAs of a cluster
constexpr int COARSE = 256;             // bins of the threads' maxima, a thread each
constexpr float RANGE = 64.0f;          // what these span: weights to 2^-64 of the largest
constexpr int ST_INVALID = 1;
// Bytes of the rows in flight, at most.  Smaller clusters have fewer barriers for the same bytes, but the second
// pass has to find its row in L2: 2304 rows of 256 KB, 200 us a call with clusters of two (78 MB in flight), 250 us of
// four, 232 us of one (156 MB); 480 rows of 304 KB, 234 us of four, 249 us of two.
constexpr long long FLIGHT = 80 << 20;
// Tokens of a CTA's part, at most: so many 16-bit halves of a bin's sums make less than 2^32.
constexpr int PART = 65536;

__device__ const FilterTable kFilterTable = filter_table();

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
    static __device__ __forceinline__ uint4 load(const void *p) { return __ldg(static_cast<const uint4 *>(p)); }
    static __device__ __forceinline__ float get(const uint4 &v, int k)
    {
        return __uint_as_float(k == 0 ? v.x : k == 1 ? v.y : k == 2 ? v.z : v.w);
    }
    static __device__ __forceinline__ f2 two(const uint4 &v, int k) { return k ? pku(v.z, v.w) : pku(v.x, v.y); }
    static __device__ __forceinline__ float one(const void *p, size_t i) { return __ldg(static_cast<const float *>(p) + i); }
    static __device__ __forceinline__ uint4 pack(const float (&x)[N])
    {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
    // a running maximum (NaN if any is)
    typedef float Max;
    static __device__ __forceinline__ Max start() { return -F_INF; }
    static __device__ __forceinline__ Max larger(Max m, const uint4 &v) { return max_nan(m, largest(v)); }
    static __device__ __forceinline__ float value(Max m) { return m; }
    static __device__ __forceinline__ float largest(const uint4 &v)
    {
        return max_nan(max_nan(get(v, 0), get(v, 1)), max_nan(get(v, 2), get(v, 3)));
    }
};
struct RowBF16 {
    static constexpr int N = 8, ES = 2;
    static constexpr uint32_t NONE = 0xff80ff80u;
    static __device__ __forceinline__ uint4 load(const void *p) { return __ldg(static_cast<const uint4 *>(p)); }
    static __device__ __forceinline__ float get(const uint4 &v, int k)
    {
        const uint32_t w = k < 2 ? v.x : k < 4 ? v.y : k < 6 ? v.z : v.w;
        return __uint_as_float(k & 1 ? w & 0xffff0000u : w << 16);
    }
    static __device__ __forceinline__ f2 two(const uint4 &v, int k)   // the k-th pair
    {
        const uint32_t w = k == 0 ? v.x : k == 1 ? v.y : k == 2 ? v.z : v.w;
        return pku(w << 16, w & 0xffff0000u);
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
    typedef uint32_t Max;
    static __device__ __forceinline__ Max start() { return NONE; }
    static __device__ __forceinline__ Max larger(Max m, const uint4 &v) { return max2(max2(max2(m, v.x), max2(v.y, v.z)), v.w); }
    static __device__ __forceinline__ float value(Max m)
    {
        return max_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
    }
    static __device__ __forceinline__ float largest(const uint4 &v)
    {
        const uint32_t w = max2(max2(v.x, v.y), max2(v.z, v.w));
        return max_nan(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
};

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

// ------------------------------------------------------------------ lists
// 256 bins for a search, a thread each.
struct Search {
    uint32_t lo[FT], hi[FT];   // a bin's sum in two words
    u64 sums[FW], base;
    int bin;
    __device__ __forceinline__ void add(int b, u64 w)
    {
        const uint32_t l = (uint32_t)w;
        const uint32_t h = (uint32_t)(w >> 32) + (atomicAdd(&lo[b], l) > ~l);
        if (h)
            atomicAdd(&hi[b], h);
    }
    // `v`: this thread's bin.  The bin at which the running sum from `ahead` on reaches `target` (which it does;
    // -1 where there is nothing); `ahead` becomes what lies ahead of it.  No barrier ahead of the return.
    __device__ __forceinline__ int find(u64 v, u64 &ahead, u64 target)
    {
        u64 all;
        const u64 at = ahead + block_scan64(v, sums, all);
        target = min(target, ahead + all);   // roundings may leave it behind the last
        if (threadIdx.x == 0)
            bin = -1;
        __syncthreads();
        if (at < target && at + v >= target) {
            bin = (int)threadIdx.x;
            base = at;
        }
        __syncthreads();
        if (bin >= 0)
            ahead = base;
        return bin;
    }
};
// How the keys in [from, to] are cut into 256 parts, largest first; the b-th part.
__device__ __forceinline__ int part_shift(u64 from, u64 to) { return max(0, 56 - __clzll((long long)(to - from))); }
__device__ __forceinline__ void part(int b, int shift, u64 &from, u64 &to)
{
    to -= (u64)b << shift;
    const u64 len = (1ull << shift) - 1;
    from = to - from <= len ? from : to - len;
}
// Sorts n <= FT keys, all different, largest first: each thread counts the keys ahead of its own.
__device__ __forceinline__ void rank_keys(u64 *key, int n)
{
    __syncthreads();
    const u64 mine = (int)threadIdx.x < n ? key[threadIdx.x] : 0;
    int at = 0;
    if ((int)(threadIdx.x & ~31u) < n)
        for (int i = 0; i < n; ++i)
            at += key[i] > mine;
    __syncthreads();
    if ((int)threadIdx.x < n)
        key[at] = mine;
    __syncthreads();
}
// Of n <= FT entries with tokens (the low words of the keys, inverted) and weights, in any order: the first, in
// ascending order of the token, at which the running sum exceeds `at`.  hit(entry, token) is called by one thread.
template <class F>
__device__ __forceinline__ void pick(const u64 *key, const u64 *w, int n, u64 at, F hit)
{
    if ((int)(threadIdx.x & ~31u) >= n)
        return;
    const int i = min((int)threadIdx.x, n - 1);
    const uint32_t mine = (uint32_t)key[i];
    u64 before = 0;
    for (int j = 0; j < n; ++j)
        before += (uint32_t)key[j] > mine ? w[j] : 0;
    if ((int)threadIdx.x < n && before <= at && before + w[i] > at)
        hit(i, (int)(0xffffffffu - mine));
}

constexpr int OCTAVES = 43;               // down to half a unit
constexpr int FINE = OCTAVES * 64 + 64;   // bins of the weights' histogram
constexpr int LISTS = 8;                  // lists of a row, at most
constexpr int RANKED = FT;                // tokens of a bin that are ranked; more are sorted into finer bins first
constexpr int STAGED = 2048;              // tokens in a CTA's own list
// 16 bits: tokens from which a row's values are counted (378 rows of 1570, most under top-p: 50 us by the histogram of
// weights, 57 us by values; 375 of 10826 52 us by values)
constexpr int MANY = 8192;
constexpr int KEYS = 2048;                // 16 bits: the values of 16 octaves, of either sign
constexpr int ODD = 1024;                 // logits closer to 0 in a CTA's part
// Top-k by a list: a quarter of an octave more may reach the threshold than are kept.  256 rows of 128256: top-k 20
// with top-p by lists 26 us, k = 1000 with top-p by lists of 1200 tokens 143 us, by the rows' values 103 us.
constexpr int FEW = FILTER_CAP / 2;
struct RowShared {
    u64 board[2][4][MAX_C * FW];   // published, by round parity: up to four numbers of every warp of the cluster
    u64 seg[2][FW];                // of this CTA's warps
    u64 sums[FW];
    Search search;
    float2 table[64];
    float top[FT];        // the threads' maxima
    uint32_t coarse[COARSE];
    uint32_t n[2 * LISTS];   // lengths of lists, and of a CTA's own
    float seg_cut;           // where the segment is cut that the uniform falls on
    uint32_t seg_last;
    u64 cut, base;
    double least;         // T ln(min_p)
    float c_hi, c_lo;
    int lo, hi;
    union {
        struct {
            uint32_t lo[FINE], hi[FINE];   // counts, or sums in two words
        } h;
        struct {
            uint32_t n[2 * KEYS + 2];      // how often each value occurs
            u64 odd[ODD];
        } v;
        u64 weight[2 * KEYS + 2];          // of the values
        struct {
            u64 key[FT], w[STAGED];        // the cluster's list, (logit, ~token) keys; this CTA's own, and weights
        } l;
    };
};
constexpr size_t ROW_SMEM = sizeof(RowShared);
static_assert(ROW_SMEM <= 48 << 10, "more has to be asked for");

// ------------------------------------------------------------------ one row
__device__ __forceinline__ void cl_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cl_wait_all() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// A row in vectors of 16 bytes, cut into a segment per warp of the cluster.
template <class T>
struct RowView {
    cg::cluster_group cl;
    const uint8_t *base;    // a 16-byte boundary at or ahead of the row
    int C, rank, lane, warp;
    int seg0, seg1, len;    // vectors: of this warp's segment, of any
    int off, V, nv;         // tokens ahead of the row in its first vector; of the row; its vectors
    bool ragged;

    __device__ __forceinline__ RowView(const uint8_t *row, int vocab)
        : cl(cg::this_cluster()), C((int)cl_size()), rank((int)cl_rank()), lane(threadIdx.x & 31),
          warp(threadIdx.x >> 5), V(vocab)
    {
        off = (int)((reinterpret_cast<uintptr_t>(row) & 15) / T::ES);
        base = row - off * T::ES;
        nv = (off + V + T::N - 1) / T::N;
        ragged = off != 0 || (off + V) % T::N != 0;
        len = ((nv + C * FW - 1) / (C * FW) + 31) & ~31;
        seg0 = min(segment() * len, nv);
        seg1 = min(seg0 + len, nv);
    }
    __device__ __forceinline__ int segment() const { return rank * FW + warp; }
    __device__ __forceinline__ int token(int v, int k) const { return v * T::N + k - off; }
    // Vector v; what is not the row's is minus infinity.
    __device__ __forceinline__ uint4 vector(int v) const
    {
        if (ragged && (v == 0 || v == nv - 1)) {
            float x[T::N];
#pragma unroll
            for (int k = 0; k < T::N; ++k) {
                const int i = token(v, k);
                x[k] = i >= 0 && i < V ? T::one(base, (size_t)(i + off)) : -F_INF;
            }
            return T::pack(x);
        }
        return T::load(base + (size_t)v * 16);
    }
    // f(vector, its number) for every vector of this warp's segment that is this lane's, U loads in flight: for short
    // f, with nothing to be asked of a vector but in the last round
    template <int U, class F>
    __device__ __forceinline__ void vectors(F f) const
    {
        int v = seg0 + lane;
        const int full = seg1 - (ragged && seg1 == nv);   // vectors that lie in the row
        if (ragged && seg0 == 0 && seg1 > 0) {            // the row's first one
            if (lane == 0) {
                f(vector(0), 0);
                v += 32;
            }
            __syncwarp();
        }
        const uint8_t *at = base + (size_t)v * 16;
#pragma unroll 1
        for (; v + 32 * (U - 1) < full; v += 32 * U, at += 512 * U) {
            uint4 q[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                q[u] = T::load(at + 512 * u);
#pragma unroll
            for (int u = 0; u < U; ++u)
                f(q[u], v + 32 * u);
        }
        if (v < seg1) {
            uint4 q[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (v + 32 * u < seg1)
                    q[u] = vector(v + 32 * u);
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (v + 32 * u < seg1)
                    f(q[u], v + 32 * u);
        }
    }
    // The same for this warp's segment, one vector at a time, the next one on its way: for longer f, which would
    // fill the instruction cache several times over
    template <class F>
    __device__ __forceinline__ void in_turn(F f) const
    {
        int v = seg0 + lane;
        uint4 next = make_uint4(0, 0, 0, 0);
        if (v < seg1)
            next = vector(v);
#pragma unroll 1
        for (; v < seg1; v += 32) {
            const uint4 q = next;
            if (v + 32 < seg1)
                next = vector(v + 32);
            f(q, v);
        }
    }
};

template <class T>
struct Row : RowView<T> {
    static constexpr bool SHORT = T::ES == 2;
    using RowView<T>::cl;
    using RowView<T>::C;
    using RowView<T>::rank;
    using RowView<T>::lane;
    using RowView<T>::warp;
    using RowView<T>::len;
    using RowView<T>::off;
    using RowView<T>::segment;
    using RowView<T>::token;
    using RowView<T>::in_turn;
    using RowView<T>::seg0;
    using RowView<T>::seg1;
    RowShared &S;
    uint32_t round = 0, lists = 0;
    __device__ __forceinline__ Row(RowShared &s, const uint8_t *row, int vocab) : RowView<T>(row, vocab), S(s) {}
    // f(logit, token) for the tokens of this warp's segment with logits of at least `from` and above minus infinity
    template <class F>
    __device__ __forceinline__ void each(float from, F f) const
    {
        in_turn([&](const uint4 &q, int v) {
            if (!(T::largest(q) >= from))
                return;
#pragma unroll
            for (int k = 0; k < T::N; ++k) {
                const float x = T::get(q, k);
                if (x >= from && x > -F_INF)
                    f(x, token(v, k));
            }
        });
    }
    // f(x0, x1, i, j, q, token): pairs of logits of this warp's segment, their split weights, and the first one's
    // token, from vectors with a logit of at least `from`
    template <class F>
    __device__ __forceinline__ void weights(const FilterWeight &W, float from, F f) const
    {
        in_turn([&](const uint4 &q, int v) {
            if (!(T::largest(q) >= from))
                return;
#pragma unroll
            for (int k = 0; k < T::N / 2; ++k) {
                const f2 x = T::two(q, k);
                float x0, x1;
                upk(x, x0, x1);
                uint32_t i, j;
                const f2 y = W.template split<SHORT>(x, i, j);
                f(x0, x1, i, j, y, token(v, 2 * k));
            }
        });
    }
    // Publishes n numbers per warp (the same in every lane): each warp writes its own to every CTA of the cluster, so
    // that they are at hand behind the barrier (read from their owners instead, each exchange took 1000 clocks more).
    struct Board {
        const u64 *at;
        __device__ __forceinline__ u64 get(int i, int segment) const { return at[i * MAX_C * FW + segment]; }
    };
    template <int N>
    __device__ __forceinline__ Board publish(const u64 (&x)[N])
    {
        u64 *at = &S.board[round & 1][0][0];
        ++round;
        if (lane < C) {
            u64 *to = cl.map_shared_rank(at + segment(), lane);
#pragma unroll
            for (int i = 0; i < N; ++i)
                to[i * MAX_C * FW] = x[i];
        }
        cl_sync();
        return Board{at};
    }
    // A number per warp: their sum ahead of this warp's (or of the first `end`), and in all
    __device__ __forceinline__ u64 ahead(const Board &b, int i, u64 &total) const { return ahead(b, i, total, segment()); }
    __device__ __forceinline__ u64 ahead(const Board &b, int i, u64 &total, int end) const
    {
        u64 x[MAX_C * FW / 32], all = 0, mine = 0;
        read(b, i, x);
#pragma unroll
        for (int k = 0; k < MAX_C * FW / 32; ++k) {
            all += x[k];
            mine += lane + 32 * k < end ? x[k] : 0;
        }
        total = warp_sum64(all);
        return warp_sum64(mine);
    }
    // This lane's part of the numbers of all warps, 0 where there are no more
    __device__ __forceinline__ void read(const Board &b, int i, u64 (&x)[MAX_C * FW / 32]) const
    {
#pragma unroll
        for (int k = 0; k < MAX_C * FW / 32; ++k)
            x[k] = lane + 32 * k < C * FW ? b.get(i, lane + 32 * k) : 0;
    }
    __device__ __forceinline__ u64 sum(const Board &b, int i) const
    {
        u64 total;
        ahead(b, i, total);
        return total;
    }
    // f associative, 0 its neutral element
    template <class F>
    __device__ __forceinline__ u64 fold(const Board &b, int i, F f) const
    {
        u64 x[MAX_C * FW / 32];
        read(b, i, x);
        u64 y = x[0];
#pragma unroll
        for (int k = 1; k < MAX_C * FW / 32; ++k)
            y = f(y, x[k]);
#pragma unroll
        for (int o = 16; o; o >>= 1)
            y = f(y, (u64)__shfl_xor_sync(0xffffffffu, y, o));
        return y;
    }
    __device__ __forceinline__ u64 most(const Board &b, int i) const
    {
        return fold(b, i, [](u64 a, u64 c) { return a > c ? a : c; });
    }
    // f(what lies at `p` in the shared memory of a CTA) for every CTA of the cluster, eight loads in flight, and none
    // for CTAs that a smaller cluster does not have
    template <class V_, class F>
    __device__ __forceinline__ void each_cta(V_ *p, F f) const
    {
        auto some = [&](int r, auto n) {
            V_ x[decltype(n)::value];
#pragma unroll
            for (int k = 0; k < decltype(n)::value; ++k)
                x[k] = *cl.map_shared_rank(p, r + k);
#pragma unroll
            for (int k = 0; k < decltype(n)::value; ++k)
                f(x[k]);
        };
        if (C == 1)
            f(*p);
        else if (C == 2)
            some(0, std::integral_constant<int, 2>{});
        else if (C == 4)
            some(0, std::integral_constant<int, 4>{});
        else
            for (int r = 0; r < C; r += 8)   // C is a power of two
                some(r, std::integral_constant<int, 8>{});
    }
    __device__ __forceinline__ u64 of_all(uint32_t *p) const   // their sum
    {
        u64 v = 0;
        each_cta(p, [&](uint32_t x) { v += x; });
        return v;
    }

    static __device__ __forceinline__ u64 key_of(float x, int token)
    {
        return (u64)filter_key(x) << 32 | (0xffffffffu - (uint32_t)token);
    }
    static __device__ __forceinline__ float value_of(u64 key) { return filter_value((uint32_t)(key >> 32)); }
    static __device__ __forceinline__ int token_of(u64 key) { return (int)(0xffffffffu - (uint32_t)key); }

    // The tokens with logits of at least `from` for which keep(x, token) holds go to this CTA's list, in any order.
    // Returns how many there are; where these are more than the list holds, they are not all in it.
    template <class F>
    __device__ __forceinline__ int stage(float from, F keep)
    {
        uint32_t *const n = &S.n[LISTS + lists];
        this->template vectors<4>([&](const uint4 &q, int v) {
            if (!(T::largest(q) >= from))
                return;
            uint32_t has = 0;
#pragma unroll
            for (int k = 0; k < T::N; ++k) {
                const float x = T::get(q, k);
                has |= (x >= from && x > -F_INF && keep(x, token(v, k)) ? 1u : 0u) << k;
            }
            if (!has)
                return;
            uint32_t at = atomicAdd(n, __popc(has));
#pragma unroll
            for (int k = 0; k < T::N; ++k)
                if (has >> k & 1) {
                    if (at < STAGED)
                        S.l.w[at] = key_of(T::get(q, k), token(v, k));
                    ++at;
                }
        });
        ++lists;
        __syncthreads();
        return (int)*n;
    }
    // Puts a key into this CTA's list of number `lists`, as `stage` does.
    __device__ __forceinline__ void put(float x, int token)
    {
        const uint32_t at = atomicAdd(&S.n[lists], 1u);
        if (at < STAGED)
            S.l.w[at] = key_of(x, token);
    }
    // All CTAs' lists, n_r keys in the r-th (number i of the board's, of warp 0), up to FT together, to this
    // CTA's S.l.key.
    __device__ __forceinline__ void gather(const Board &b, int i)
    {
        // where the CTAs' lists begin
        u64 n = lane < C ? b.get(i, lane * FW) : 0;
        const int end = (int)warp_scan64(n, lane), all = __shfl_sync(0xffffffffu, end, 31);
        const int begin = end - (int)n;
        const int k = threadIdx.x;
        int r = 0, at = k;
        for (int c = 1; c < C; ++c) {
            const int o = __shfl_sync(0xffffffffu, begin, c);
            if (k >= o)
                r = c, at = k - o;
        }
        if (k < all)
            S.l.key[k] = cl.map_shared_rank(S.l.w, r)[at];
        __syncthreads();
    }

    // Where the head ends that has `count` tokens (SUM = false), or ahead of whose last token less than `p` of
    // the whole lies, among the tokens with keys from `floor` on: the bin of 1/64 octave that holds its last token,
    // with what lies ahead of the bin, and the whole (`target`: of which that is to be reached).  -1: there are no
    // more tokens of any weight.
    template <bool SUM>
    __device__ __forceinline__ int bin_of_cut(const FilterWeight &W, float p, int count, u64 floor, u64 &ahead_, u64 &target)
    {
        __syncthreads();
        for (int i = threadIdx.x; i < FINE; i += FT) {
            S.h.lo[i] = 0;
            if (SUM)
                S.h.hi[i] = 0;
        }
        __syncthreads();
        const float x0 = floor ? fmaxf(value_of(floor), W.low) : W.low;
        auto stays = [&](float x, int token) { return x >= x0 && (x > x0 || key_of(x, token) >= floor); };
        constexpr uint32_t BASE = 0x48400000u;   // ROUND's bits
        if constexpr (SUM) {
            weights(W, x0, [&](float a, float b, uint32_t i, uint32_t j, f2 q, int token) {
                // (1 + q) 2^29, |q| < 0.0055
                float v, w;
                upk(fma2(q, pk(0x1p-4f, 0x1p-4f), pk(12582912.0f, 12582912.0f)), v, w);
                const uint32_t y = __float_as_uint(v) - 0x4b400000u + 0x20000000u;
                const uint32_t z = __float_as_uint(w) - 0x4b400000u + 0x20000000u;
                if (stays(a, token)) {
                    atomicAdd(&S.h.lo[BASE - i], y & 0xffffu);
                    atomicAdd(&S.h.hi[BASE - i], y >> 16);
                }
                if (stays(b, token + 1)) {
                    atomicAdd(&S.h.lo[BASE - j], z & 0xffffu);
                    atomicAdd(&S.h.hi[BASE - j], z >> 16);
                }
            });
        } else {
            each(x0, [&](float x, int token) {
                if (stays(x, token))
                    atomicAdd(&S.h.lo[-W.place(x)], 1u);
            });
        }
        __syncthreads();
        cl_sync();
        // this CTA's share of the bins, a thread's in a row
        const int per = (FINE + C * FT - 1) / (C * FT), first = (rank * FT + threadIdx.x) * per;
        auto of_bin = [&](int bin) -> u64 {
            if (bin >= FINE)
                return 0;
            const u64 v = of_all(&S.h.lo[bin]) + (SUM ? of_all(&S.h.hi[bin]) << 16 : 0);
            if (!SUM)
                return v;
            return W.of_bin(v, bin);
        };
        u64 s = 0;
        for (int e = 0; e < per; ++e)
            s += of_bin(first + e);
        const u64 in = warp_scan64(s, lane);
        const u64 x[1] = {__shfl_sync(0xffffffffu, in, 31)};
        u64 all;
        u64 at = ahead(publish(x), 0, all) + in - s;
        // less than p of the whole: the same as less than the next whole number
        target = SUM ? max(share_up(p, all), 1ull) : (u64)count;
        u64 found = 0, before = 0;
        if (at < target && at + s >= target)
            for (int e = 0; e < per && !found; ++e) {
                const u64 w = of_bin(first + e);
                if (at + w >= target)
                    found = (u64)(first + e) + 1, before = at;
                at += w;
            }
        const unsigned who = __ballot_sync(0xffffffffu, found != 0);
        const int from = who ? __ffs(who) - 1 : 0;
        const u64 y[2] = {__shfl_sync(0xffffffffu, found, from), __shfl_sync(0xffffffffu, before, from)};
        const auto board = publish(y);
        found = most(board, 0);
        ahead_ = most(board, 1);
        return (int)found - 1;
    }
    // A logit a little below those of the bin.
    static __device__ __forceinline__ float below_bin(const FilterWeight &W, int bin)
    {
        return W.m - ((float)bin + 0.51f) * (1.0f / 64.0f) / W.c_hi * 1.00001f - fabsf(W.m) * 0x1p-21f;
    }

    // The key of the head's last token, among those with keys in [from, to], `ahead_` lying ahead of them: these
    // are in the CTAs' lists, `n` in this one's, or (LIST = false) only in the row.
    template <bool SUM, bool LIST>
    __device__ __noinline__ u64 refine(const FilterWeight &W, int n, u64 from, u64 to, u64 ahead_, u64 target)
    {
        Search &Q = S.search;
#pragma unroll 1
        while (from < to) {
            const int shift = part_shift(from, to);
            __syncthreads();
            Q.lo[threadIdx.x] = Q.hi[threadIdx.x] = 0;
            __syncthreads();
            auto add = [&](u64 k) { Q.add((int)((to - k) >> shift), SUM ? W(value_of(k)) : 1); };
            if constexpr (LIST) {
                for (int i = threadIdx.x; i < n; i += FT)
                    if (S.l.w[i] >= from && S.l.w[i] <= to)
                        add(S.l.w[i]);
            } else {
                const float high = value_of(to);
                each(value_of(from), [&](float x, int token) {
                    const u64 k = x > high ? 0 : key_of(x, token);
                    if (k >= from && k <= to)
                        add(k);
                });
            }
            cl_sync();
            const int bin = Q.find(of_all(&Q.lo[threadIdx.x]) + (of_all(&Q.hi[threadIdx.x]) << 32), ahead_, target);
            cl_sync();     // all have read the bins
            if (bin < 0)
                break;     // nothing of any weight
            part(bin, shift, from, to);
        }
        return from;
    }

    // The key of the head's last token, which is in the bin (bin_of_cut).  By sums, where the bin has few tokens, the
    // segments' weights as well: the sum of those that stay (keys from the cut and from `c_min` on), what lies ahead
    // of this warp's segment, and its own.
    template <bool SUM>
    __device__ __forceinline__ u64 cut_in_bin(const FilterWeight &W, int bin, u64 floor, u64 ahead_, u64 target, u64 c_min,
                                              bool &done, u64 &Z, u64 &before, u64 &mine)
    {
        u64 above = 0;   // the bin
        u64 none = 0, most_ = 0;   // ~ the least and the largest key in it
        const float low = fmaxf(below_bin(W, bin), W.low);
        auto in_bin = [&](float x, int token) {
            const u64 k = key_of(x, token);
            if (k < floor)
                return;
            put(x, token);
            none = max(none, ~k);
            most_ = max(most_, k);
        };
        constexpr uint32_t BASE = 0x48400000u;   // ROUND's bits
        if constexpr (SUM) {
            weights(W, low, [&](float x0, float x1, uint32_t i, uint32_t j, f2 y, int token) {
                const int a = x0 >= low ? (int)(BASE - i) : FINE, b = x1 >= low ? (int)(BASE - j) : FINE;
                if (min(a, b) < bin) {
                    float q, r;
                    upk(y, q, r);
                    above += (a < bin ? W.units(i, q) : 0) + (b < bin ? W.units(j, r) : 0);
                }
                if (a == bin)
                    in_bin(x0, token);
                if (b == bin)
                    in_bin(x1, token + 1);
            });
        } else {
            each(low, [&](float x, int token) {
                if (-W.place(x) == bin)
                    in_bin(x, token);
            });
        }
        __syncthreads();
        const int n = (int)S.n[lists++];
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            none = max(none, (u64)__shfl_xor_sync(0xffffffffu, none, o));
            most_ = max(most_, (u64)__shfl_xor_sync(0xffffffffu, most_, o));
        }
        const u64 seg = SUM ? warp_sum64(above) : 0;
        const u64 told[4] = {warp == 0 ? (u64)n : 0, none, most_, seg};
        const Board board = publish(told);
        const int all = (int)sum(board, 0);
        if (all > RANKED) {
            const u64 from = ~most(board, 1), to = most(board, 2);
            return most(board, 0) <= STAGED ? refine<SUM, true>(W, n, from, to, ahead_, target)
                                            : refine<SUM, false>(W, n, from, to, ahead_, target);
        }
        // every CTA ranks all of them
        gather(board, 0);
        if constexpr (!SUM)
            cl_sync();   // the lists have been read: bins take their place
        if (all == 0)
            return floor;
        rank_keys(S.l.key, all);
        if constexpr (!SUM)
            return S.l.key[min((int)(target - ahead_), all) - 1];
        const u64 key = (int)threadIdx.x < all ? S.l.key[threadIdx.x] : 0;
        u64 w = key ? W(value_of(key)) : 0, sum_;
        const u64 at = ahead_ + block_scan64(w, S.sums, sum_);
        if (threadIdx.x == 0)
            S.cut = S.l.key[all - 1];   // where roundings leave the target behind the last
        __syncthreads();
        // the token whose weight reaches the target is the last
        if (at < target && at + w >= target)
            S.cut = key;
        __syncthreads();
        const u64 cut = max(S.cut, c_min);
        // what stays of the bin, by segment
        const int s = key >= cut && key ? ((token_of(key) + off) / T::N) / len : -1;
        w = s >= 0 ? w : 0;
        u64 total;
        before = ahead(board, 3, total);
        block_scan64(w, S.sums, sum_);
        Z = total + sum_;
        // ahead of this CTA's segments, and in them
        block_scan64(s < rank * FW ? w : 0, S.sums, sum_);
        before += sum_;
        mine = seg;
#pragma unroll 1
        for (int k = 0; k < FW; ++k) {
            block_scan64(s == rank * FW + k ? w : 0, S.sums, sum_);
            before += k < warp ? sum_ : 0;
            mine += k == warp ? sum_ : 0;
        }
        done = true;
        return cut;
    }

    // ---- logits of 16 bits take few values: how often each occurs says all that a cut needs, and a value's weight is
    // computed once, not once a token (128 rows of 262144 under top-p: 104 us, 147 us by the histogram of weights).
    // Values in their order, largest first: 16 octaves of positive ones, those
    // closer to 0 (one place for all, and a list: about 1 in 2^11 of a row's), 16 octaves of negative ones.
    struct Values {
        int base;   // of the 16 octaves' absolute bits
        __device__ __forceinline__ explicit Values(const FilterWeight &W)
        {
            base = (int)((__float_as_uint(fmaxf(fabsf(W.m), fabsf(W.low))) + 0xffffu) >> 16) - (KEYS - 1);
        }
        // of a logit at or above W.low
        __device__ __forceinline__ int place(float x) const
        {
            const uint32_t b = __float_as_uint(x + 0.0f);   // -0 is 0
            const int t = (int)((b >> 16) & 0x7fffu) - base + 1;   // 1 .. KEYS, or less
            return t <= 0 ? KEYS : (int)b < 0 ? KEYS + t : KEYS - t;
        }
        __device__ __forceinline__ float at(int place) const
        {
            const int t = place < KEYS ? KEYS - place : place - KEYS;
            const int a = max(t - 1 + base, 0);
            return __uint_as_float((uint32_t)(a << 16) | (place > KEYS ? 0x80000000u : 0u));
        }
    };
    // The cut by top-k (k <= 0: none), top-p (p >= 1: none) and min-p, and Z.  DRAW: in the CTA on which the uniform u
    // falls, what lies ahead of this warp's segment and in it (`mine`; 0 elsewhere), and where the cut lies in the
    // segment.  `owner`: this lane has the row's cut.  False: not found this way.
    template <bool DRAW>
    __device__ __forceinline__ bool by_values(const FilterWeight &W, int k, float p, float xmin, float u, u64 &Z, u64 &before,
                                              u64 &mine, float &cut_x, uint32_t &cut_last, bool &owner)
    {
        const Values values(W);
        constexpr int N = 2 * KEYS + 1;
        __syncthreads();
        for (int i = threadIdx.x; i < N; i += FT)
            S.v.n[i] = 0;
        uint32_t *const odd = &S.n[LISTS + lists++];
        __syncthreads();
        in_turn([&](const uint4 &q, int v) {
            if (!(T::largest(q) >= W.low))
                return;
#pragma unroll
            for (int e = 0; e < T::N; ++e) {
                const float x = T::get(q, e);
                if (!(x >= W.low))
                    continue;
                const int at = values.place(x);
                if (at != KEYS) {
                    atomicAdd(&S.v.n[at], 1u);
                } else {
                    const uint32_t i = atomicAdd(odd, 1u);
                    if (i < ODD)
                        S.v.odd[i] = key_of(x, token(v, e));
                }
            }
        });
        __syncthreads();
        const int nodd = (int)*odd;
        u64 w_odd = 0;
        for (int i = threadIdx.x; i < min(nodd, ODD); i += FT)
            w_odd += W(value_of(S.v.odd[i]));
        const u64 told[2] = {(u64)nodd, warp_sum64(w_odd)};
        const Board board = publish(told);
        if (most(board, 0) > ODD)
            return false;
        const u64 all_odd = sum(board, 0) / FW, sum_odd = sum(board, 1);
        // this CTA's share of the values, a thread's in a row: their numbers and weights
        const int per = (N + C * FT - 1) / (C * FT), first = (rank * FT + threadIdx.x) * per;
        auto value_at = [&](int i, u64 &n, u64 &w) {
            n = w = 0;
            if (i == KEYS) {
                n = all_odd;
                w = sum_odd;
            } else if (i < N) {
                n = of_all(&S.v.n[i]);
                w = n ? n * W(values.at(i)) : 0;
            }
        };
        u64 sn = 0, sw = 0;
        for (int e = 0; e < per; ++e) {
            u64 n, w;
            value_at(first + e, n, w);
            sn += n;
            sw += w;
        }
        const u64 in_n = warp_scan64(sn, lane), in_w = warp_scan64(sw, lane);
        const u64 ours[2] = {__shfl_sync(0xffffffffu, in_n, 31), __shfl_sync(0xffffffffu, in_w, 31)};
        const Board b2 = publish(ours);
        u64 total, total_n;
        const u64 at_n = ahead(b2, 0, total_n) + in_n - sn, at_w = ahead(b2, 1, total) + in_w - sw;
        // the value that holds the cut: found by one thread, told to all with what lies ahead of it
        auto find = [&](bool here, auto reached, u64 &n0, u64 &w0) {
            u64 found = 0, n_ahead = at_n, w_ahead = at_w;
            if (here)
                for (int e = 0; e < per && !found; ++e) {
                    u64 n, w;
                    value_at(first + e, n, w);
                    if (reached(n_ahead + n, w_ahead + w)) {
                        found = (u64)(first + e) + 1;
                    } else {
                        n_ahead += n;
                        w_ahead += w;
                    }
                }
            const unsigned who = __ballot_sync(0xffffffffu, found != 0);
            const int from = who ? __ffs(who) - 1 : 0;
            const u64 x[3] = {__shfl_sync(0xffffffffu, found, from), who ? (u64)__shfl_sync(0xffffffffu, n_ahead, from) : 0,
                              who ? (u64)__shfl_sync(0xffffffffu, w_ahead, from) : 0};
            const Board b = publish(x);
            found = most(b, 0);
            n0 = most(b, 1);
            w0 = most(b, 2);
            return (int)found - 1;
        };
        int place = -1;
        u64 ties = ~0ull, n0, w0;   // tokens of that value that stay
        if (k > 0 && (u64)k < total_n) {
            place = find(at_n < (u64)k && at_n + sn >= (u64)k, [&](u64 n, u64) { return n >= (u64)k; }, n0, w0);
            if (place == KEYS)
                return false;
            ties = (u64)k - n0;
            total = w0 + ties * W(values.at(place));
        }
        if (p < 1.0f) {
            // less than p of the whole: the same as less than the next whole number
            const u64 target = max(share_up(fmaxf(p, 0.0f), total), 1ull);
            place = find(at_w < target && at_w + sw >= target, [&](u64, u64 w) { return w >= target; }, n0, w0);
            if (place == KEYS)
                return false;
            const u64 w = W(values.at(place));
            ties = (target - w0 + w - 1) / w;
        }
        float x0 = place >= 0 ? values.at(place) : W.low;
        if (place < 0)
            ties = ~0ull;
        if (xmin > x0) {
            x0 = xmin;
            ties = ~0ull;
        }
        x0 = fmaxf(x0, W.low);
        // ---- each CTA's weights above x0, and how many of its tokens have x0, from its own numbers
        const u64 w0_ = W(x0);
        u64 m = 0, tied = 0;
        for (int i = threadIdx.x; i < N; i += FT) {
            const uint32_t n = S.v.n[i];
            const float x = values.at(i);
            if (n && x >= x0) {
                if (x > x0)
                    m += n * W(x);
                else
                    tied += n;
            }
        }
        for (int i = threadIdx.x; i < nodd; i += FT) {
            const float x = value_of(S.v.odd[i]);
            if (x > x0)
                m += W(x);
            tied += x == x0;
        }
        const u64 parts[2] = {warp_sum64(m), warp_sum64(tied)};
        const Board b3 = publish(parts);
        u64 all, all_tied;
        const u64 m_ahead = ahead(b3, 0, all, rank * FW), tied_ahead = ahead(b3, 1, all_tied, rank * FW);
        const u64 m_to = ahead(b3, 0, all, rank * FW + FW), tied_to = ahead(b3, 1, all_tied, rank * FW + FW);
        ties = min(ties, all_tied);
        Z = all + ties * w0_;
        cut_x = x0;
        cut_last = 0xffffffffu;
        owner = rank == 0 && threadIdx.x == 0 && ties == all_tied;
        before = m_ahead + min(tied_ahead, ties) * w0_;
        mine = 0;
        const bool splits = ties < all_tied && tied_ahead < ties && ties <= tied_to;   // the last tie that stays is here
        const bool drawn = DRAW && before <= share_down(u, Z) && share_down(u, Z) < m_to + min(tied_to, ties) * w0_;
        if (!splits && !drawn)
            return true;
        // ---- the same for each warp's segment of this CTA: by a pass over its part, the values' weights at hand.  They
        // are the numbers that the CTA's share is made of, so the segments end where it ends: a uniform on this CTA
        // falls on one of its segments, and on no other CTA's.
        const int top = values.place(W.highest()), end = values.place(x0);
        __syncthreads();
        if (DRAW)
            for (int i = top + threadIdx.x; i <= end; i += FT)
                if (i != KEYS)
                    S.weight[i] = W(values.at(i));
        __syncthreads();
        u64 above = 0;
        tied = 0;
        in_turn([&](const uint4 &q, int) {
            if (!(T::largest(q) >= x0))
                return;
#pragma unroll
            for (int e = 0; e < T::N; ++e) {
                const float x = T::get(q, e);
                if (DRAW && x > x0) {
                    const int at = values.place(x);
                    above += at != KEYS ? S.weight[at] : W(x);
                }
                tied += x == x0;
            }
        });
        tied = warp_sum64(tied);
        const u64 seg = DRAW ? warp_sum64(above) : 0;
        if (lane == 0) {
            S.seg[0][warp] = seg;
            S.seg[1][warp] = tied;
        }
        __syncthreads();
        u64 t_ahead = tied_ahead;
        before = m_ahead;
        for (int k = 0; k < warp; ++k) {
            before += S.seg[0][k];
            t_ahead += S.seg[1][k];
        }
        const u64 here = t_ahead >= ties ? 0 : min(ties - t_ahead, tied);   // of this segment's
        before += min(t_ahead, ties) * w0_;
        mine = seg + here * w0_;
        if (here == 0 && ties < all_tied) {
            cut_x = __int_as_float(__float_as_int(x0 + 0.0f) + (x0 >= 0.0f ? 1 : -1));   // nothing at x0 stays
        } else if (t_ahead + here == ties && ties < all_tied) {
            // the token of the last one that stays
            u64 seen = 0;
            for (int v = seg0; v < seg1; v += 32) {
                const uint4 q = v + lane < seg1 ? this->vector(v + lane) : make_uint4(T::NONE, T::NONE, T::NONE, T::NONE);
                int n = 0;
#pragma unroll
                for (int e = 0; e < T::N; ++e)
                    n += T::get(q, e) == x0;
                u64 upto = seen + warp_scan64((u64)n, lane);
                const unsigned who = __ballot_sync(0xffffffffu, upto >= here);
                if (who == 0) {
                    seen = __shfl_sync(0xffffffffu, upto, 31);
                    continue;
                }
                const int l = __ffs(who) - 1;
                int t = -1;
                upto -= n;
#pragma unroll
                for (int e = 0; e < T::N; ++e)
                    if (T::get(q, e) == x0 && ++upto == here)
                        t = token(v + lane, e);
                cut_last = (uint32_t)__shfl_sync(0xffffffffu, t, l);
                break;
            }
            owner = lane == 0;
        }
        return true;
    }

    // The sum of the weights from `cut` on, of this warp's segment.
    __device__ __forceinline__ u64 mass(const FilterWeight &W, u64 cut) const
    {
        const float x0 = cut ? fmaxf(value_of(cut), W.low) : W.low;
        u64 s = 0;
        weights(W, x0, [&](float a, float b, uint32_t i, uint32_t j, f2 y, int token) {
            float q, r;
            upk(y, q, r);
            // both, needed or not: weights that are chosen ahead of the sum took 81 us for 256 rows of 128256, 71 us so
            const u64 wa = W.units(i, q), wb = W.units(j, r);
            if (a > x0 || (a == x0 && key_of(a, token) >= cut))
                s += wa;
            if (b > x0 || (b == x0 && key_of(b, token + 1) >= cut))
                s += wb;
        });
        return warp_sum64(s);
    }
};

template <class T, bool VERIFY>
__global__ void __launch_bounds__(FT, 4) filter_rows(const __grid_constant__ FilterParams P)
{
    extern __shared__ __align__(128) uint8_t smem[];
    RowShared &S = *reinterpret_cast<RowShared *>(smem);
    using R_ = Row<T>;
    // waited for ahead of the first exchange: the other CTAs' shared memory is there once they run.  Nothing written is
    // told by it (256 x K = 4: 190 us; with release 194 us; without the barrier 189 us)
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    const int row = (int)cl_id(), V = P.V, tid = threadIdx.x;
    const int per = VERIFY ? 2 * P.K + 1 : P.K;
    const int b = row / per, i = row - b * per;
    const bool draft = VERIFY && i > P.K;
    const FilterSet &F = draft ? P.df : P.f;
    const uint8_t *src = static_cast<const uint8_t *>(draft ? P.draft : P.logits) +
                         (size_t)(VERIFY ? draft ? b * P.K + i - P.K - 1 : b * (P.K + 1) + i : row) * V * T::ES;
    R_ R(S, src, V);
    const int rank = R.rank;
    if (VERIFY)
        pdl_trigger();   // the kernel behind waits for this one's results itself

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
    else if (tid < 64 + 2 * LISTS)
        S.n[tid - 64] = 0;
    S.coarse[tid] = 0;
    if (tid == FT - 32) {
        // temperatures beyond 2^-100 and 2^100 count as these
        const double t = fmin(fmax((double)temp, 0x1p-100), 0x1p100), c = 1.4426950408889634 / t;
        S.c_hi = temp > 0.0f ? (float)c : 0.0f;
        S.c_lo = temp > 0.0f ? (float)(c - (double)S.c_hi) : 0.0f;
        S.least = least > 0.0f ? t * log((double)least) : 0.0;
    }
    typename T::Max most = T::start();
    R.template vectors<8>([&](const uint4 &q, int) { most = T::larger(most, q); });
    float m = T::value(most);
    S.top[tid] = m;
#pragma unroll
    for (int o = 16; o; o >>= 1)
        m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    {
        __syncthreads();
        cl_wait_all();
        const u64 x[1] = {1ull << 32 | __float_as_uint(m)};
        m = __uint_as_float((uint32_t)R.fold(R.publish(x), 0, [](u64 a, u64 c) {
            return a == 0 || c == 0 ? a | c
                                    : 1ull << 32 | __float_as_uint(max_nan(__uint_as_float((uint32_t)a), __uint_as_float((uint32_t)c)));
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
        u64 first = 0;   // ~token
        R.each(m, [&](float, int token) { first = max(first, (u64)(0xffffffffu - (uint32_t)token)); });
#pragma unroll
        for (int o = 16; o; o >>= 1)
            first = max(first, (u64)__shfl_xor_sync(0xffffffffu, first, o));
        const u64 x[1] = {first};
        first = 0xffffffffu - (uint32_t)R.most(R.publish(x), 0);
        rec.cut = m;
        rec.last = (uint32_t)first;
        rec.Z = 1ull << 43;
        if (rank == 0 && tid == 0) {
            if (VERIFY && !draft) {
                const size_t list = (size_t)(b * (P.K + 1) + i) * FILTER_CAP;
                P.list_x[list] = (int32_t)first;
                P.list_w[list] = rec.Z;
                rec.n = 1;
            }
            finish((int)first, 1.0f);
        }
        cl_sync();
        return;
    }

    const float xmin = least > 0.0f ? __double2float_ru((double)m + S.least) : -F_INF;
    // ---- a threshold that what is kept reaches, for lists
    const bool few = k <= FEW;
    bool listed = V <= FILTER_CAP;
    float t0 = p < 1.0f ? -F_INF : xmin;   // top-p's total counts what min-p drops
    if (!listed && few) {
        if (tid == 0)
            S.lo = COARSE - 1;
        __syncthreads();
        R.each_cta(&S.top[tid], [&](float x) {
            if (x > -F_INF)
                atomicAdd(&S.coarse[min(COARSE - 1, (int)((m - x) * (W.c_hi * (COARSE / RANGE))))], 1u);
        });
        __syncthreads();
        const u64 n = S.coarse[tid];
        u64 all;
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
        const int own = R.stage(t0, [](float, int) { return true; });
        const u64 x[1] = {R.warp == 0 ? (u64)own : 0};
        const auto board = R.publish(x);
        const int count = (int)R.sum(board, 0);
        if (count <= FILTER_CAP) {
            if (rank == 0)
                R.gather(board, 0);
            cl_arrive();
            if (rank != 0) {
                cl_wait_all();   // their lists have been read
                return;
            }
            u64 Z, all;
            // ranked, a token per thread
            rank_keys(S.l.key, count);
            const u64 key = tid < count ? S.l.key[tid] : 0;
            u64 w = tid < count && tid < k ? W(R_::value_of(key)) : 0;
            const u64 at = block_scan64(w, S.sums, all);
            const bool stays = tid < count && (tid == 0 || (tid < k && (p >= 1.0f || at < max(share_up(fmaxf(p, 0.0f), all), 1ull)) && R_::value_of(key) >= xmin));
            w = stays ? w : 0;
            S.l.w[tid] = w;
            block_scan64(w, S.sums, Z);
            block_scan64(stays, S.search.sums, all);
            const int n = (int)all;
            const u64 last = S.l.key[n - 1];
            if (VERIFY) {
                if (!draft && tid < n) {
                    const size_t list = (size_t)(b * (P.K + 1) + i) * FILTER_CAP;
                    P.list_x[list + tid] = R_::token_of(key);
                    P.list_w[list + tid] = w;
                }
                rec.n = draft ? -1 : n;
                rec.cut = R_::value_of(last);
                rec.last = (uint32_t)R_::token_of(last);
                rec.Z = Z;
                if (tid == 0)
                    finish(-1, 0.0f);
            } else {
                pick(S.l.key, S.l.w, n, share_down(u, Z), [&](int e, int token) {
                    finish(token, (float)((double)S.l.w[e] / (double)Z));
                });
            }
            __syncthreads();
            cl_wait_all();
            return;
        }
    }

    // ---- the cut by histograms over the row
    u64 cut = 0, mine = 0, ahead, target, Z = 0, before = 0;
    bool done = false;   // Z and `before`, the weights ahead of this warp's segment, are known
    bool owner = rank == 0 && tid == 0;   // writes the record
    if (R_::SHORT && V >= MANY && (k < V || p < 1.0f))
        done = R.template by_values<!VERIFY>(W, k < V ? k : 0, p, xmin, u, Z, before, mine, rec.cut, rec.last, owner);
    const bool valued = done;
    if (!done && k < V) {
        const int bin = R.template bin_of_cut<false>(W, 0.0f, k, 0, ahead, target);
        if (bin >= 0)
            cut = R.template cut_in_bin<false>(W, bin, 0, ahead, target, 0, done, Z, before, mine);
    }
    const u64 c_min = least > 0.0f ? (u64)filter_key(xmin) << 32 : 0;
    if (!done && p < 1.0f) {
        const int bin = R.template bin_of_cut<true>(W, fmaxf(p, 0.0f), 0, cut, ahead, target);
        if (!(least > 0.0f && (xmin >= W.low ? -W.place(xmin) : FINE) < bin))   // else min-p cuts ahead of that bin
            cut = R.template cut_in_bin<true>(W, bin, cut, ahead, target, c_min, done, Z, before, mine);
    }
    cut = c_min > cut ? c_min : cut;
    if (!done) {
        mine = R.mass(W, cut);
        const u64 x[1] = {mine};
        before = R.ahead(R.publish(x), 0, Z);
    }
    cl_arrive();   // nothing of another CTA is read from here on
    if (!valued) {
        rec.cut = cut ? R_::value_of(cut) : -F_INF;
        rec.last = (uint32_t)R_::token_of(cut);
    }
    rec.Z = Z;
    if (VERIFY) {
        if (owner)
            finish(-1, 0.0f);
    } else {
        // the segment on which the uniform falls, then the vector, by its whole CTA
        const u64 v = share_down(u, Z);
        if (tid == 0)
            S.hi = 0;
        __syncthreads();
        if (R.lane == 0 && before <= v && before + mine > v) {
            S.hi = 1;
            S.lo = R.warp;
            S.base = before;
            S.seg_cut = rec.cut;   // as that segment has it
            S.seg_last = rec.last;
        }
        __syncthreads();
        if (S.hi) {
            rec.cut = S.seg_cut;
            rec.last = S.seg_last;
            const int a0 = min((rank * FW + S.lo) * R.len, R.nv), a1 = min(a0 + R.len, R.nv);
            const u64 base = S.base;
            // the segment's tokens have the weights that it was weighed by, so the uniform falls on one of them
            const u64 to = v - base;
            u64 at = 0, all;
#pragma unroll 1
            for (int a = a0; a < a1 && at <= to; a += FT) {
                u64 w[T::N], s = 0;
                const uint4 q = a + tid < a1 ? R.vector(a + tid) : make_uint4(T::NONE, T::NONE, T::NONE, T::NONE);
#pragma unroll
                for (int e = 0; e < T::N; ++e) {
                    const float y = T::get(q, e);
                    const bool in = y > rec.cut || (y == rec.cut && (uint32_t)R.token(a + tid, e) <= rec.last);
                    w[e] = in ? W(y) : 0;
                    s += w[e];
                }
                u64 upto = at + block_scan64(s, S.sums, all);
                at += all;
                if (upto <= to && upto + s > to) {
#pragma unroll
                    for (int e = 0; e < T::N; ++e) {
                        if (w[e] && upto <= to && upto + w[e] > to)
                            finish(R.token(a + tid, e), (float)((double)w[e] / (double)Z));
                        upto += w[e];
                    }
                }
            }
        }
    }
    __syncthreads();
    cl_wait_all();
}

// ------------------------------------------------------------------ the rule
struct DecideShared {
    u64 slot[2][FW];
    u64 sums[FW];
    float2 table[64];
    int j, code, seg;
    u64 before;
    FilterShare sq, sp;
    u64 key[FILTER_CAP], w[FILTER_CAP];
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
    if (tid == 0)
        S.sq = FilterShare(q.Z);
    else if (tid == 32 && !bonus)
        S.sp = FilterShare(p.Z);
    __syncthreads();
    const FilterShare share_q = S.sq, share_p = S.sp;
    const float v = __ldg(P.uniforms + ((size_t)b * (K + 1) + j) * 2 + 1);
    const size_t row_q = (size_t)j * V;
    // (q - p)+ in units of 2^-62; nothing for equal ones
    auto left = [&](u64 wq, u64 wp) -> u64 {
        const u64 x = share_q(wq), y = share_p(wp);
        return x > y ? x - y : 0;
    };
    int32_t *out = P.out_tokens + (size_t)b * (K + 1) + j;
    if (q.n >= 0) {
        if (rank != 0)
            return;
        const size_t list = ((size_t)b * (K + 1) + j) * FILTER_CAP;
        u64 w = 0, all;
        if (tid < q.n) {
            const int x = P.list_x[list + tid];
            w = P.list_w[list + tid];
            S.key[tid] = 0xffffffffu - (uint32_t)x;
            S.w[tid] = w;
            if (!bonus)
                w = left(w, weight(p, Wp, T::one(drf, row_q + x), x));
        }
        block_scan64(w, S.sums, all);
        // where nothing is left of the target beside the draft, from the target itself
        if (all == 0)
            all = q.Z;
        else if (tid < q.n)
            S.w[tid] = w;
        __syncthreads();
        pick(S.key, S.w, q.n, share_down(v, all), [&](int, int token) { *out = token; });
        return;
    }
    // over the vocabulary: a segment per warp, then the segment on which the uniform falls
    const RowView<T> R(tgt + row_q * T::ES, V);
    const int me = R.segment();
    auto rest = [&](float x, int token, u64 &wq) -> u64 {
        wq = weight(q, Wq, x, token);
        return bonus || wq == 0 ? wq : left(wq, weight(p, Wp, T::one(drf, row_q + token), token));
    };
    u64 s = 0, sq = 0;
    R.in_turn([&](const uint4 &y, int at) {
        if (!(T::largest(y) >= q.cut))
            return;
#pragma unroll
        for (int k = 0; k < T::N; ++k) {
            const float x = T::get(y, k);
            if (x >= q.cut && x > -F_INF) {
                u64 wq;
                s += rest(x, R.token(at, k), wq);
                sq += wq;
            }
        }
    });
    s = warp_sum64(s);
    sq = warp_sum64(sq);
    if (lane == 0) {
        S.slot[0][warp] = s;
        S.slot[1][warp] = sq;
    }
    if (tid == 0)
        S.seg = -1;
    cl_sync();
    u64 all = 0, all_q = 0, before = 0, before_q = 0;
    for (int g = lane; g < C * FW; g += 32) {
        const u64 a = *cl.map_shared_rank(&S.slot[0][g % FW], g / FW), c = *cl.map_shared_rank(&S.slot[1][g % FW], g / FW);
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
    const u64 at = share_down(v, all);
    if (lane == 0 && before <= at && before + s > at) {
        S.seg = warp;
        S.before = before;
    }
    __syncthreads();
    if (S.seg >= 0) {
        // the same weights as above, so the uniform falls on one of them
        const int a0 = min((rank * FW + S.seg) * R.len, R.nv), a1 = min(a0 + R.len, R.nv);
        u64 upto = S.before;
        for (int a = a0; a < a1; a += FT) {
            u64 r[T::N], sum, mine = 0;
            const uint4 y = a + tid < a1 ? R.vector(a + tid) : make_uint4(T::NONE, T::NONE, T::NONE, T::NONE);
#pragma unroll
            for (int k = 0; k < T::N; ++k) {
                const float x = T::get(y, k);
                r[k] = 0;
                if (x >= q.cut && x > -F_INF) {
                    u64 wq;
                    r[k] = rest(x, R.token(a + tid, k), wq);
                    r[k] = whole ? wq : r[k];
                }
                mine += r[k];
            }
            u64 to = upto + block_scan64(mine, S.sums, sum);
#pragma unroll
            for (int k = 0; k < T::N; ++k) {
                if (r[k] && to <= at && to + r[k] > at)
                    *out = R.token(a + tid, k);
                to += r[k];
            }
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
    // of a cluster of C, where the row begins at the last element of a vector: RowView's segments
    auto part = [&](int C) {
        const int nv = (T::N - 1 + P.V + T::N - 1) / T::N;
        return (((nv + C * FW - 1) / (C * FW) + 31) & ~31) * FW * T::N;
    };
    // four CTAs to an SM: as many rows in flight as L2 holds beside other things, and where there are few rows,
    // clusters as large as all run at once (60 rows of 122187: 46 us under top-p, 71 us with twice as large ones, which
    // do not), with no part so short that the barriers are all there is; one step further for parts above 64 KB.
    // Clusters of 1, 2, 4, 8, 16, in us.  Parts down to 4 KB: one row of 32000 floats 41.9, 30.8, 23.0, 19.7, 19.1 under
    // top-p, 11.6, 10.1, 8.9, 9.1, 9.9 under top-k, 16 taken; one of 8000 16-bit logits 24.0, 23.6, 20.9, 21.6, 22.2, 4
    // taken.  Up to 64 KB where that fills the SMs: 120 rows of 128256 16-bit logits under top-p 82, 82, 62, 74, 125, 4
    // taken; 200 of 32000 floats 64, 51, 63, 86, 164, 2 taken.
    int C = 1;
    while (C < MAX_C && (std::min(n, (long long)(4 * sms / C)) * bytes > FLIGHT || part(C) > PART || (bytes / C > (2 * n * C <= 4 * sms ? 4096 : n * C < 4 * sms ? 65536 : bytes))))
        C *= 2;
    static std::atomic<uint64_t> raised{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(raised.load(std::memory_order_relaxed) & bit)) {
        e = cudaFuncSetAttribute(filter_rows<T, VERIFY>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess)
            return e;
        raised.fetch_or(bit, std::memory_order_relaxed);
    }
    return launch_clusters(filter_rows<T, VERIFY>, n, C, ROW_SMEM, false, stream, P);
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
    // a row that is not listed keeps a cluster busy; there are CTAs enough from 128 sequences on.  K = 4, 32000, clusters
    // of 4 and 8, in us: under top-p 32 sequences 66.7 and 59.7, 100 117.5 and 118.9, 128 139.0 and 138.8, 256 236 and
    // 251; eight kinds of requests 64 76.1 and 71.3, 160 126.9 and 130.0; listed rows 64 21.0 and 23.4, 256 74.5 and 83.7
    const int C = P.B >= 128 ? 4 : 8;
    e = tdt ? launch_clusters(filter_decide<RowBF16>, P.B, C, 0, true, stream, P)
            : launch_clusters(filter_decide<RowF32>, P.B, C, 0, true, stream, P);
    if (e == cudaSuccess)
        ++*launches;
    return e;
}

}  // namespace sv
