// k_kvq.cu -- the KV cache in 8 bits: the commit that quantises, and reading
// back.
//
// One head's D elements of an entry (a key or a value) share a power of two:
// with amax the largest magnitude, e is the least integer with
// amax <= 448 * 2^e (448 is the largest e4m3 number), clamped to >= -126; the
// entry holds code(x) = e4m3(x * 2^-e), rounded to nearest even, and the byte
// e + 127.  x * 2^-e is exact in float32 (or so small that its code is 0), so a
// code is off by at most half a step of its format and nothing else, and it
// depends on no order of evaluation.  code * 2^e has 4 significant bits: exact in
// float32 up to byte 246, past which it may overflow, and in bfloat16 from byte 3
// on as well (its smallest step is 2^-133, the smallest code is 2^-9).
// A head whose elements include a NaN or an infinity gets the byte 255, which
// reads back as NaN everywhere.
//
// Both kernels are bound by HBM: the commit reads 2 D (or 4 D) bytes and
// writes D + 1 per head, reading back the reverse.  A thread takes pieces of
// eight elements: a warp's 16-byte loads (8-byte for codes) cover contiguous
// memory, a head's amax is a shuffle reduction over D / 8 lanes, and QU pieces
// are in flight per thread.  Reading 32 layers x 16 sequences x 512 entries of 8
// heads of 128 takes 207 us, all of the measured copy bandwidth.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "sv_fp8.cuh"
#include "sv_launch.h"

namespace sv {
namespace {

constexpr int QT = 128;   // threads of a CTA
constexpr int QU = 4;     // pieces in flight per thread (of a piece: 8 elements)
constexpr int QC = 1824;  // CTAs that a commit is spread over: as many as are resident

// ---------------------------------------------------------------- commit
__device__ __forceinline__ int commit_count(const KvQuantParams &P, int b)
{
    // entries that sequence b commits, -1 for one that reports an error
    const int a = __ldg(P.acc + b), n = P.len[b];
    if (a < 0)
        return 0;
    const long long m = (long long)a + P.lead;
    if (m > P.K || n < 0 || (long long)n + m > P.L)
        return -1;
    return (int)m;
}

// Eight elements as they lie in memory.
template <class E>
struct Piece {
    uint32_t w[2 * sizeof(E)];
};
template <class E>
__device__ __forceinline__ Piece<E> load_piece(const void *src, size_t at)
{
    Piece<E> x;
    const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const E *>(src) + at);
#pragma unroll
    for (int k = 0; k < (int)sizeof(E) / 2; ++k) {
        const uint4 v = __ldcs(p + k);   // read once
        x.w[4 * k] = v.x, x.w[4 * k + 1] = v.y, x.w[4 * k + 2] = v.z, x.w[4 * k + 3] = v.w;
    }
    return x;
}
// The largest of the absolute values' float32 bits.
template <class E>
__device__ __forceinline__ uint32_t piece_top(const Piece<E> &x)
{
    uint32_t m = 0;
    if constexpr (sizeof(E) == 2) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            m = __vmaxu2(m, x.w[k] & 0x7fff7fffu);
        return max(m << 16, m & 0xffff0000u);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            m = max(m, x.w[k] & 0x7fffffffu);
        return m;
    }
}
template <class E>
__device__ __forceinline__ float piece_at(const Piece<E> &x, int k)
{
    if constexpr (sizeof(E) == 2)
        return __uint_as_float((k & 1) ? x.w[k / 2] & 0xffff0000u : x.w[k / 2] << 16);
    else
        return __uint_as_float(x.w[k]);
}

// One CTA per (layer, sequence), QU pieces in flight per thread; where these are
// fewer than QC, several, which take its pieces in turn (a prompt of 16384
// entries, one layer and sequence, 8 heads of 128: 24.6 us with the length update,
// 4.1 TB/s; 15 ms by one CTA).  32 layers x 256 sequences with 3 entries each: 35 us with the length
// update, 4.3 TB/s, about 6 us of it the second launch.
template <class E, int D>
__global__ void __launch_bounds__(QT, sizeof(E) == 2 ? 12 : 8) kvq_commit(const __grid_constant__ KvQuantParams P)
{
    constexpr int G = D / 8;   // lanes of a head
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (blockIdx.x == 0 && threadIdx.x == 0 && P.status)
        *P.status = 0;   // only the length update, after this launch, reports
    const size_t lb = blockIdx.x / (unsigned)P.nch;   // layer * B + b
    const unsigned ch = blockIdx.x % (unsigned)P.nch;
    const int b = (int)(lb % (unsigned)P.B);
    const int n = commit_count(P, b);
    if (n <= 0)
        return;
    const int32_t *nodes = P.nodes ? P.nodes + (size_t)b * P.K : nullptr;
    if (nodes) {
        bool bad = false;
        for (int i = threadIdx.x; i < n - P.lead; i += QT)
            bad |= (unsigned)__ldg(nodes + i) >= (unsigned)P.K;
        if (__syncthreads_or(bad))
            return;
    }
    const unsigned per = 2 * P.H * G;            // pieces of an entry
    const unsigned total = n * per;              // a multiple of G: heads never end inside a lane group
    const size_t entry = (size_t)2 * P.H * D;    // elements of an entry
    const size_t src0 = lb * P.K, dst0 = lb * P.L + P.len[b];
    for (unsigned p0 = ch * (QT * QU) + threadIdx.x; p0 - threadIdx.x < total; p0 += P.nch * (QT * QU)) {
        Piece<E> x[QU];
        uint32_t top[QU];
#pragma unroll
        for (int u = 0; u < QU; ++u) {
            const unsigned p = p0 + u * QT;
            if (p < total) {
                const unsigned i = p / per;
                const int s = (nodes && (int)i >= P.lead) ? __ldg(nodes + i - P.lead) : (int)i;
                x[u] = load_piece<E>(P.staged, (src0 + s) * entry + (size_t)(p - i * per) * 8);
            } else {
                x[u] = Piece<E>{};
            }
        }
#pragma unroll
        for (int u = 0; u < QU; ++u) {
            top[u] = piece_top<E>(x[u]);
#pragma unroll
            for (int o = G / 2; o; o >>= 1)
                top[u] = max(top[u], __shfl_xor_sync(0xffffffffu, top[u], o));
            const unsigned p = p0 + u * QT;
            if (p >= total)
                continue;
            float inv;
            const uint32_t byte = fp8_scale(top[u], inv);
            float y[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                y[k] = piece_at<E>(x[u], k) * inv;
            // entries follow one another in the cache as the pieces do
            *reinterpret_cast<uint2 *>(P.cache + dst0 * entry + (size_t)p * 8) =
                make_uint2(pack_e4m3(y[0], y[1], y[2], y[3]), pack_e4m3(y[4], y[5], y[6], y[7]));
            if (p % G == 0)
                P.scale[dst0 * (2 * P.H) + p / G] = (uint8_t)byte;
        }
    }
}

// One warp per sequence: the length update.
__global__ void kvq_len(const __grid_constant__ KvQuantParams P)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");   // every copy has read the old lengths
    const int b = (blockIdx.x * blockDim.x + threadIdx.x) / 32, lane = threadIdx.x % 32;
    if (b >= P.B)
        return;
    const int n = commit_count(P, b);
    bool bad = n < 0;
    if (P.nodes)
        for (int i = lane; i < n - P.lead; i += 32)
            bad |= (unsigned)__ldg(P.nodes + (size_t)b * P.K + i) >= (unsigned)P.K;
    bad = __any_sync(0xffffffffu, bad);
    if (lane != 0)
        return;
    if (!bad)
        P.len[b] += n;
    else if (P.status)
        atomicCAS(P.status, 0, 1);   // past the capacity, above K, or a node outside [0, K)
}

// ---------------------------------------------------------------- read back
template <class E, int D>
__global__ void __launch_bounds__(QT) kvq_read(const __grid_constant__ KvQuantParams P)
{
    constexpr int G = D / 8;
    const int ch = blockIdx.x % P.nch;
    const long long lb = blockIdx.x / P.nch;
    const int b = (int)(lb % P.B);
    const int len = P.len_in ? __ldg(P.len_in + b) : P.L, start = P.start ? __ldg(P.start + b) : 0;
    const bool bad = len < 0 || len > P.L || start < 0;
    if (bad && threadIdx.x == 0 && P.status)
        atomicCAS(P.status, 0, 1);
    const int per = 2 * P.H * G;
    const long long total = (long long)P.K * per;                       // K: entries of the window
    const long long have = bad || start >= len ? 0 : (long long)min(P.K, len - start) * per;
    const long long p0 = (long long)ch * QT * QU + threadIdx.x;
    const uint8_t *codes = P.cache + ((size_t)lb * P.L + start) * per * 8;
    const uint8_t *scale = P.scale + ((size_t)lb * P.L + start) * (2 * P.H);
    E *out = static_cast<E *>(P.out) + (size_t)lb * total * 8;
    uint2 c[QU];
    uint32_t byte[QU];
#pragma unroll
    for (int u = 0; u < QU; ++u) {
        const long long p = p0 + u * QT;
        c[u] = make_uint2(0, 0);
        byte[u] = 127;
        if (p < have) {
            c[u] = __ldg(reinterpret_cast<const uint2 *>(codes) + p);
            byte[u] = __ldg(scale + p / G);
        }
    }
#pragma unroll
    for (int u = 0; u < QU; ++u) {
        const long long p = p0 + u * QT;
        if (p >= total)
            continue;
        float x[8];
        const float f = fp8_factor(byte[u]);
        unpack_e4m3(c[u].x, x);
        unpack_e4m3(c[u].y, x + 4);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            x[k] *= f;
        if constexpr (sizeof(E) == 2) {
            uint4 w;   // exact from byte 3 on: four significant bits
            w.x = pack_bf16(x[0], x[1]);
            w.y = pack_bf16(x[2], x[3]);
            w.z = pack_bf16(x[4], x[5]);
            w.w = pack_bf16(x[6], x[7]);
            *reinterpret_cast<uint4 *>(out + p * 8) = w;
        } else {
            float4 *o = reinterpret_cast<float4 *>(out + p * 8);
            o[0] = make_float4(x[0], x[1], x[2], x[3]);
            o[1] = make_float4(x[4], x[5], x[6], x[7]);
        }
    }
}

template <class E>
cudaError_t commit_any(const KvQuantParams &P, unsigned grid, cudaStream_t stream)
{
    if (P.D == 128)
        kvq_commit<E, 128><<<grid, QT, 0, stream>>>(P);
    else
        kvq_commit<E, 64><<<grid, QT, 0, stream>>>(P);
    return cudaGetLastError();
}

template <class E>
cudaError_t read_any(const KvQuantParams &P, unsigned grid, cudaStream_t stream)
{
    if (P.D == 128)
        kvq_read<E, 128><<<grid, QT, 0, stream>>>(P);
    else
        kvq_read<E, 64><<<grid, QT, 0, stream>>>(P);
    return cudaGetLastError();
}

}  // namespace

long long kvq_chunks(int K, int H, int D)
{
    const long long pieces = (long long)K * 2 * H * (D / 8);
    return (pieces + QT * QU - 1) / (QT * QU);
}

cudaError_t launch_kvq_commit(KvQuantParams P, bool wide, cudaStream_t stream, int *launches)
{
    const long long rows = (long long)P.NL * P.B, chunks = kvq_chunks(P.K, P.H, P.D), want = QC / rows;
    P.nch = (int)(want < 1 ? 1 : want < chunks ? want : chunks);
    const unsigned grid = (unsigned)(rows * P.nch);
    *launches = 0;
    const cudaError_t e = wide ? commit_any<float>(P, grid, stream) : commit_any<__nv_bfloat16>(P, grid, stream);
    if (e != cudaSuccess)
        return e;
    ++*launches;
    const cudaError_t f = launch_after(kvq_len, (P.B + 7) / 8, 256, 0, stream, P);
    if (f == cudaSuccess)
        ++*launches;
    return f;
}

cudaError_t launch_kvq_read(KvQuantParams P, bool wide, cudaStream_t stream)
{
    P.nch = (int)kvq_chunks(P.K, P.H, P.D);
    if (P.status) {
        const cudaError_t e = cudaMemsetAsync(P.status, 0, sizeof(int32_t), stream);
        if (e != cudaSuccess)
            return e;
    }
    const unsigned grid = (unsigned)((long long)P.NL * P.B * P.nch);
    return wide ? read_any<float>(P, grid, stream) : read_any<__nv_bfloat16>(P, grid, stream);
}

}  // namespace sv
