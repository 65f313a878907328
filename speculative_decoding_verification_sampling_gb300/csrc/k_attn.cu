// k_attn.cu -- attention of the verification pass.
//
// One target forward pass verifies the drafts of a sequence: its T query
// tokens (the last emitted token and K drafts, or the nodes of a draft tree,
// nextadmin.net lesson "Speculative Decoding", § KV cache management;
// aiengineeringfromscratch.com Phase 10 lesson 25, § Tree attention
// verification) attend to
//   - a prefix of P entries shared by every sequence of the batch,
//   - the sequence's own cache entries [0, len[b]),
//   - the T staged entries of this pass, under the tree mask or causally.
// For query row r with score s_j = c q_r . k_j (c = scale * log2 e) over its
// visible entries j: out_r = sum_j 2^(s_j - m) v_j / sum_j 2^(s_j - m), and
// lse_r = ln sum_j e^(scale q_r . k_j).  A row that sees nothing gives 0 and
// -inf.  Scores, statistics and sums are float32.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "sv_fp8.cuh"
#include "sv_launch.h"

namespace sv {
namespace {

constexpr int RW = 4;   // rows (warps) of a row CTA

// N = 2 or 4 elements of a bfloat16 row
template <int N>
__device__ __forceinline__ void load_bf16(const uint16_t *p, float *x)
{
    uint32_t w[N / 2];
    if constexpr (N == 4) {
        const uint2 v = __ldg(reinterpret_cast<const uint2 *>(p));
        w[0] = v.x, w[1] = v.y;
    } else {
        w[0] = __ldg(reinterpret_cast<const uint32_t *>(p));
    }
#pragma unroll
    for (int k = 0; k < N / 2; ++k) {
        x[2 * k] = __uint_as_float(w[k] << 16);
        x[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
    }
}

// N = 2 or 4 elements of an e4m3 row with its factor (exact)
template <int N>
__device__ __forceinline__ void load_fp8(const uint8_t *p, float f, float *x)
{
    float y[4];
    unpack_e4m3(N == 4 ? __ldg(reinterpret_cast<const uint32_t *>(p)) : __ldg(reinterpret_cast<const uint16_t *>(p)),
                y);
#pragma unroll
    for (int k = 0; k < N; ++k)
        x[k] = y[k] * f;
}

// One warp per query row, the entries one after another.
template <int D, bool Q8>
__global__ void __launch_bounds__(RW * 32) va_rows(const __grid_constant__ AttnParams P)
{
    constexpr int N = D / 32;   // elements per lane
    const int lane = threadIdx.x & 31;
    const long long r = (long long)blockIdx.x * RW + threadIdx.x / 32;
    if (r >= (long long)P.B * P.T * P.Hq)
        return;
    const int hq = (int)(r % P.Hq), h = hq / P.G;
    const long long bt = r / P.Hq;
    const int t = (int)(bt % P.T), b = (int)(bt / P.T);
    uint16_t *out = static_cast<uint16_t *>(P.out) + (size_t)r * D + lane * N;
    const int len = __ldg(P.len + b);
    float o[N] = {}, q[N], m = -__int_as_float(0x7f800000), l = 0.0f;
    load_bf16<N>(static_cast<const uint16_t *>(P.q) + (size_t)r * D + lane * N, q);
#pragma unroll
    for (int k = 0; k < N; ++k)
        q[k] *= P.c;
    auto entry = [&](const float (&kx)[N], const float (&vx)[N]) {
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < N; ++k)
            s = fmaf(q[k], kx[k], s);
#pragma unroll
        for (int w = 16; w; w >>= 1)
            s += __shfl_xor_sync(0xffffffffu, s, w);
        const float mn = fmaxf(m, s);
        const float ref = mn == -__int_as_float(0x7f800000) ? 0.0f : mn;
        const float f = exp2f(m - ref), p = exp2f(s - ref);
        m = mn;
        l = l * f + p;
#pragma unroll
        for (int k = 0; k < N; ++k)
            o[k] = fmaf(p, vx[k], o[k] * f);
    };
    // entries [0, n) of a prefix or a cache whose first entry is `first`
    auto stretch = [&](const void *base, const uint8_t *scale, size_t first, int n) {
        const size_t step = (size_t)2 * P.H * D;
        float kx[N], vx[N];
        for (int j = 0; j < n; ++j) {
            const size_t e = first + j, at = e * step + (size_t)h * D + lane * N, av = at + (size_t)P.H * D;
            if constexpr (Q8) {
                const uint8_t *s = scale + e * 2 * P.H + h, *x = static_cast<const uint8_t *>(base);
                load_fp8<N>(x + at, fp8_factor(__ldg(s)), kx);
                load_fp8<N>(x + av, fp8_factor(__ldg(s + P.H)), vx);
            } else {
                load_bf16<N>(static_cast<const uint16_t *>(base) + at, kx);
                load_bf16<N>(static_cast<const uint16_t *>(base) + av, vx);
            }
            entry(kx, vx);
        }
    };
    const bool bad = len < 0 || len > P.L;
    if (!bad) {
        stretch(P.prefix, P.pscale, 0, P.P);
        stretch(P.cache, P.cscale, (size_t)b * P.L, len);
        if (P.staged) {
            const uint8_t *mask = P.mask ? P.mask + (size_t)bt * P.T : nullptr;
            const uint16_t *x = static_cast<const uint16_t *>(P.staged);
            for (int j = 0; j < P.T; ++j) {
                if (mask ? !__ldg(mask + j) : j > t)
                    continue;
                const size_t at = ((size_t)b * P.T + j) * 2 * P.H * D + (size_t)h * D + lane * N;
                float kx[N], vx[N];
                load_bf16<N>(x + at, kx);
                load_bf16<N>(x + at + (size_t)P.H * D, vx);
                entry(kx, vx);
            }
        }
    } else if (lane == 0 && P.status) {
        atomicCAS(P.status, 0, 1);
    }
    const float nan = __int_as_float(0x7fc00000), inv = bad ? nan : l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
    for (int k = 0; k < N; k += 2)
        *reinterpret_cast<uint32_t *>(out + k) = pack_bf16(o[k] * inv, o[k + 1] * inv);
    if (P.lse && lane == 0)
        P.lse[r] = bad ? nan : 0.6931471805599453f * (m + log2f(l));
}

}  // namespace

cudaError_t launch_attention(const AttnParams &P, bool quant, cudaStream_t stream, int *launches)
{
    *launches = 0;
    if (P.status) {
        const cudaError_t e = cudaMemsetAsync(P.status, 0, sizeof(int32_t), stream);
        if (e != cudaSuccess)
            return e;
    }
    const unsigned grid = (unsigned)(((long long)P.B * P.T * P.Hq + RW - 1) / RW);
    if (P.D == 128)
        quant ? va_rows<128, true><<<grid, RW * 32, 0, stream>>>(P) : va_rows<128, false><<<grid, RW * 32, 0, stream>>>(P);
    else
        quant ? va_rows<64, true><<<grid, RW * 32, 0, stream>>>(P) : va_rows<64, false><<<grid, RW * 32, 0, stream>>>(P);
    ++*launches;
    return cudaGetLastError();
}

}  // namespace sv
