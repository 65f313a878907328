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
//
// Two launches: the tile kernel (k_attn_tiles.cu) works on the prefix and the
// caches and leaves partial results, each a reference exponent m, a sum l and
// weighted values o of a row over some of its entries.  The kernel here, one
// warp per row, attends to the staged entries (no partial result is awaited
// for that, so it overlaps the tile kernel's tail), joins the partial results
// (sums of 2^(m - max) l and 2^(m - max) o) and writes the row.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "sv_attn.cuh"
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

// One warp per query row.
template <int D>
__global__ void __launch_bounds__(RW * 32)
    va_finish(const __grid_constant__ AttnParams P, const __grid_constant__ AttnWork W, int ctas)
{
    constexpr int N = D / 32;   // elements per lane
    const float inf = __int_as_float(0x7f800000), nan = __int_as_float(0x7fc00000);
    const int lane = threadIdx.x & 31;
    const long long r = (long long)blockIdx.x * RW + threadIdx.x / 32;
    const bool real = r < (long long)P.B * P.T * P.Hq;
    const int hq = real ? (int)(r % P.Hq) : 0, h = hq / P.G, g = hq % P.G;
    const long long bt = real ? r / P.Hq : 0;
    const int t = (int)(bt % P.T), b = (int)(bt / P.T);
    const int len = __ldg(P.len + b);
    const bool bad = len < 0 || len > P.L;
    float o[N] = {}, m = -inf, l = 0.0f;
    if (real && P.staged && !bad) {
        float q[N];
        load_bf16<N>(static_cast<const uint16_t *>(P.q) + (size_t)r * D + lane * N, q);
#pragma unroll
        for (int k = 0; k < N; ++k)
            q[k] *= P.c;
        const uint8_t *mask = P.mask ? P.mask + (size_t)bt * P.T : nullptr;
        const uint16_t *x = static_cast<const uint16_t *>(P.staged);
        for (int j = 0; j < P.T; ++j) {
            if (mask ? !__ldg(mask + j) : j > t)
                continue;
            const size_t at = ((size_t)b * P.T + j) * 2 * P.H * D + (size_t)h * D + lane * N;
            float kx[N], vx[N];
            load_bf16<N>(x + at, kx);
            load_bf16<N>(x + at + (size_t)P.H * D, vx);
            float s = 0.0f;
#pragma unroll
            for (int k = 0; k < N; ++k)
                s = fmaf(q[k], kx[k], s);
#pragma unroll
            for (int w = 16; w; w >>= 1)
                s += __shfl_xor_sync(0xffffffffu, s, w);
            const float mn = fmaxf(m, s), ref = mn == -inf ? 0.0f : mn;
            const float f = exp2f(m - ref), p = exp2f(s - ref);
            m = mn;
            l = l * f + p;
#pragma unroll
            for (int k = 0; k < N; ++k)
                o[k] = fmaf(p, vx[k], o[k] * f);
        }
    }
    int code = bad ? 1 : 0;
    if (ctas > 0) {
        asm volatile("griddepcontrol.wait;" ::: "memory");   // the tile kernel's results
        if (real && !bad) {
            // where this row's partial results are: over the prefix, then over its cache
            const int HS = P.H * W.own.tiles, UP = W.ppairs * W.pu;
            const long long U = UP + (long long)HS * __ldcg(W.base + P.B);
            auto owner = [&](int u) { return attn_owner(u, U, ctas); };
            int cnt0 = 0, c0 = 0, pair0 = 0, grp0 = 0, row0 = 0, cnt1 = 0, c1 = 0, pair1 = 0, grp1 = 0, row1 = 0;
            const int per0 = 2 - W.pre.two, per1 = 2 - W.own.two;   // partial results per CTA
            if (W.ppairs) {
                const int wide = W.pre.tq * (1 + W.pre.two), in = (int)(bt % wide);
                pair0 = h * W.pre.tiles + (int)(bt / wide);
                grp0 = in / W.pre.tq;
                row0 = (in % W.pre.tq) * P.G + g;
                c0 = owner(pair0 * W.pu);
                cnt0 = (owner((pair0 + 1) * W.pu - 1) - c0 + 1) * per0;
            }
            if (len > 0) {
                const int wide = W.own.tq * (1 + W.own.two), in = t % wide, ub = (len + AT_UNIT - 1) / AT_UNIT;
                const int i = h * W.own.tiles + t / wide, u = UP + __ldcg(W.base + b) * HS + i * ub;
                pair1 = b * HS + i;
                grp1 = in / W.own.tq;
                row1 = (in % W.own.tq) * P.G + g;
                c1 = owner(u);
                cnt1 = (owner(u + ub - 1) - c1 + 1) * per1;
            }
            const int all = cnt0 + cnt1;
            for (int i0 = 0; i0 < all; i0 += 32) {
                // lane i looks up partial result i0 + i, then all lanes read its values
                const int n = min(32, all - i0);
                const bool own = i0 + lane >= cnt0;
                const int i = i0 + lane - (own ? cnt0 : 0), per = own ? per1 : per0;
                float pm = -inf, pl = 0.0f;
                const float *src = nullptr;
                bool gave_up = false;
                if (lane < n) {
                    const int c = (own ? c1 : c0) + i / per;
                    const int gr = per == 2 ? i % 2 : own ? grp1 : grp0;
                    const int rows = (own ? W.own.tq : W.pre.tq) * P.G;
                    const size_t at = ((size_t)(c + (own ? pair1 : pair0)) * 2 + gr) * rows + (own ? row1 : row0);
                    const float2 ml = __ldcg((own ? W.ml_s : W.ml_p) + at);
                    pm = ml.x;
                    pl = ml.y;
                    src = (own ? W.o_s : W.o_p) + at * D;
                    gave_up = __ldcg(W.stat + c) != 0;
                }
                if (__any_sync(0xffffffffu, gave_up)) {
                    code = 7;
                    break;
                }
                float top = pm;
#pragma unroll
                for (int w = 16; w; w >>= 1)
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
                const float mn = fmaxf(m, top), ref = mn == -inf ? 0.0f : mn;
                const float f = exp2f(m - ref), wt = pl == 0.0f ? 0.0f : exp2f(pm - ref);
                float add = wt == 0.0f ? 0.0f : wt * pl;
#pragma unroll
                for (int w = 16; w; w >>= 1)
                    add += __shfl_xor_sync(0xffffffffu, add, w);
                m = mn;
                l = l * f + add;
#pragma unroll
                for (int k = 0; k < N; ++k)
                    o[k] *= f;
                for (int j = 0; j < n; ++j) {
                    const float wj = __shfl_sync(0xffffffffu, wt, j);
                    const float *sj = reinterpret_cast<const float *>(
                        __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(src), j));
                    if (wj == 0.0f)
                        continue;   // its values are not written when it has no entries
#pragma unroll
                    for (int k = 0; k < N; k += 2) {
                        const float2 v = __ldcg(reinterpret_cast<const float2 *>(sj + lane * N + k));
                        o[k] = fmaf(wj, v.x, o[k]);
                        o[k + 1] = fmaf(wj, v.y, o[k + 1]);
                    }
                }
            }
        }
    }
    if (!real)
        return;
    if (code && lane == 0 && P.status)
        atomicCAS(P.status, 0, code);
    const float inv = code ? nan : l == 0.0f ? 0.0f : 1.0f / l;
    uint16_t *out = static_cast<uint16_t *>(P.out) + (size_t)r * D + lane * N;
#pragma unroll
    for (int k = 0; k < N; k += 2)
        *reinterpret_cast<uint32_t *>(out + k) = pack_bf16(o[k] * inv, o[k + 1] * inv);
    if (P.lse && lane == 0)
        P.lse[r] = code ? nan : 0.6931471805599453f * (m + log2f(l));
}

template <int D>
cudaError_t finish(const AttnParams &P, const AttnWork &W, int ctas, unsigned grid, cudaStream_t stream)
{
    if (ctas == 0) {
        va_finish<D><<<grid, RW * 32, 0, stream>>>(P, W, 0);
        return cudaGetLastError();
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(RW * 32);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, va_finish<D>, P, W, ctas);
}

}  // namespace

bool attention_fits(int B, int T, int H, int G, int D, int P, int L)
{
    // units of the whole call, and every slot index, in 31 bits
    const AttnPlan a = attn_plan(B, T, H, G, D, P, L);
    return a.max_units < (1LL << 31) && (long long)B * H * a.own.tiles < (1LL << 30);
}

size_t attention_workspace(int B, int T, int H, int G, int D, int P, int L)
{
    return attn_plan(B, T, H, G, D, P, L).total;
}

cudaError_t launch_attention(const AttnParams &P, bool quant, void *workspace, int sms, uint32_t spin_limit,
                             cudaStream_t stream, int *launches)
{
    *launches = 0;
    if (P.status) {
        const cudaError_t e = cudaMemsetAsync(P.status, 0, sizeof(int32_t), stream);
        if (e != cudaSuccess)
            return e;
    }
    const AttnPlan a = attn_plan(P.B, P.T, P.H, P.G, P.D, P.P, P.L);
    char *w = static_cast<char *>(workspace);
    AttnWork W{};
    W.pre = a.pre;
    W.own = a.own;
    W.ppairs = a.ppairs;
    W.pu = a.pu;
    W.base = reinterpret_cast<int32_t *>(w + a.base);
    W.stat = reinterpret_cast<int32_t *>(w + a.stat);
    W.ml_p = reinterpret_cast<float2 *>(w + a.ml_p);
    W.o_p = reinterpret_cast<float *>(w + a.o_p);
    W.ml_s = reinterpret_cast<float2 *>(w + a.ml_s);
    W.o_s = reinterpret_cast<float *>(w + a.o_s);
    // one CTA per SM, fewer where even full caches have fewer units
    const int most = sms < AT_MAX_CTAS ? sms : AT_MAX_CTAS;
    const int ctas = (int)(a.max_units < most ? a.max_units : most);
    if (ctas > 0) {
        const cudaError_t e = launch_attn_tiles(P, W, quant, ctas, spin_limit, stream);
        if (e != cudaSuccess)
            return e;
        ++*launches;
    }
    const unsigned grid = (unsigned)(((long long)P.B * P.T * P.Hq + RW - 1) / RW);
    const cudaError_t e = P.D == 128 ? finish<128>(P, W, ctas, grid, stream) : finish<64>(P, W, ctas, grid, stream);
    if (e == cudaSuccess)
        ++*launches;
    return e;
}

}  // namespace sv
