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
// weighted values o of a row over some of its entries.  The kernel here, four
// rows per warp, attends to the staged entries (no partial result is awaited
// for that, so it overlaps the tile kernel's tail), joins the partial results
// (sums of 2^(m - max) l and 2^(m - max) o) and writes the row.
#include <cstdint>
#include <type_traits>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "sv_attn.cuh"
#include "sv_cluster.cuh"
#include "sv_fp8.cuh"
#include "sv_launch.h"

namespace sv {
namespace {

constexpr size_t WORK_ALIGN = 256;     // partial results are read and written 32 bytes at a time
constexpr long long WIDE_ROWS = 2048;   // rows up to which each has a CTA of its own
constexpr long long WIDER_ROWS = 256;   // rows up to which that has 16 warps, not four

// E elements of a row per lane, as pairs.  Eight lanes to a row: lane s holds
// elements 8 s .. 8 s + 7 and, with E = 16, the same 64 further on.  A warp to a
// row: lane s holds E s .. E s + E - 1.  Every load of a row is contiguous.
template <int E>
struct RawRow {
    uint32_t w[E / 2];
};
template <int E>
__device__ __forceinline__ RawRow<E> load_row(const uint16_t *p)
{
    RawRow<E> r;
    if constexpr (E >= 8) {
#pragma unroll
        for (int k = 0; k < E / 8; ++k) {
            const uint4 v = __ldg(reinterpret_cast<const uint4 *>(p + k * 64));
            r.w[4 * k] = v.x, r.w[4 * k + 1] = v.y, r.w[4 * k + 2] = v.z, r.w[4 * k + 3] = v.w;
        }
    } else if constexpr (E == 4) {
        const uint2 v = __ldg(reinterpret_cast<const uint2 *>(p));
        r.w[0] = v.x, r.w[1] = v.y;
    } else {
        r.w[0] = __ldg(reinterpret_cast<const uint32_t *>(p));
    }
    return r;
}
template <int E>
__device__ __forceinline__ f2 pair_of(const RawRow<E> &r, int k)
{
    return pku(r.w[k] << 16, r.w[k] & 0xffff0000u);
}
// The same of a row of e4m3 codes, as bfloat16 (which holds them).
template <int E>
__device__ __forceinline__ RawRow<E> load_codes(const uint8_t *p)
{
    RawRow<E> r;
    uint32_t w[E / 4 > 0 ? E / 4 : 1];
    if constexpr (E >= 8) {
#pragma unroll
        for (int k = 0; k < E / 8; ++k) {
            const uint2 v = __ldg(reinterpret_cast<const uint2 *>(p + k * 64));
            w[2 * k] = v.x, w[2 * k + 1] = v.y;
        }
    } else if constexpr (E == 4) {
        w[0] = __ldg(reinterpret_cast<const uint32_t *>(p));
    } else {
        w[0] = __ldg(reinterpret_cast<const uint16_t *>(p));
    }
#pragma unroll
    for (int k = 0; k < E / 2; k += 2) {
        float x[4];
        unpack_e4m3(w[k / 2], x);
        r.w[k] = pack_bf16(x[0], x[1]);
        if (k + 1 < E / 2)
            r.w[k + 1] = pack_bf16(x[2], x[3]);
    }
    return r;
}
// E float32 of a row of a partial result; `step` floats from eight columns to the next eight
template <int E>
__device__ __forceinline__ void load_values(const float *p, int step, float (&y)[E])
{
    if constexpr (E >= 8) {
#pragma unroll
        for (int k = 0; k < E / 8; ++k)
            asm volatile("ld.global.cg.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                         : "=f"(y[8 * k]), "=f"(y[8 * k + 1]), "=f"(y[8 * k + 2]), "=f"(y[8 * k + 3]),
                           "=f"(y[8 * k + 4]), "=f"(y[8 * k + 5]), "=f"(y[8 * k + 6]), "=f"(y[8 * k + 7])
                         : "l"(p + k * 8 * step)
                         : "memory");
    } else if constexpr (E == 4) {
        const float4 v = __ldcg(reinterpret_cast<const float4 *>(p));
        y[0] = v.x, y[1] = v.y, y[2] = v.z, y[3] = v.w;
    } else {
        const float2 v = __ldcg(reinterpret_cast<const float2 *>(p));
        y[0] = v.x, y[1] = v.y;
    }
}

// Many rows (WIDE = false): eight lanes per query row.  A warp works on four
// heads of a token, and the index arithmetic and the loops over what they see
// serve four rows.  Seven CTAs to an SM and two partial results in flight:
// 124928 rows of 61-node trees take 66 us after the tile kernel so, 85 us with
// four in flight and four CTAs (118 registers).  Few rows: a CTA per row,
// of WIDE warps, each taking a share of what the row sees and of its partial
// results, of which there may be hundreds; the shares are joined in shared memory.
// 16 warps where there are CTAs for a part of the SMs only (131072 entries under
// 32 rows of one key/value head: 23 us a call, 46 us with four warps), else four
// (1280 rows: 19 us, 42 us with 16).
template <int D, int WIDE, int WIN>
__global__ void __launch_bounds__(WIDE ? WIDE * 32 : 128, WIDE ? 1 : WIN ? 6 : 7)
    va_finish(const __grid_constant__ AttnParams P, const __grid_constant__ AttnWork W, int launches, int per_token)
{
    constexpr int FW = WIDE ? WIDE : 4;   // warps
    constexpr int LPR = WIDE ? 32 : 8, E = D / LPR, NP = E / 2, AT = E < 8 ? E : 8;
    constexpr int STEP = WIDE ? LPR * FW : LPR;   // partial results looked up at a time
    constexpr int FLY = WIDE ? 8 : 2;             // of their values in flight
    const float inf = __int_as_float(0x7f800000), nan = __int_as_float(0x7fc00000);
    const int lane = threadIdx.x & 31, sub = lane % LPR;
    const int warp = threadIdx.x / 32;
    const int bt = blockIdx.x / per_token;
    const int hq = WIDE ? blockIdx.x - bt * per_token : (blockIdx.x - bt * per_token) * (FW * 4) + threadIdx.x / LPR;
    const bool real = hq < P.Hq;
    const int h = real ? hq / P.G : 0, g = real ? hq - h * P.G : 0;
    const int b = bt / P.T, t = bt - b * P.T;
    const size_t r = (size_t)bt * P.Hq + (real ? hq : 0);
    const int len = __ldg(P.len + b);
    const bool bad = len < 0 || len > P.L;
    f2 o[NP];
#pragma unroll
    for (int k = 0; k < NP; ++k)
        o[k] = pk(0.0f, 0.0f);
    float m = -inf, l = 0.0f;
    // joins n scores (-inf: none) and their values
    auto rescale = [&](float top) {
        const float mn = fmaxf(m, top), ref = mn == -inf ? 0.0f : mn, f = ex2a(m - ref);
        const f2 ff = pk(f, f);
        m = mn;
        l *= f;
#pragma unroll
        for (int k = 0; k < NP; ++k)
            o[k] = mul2(o[k], ff);
        return ref;
    };
    if (!bad && (WIN || P.staged)) {
        f2 q[NP];
        {
            const RawRow<E> raw = load_row<E>(static_cast<const uint16_t *>(P.q) + r * D + sub * AT);
            const f2 cc = pk(P.c, P.c);
#pragma unroll
            for (int k = 0; k < NP; ++k)
                q[k] = mul2(pair_of<E>(raw, k), cc);
        }
        // two entries at a time (`two` false: the second is the first once more), each `fk` and `fv` times its key
        // and value
        auto attend = [&](const RawRow<E> &ka, const RawRow<E> &va, float fka, float fva, const RawRow<E> &kb,
                          const RawRow<E> &vb, float fkb, float fvb, bool two) {
            f2 da = pk(0.0f, 0.0f), db = da;
#pragma unroll
            for (int k = 0; k < NP; ++k) {
                da = fma2(q[k], pair_of<E>(ka, k), da);
                db = fma2(q[k], pair_of<E>(kb, k), db);
            }
            float a0, a1, b0, b1;
            upk(da, a0, a1);
            upk(db, b0, b1);
            float sa = a0 + a1, sb = b0 + b1;
#pragma unroll
            for (int w = LPR / 2; w; w >>= 1) {
                sa += __shfl_xor_sync(0xffffffffu, sa, w);
                sb += __shfl_xor_sync(0xffffffffu, sb, w);
            }
            sa *= fka;
            sb *= fkb;
            const float ref = rescale(two ? fmaxf(sa, sb) : sa);
            const float pa = ex2a(sa - ref), pb = two ? ex2a(sb - ref) : 0.0f;
            l += pa + pb;
            const f2 wa = pk(pa * fva, pa * fva), wb = pk(pb * fvb, pb * fvb);
#pragma unroll
            for (int k = 0; k < NP; ++k) {
                o[k] = fma2(wa, pair_of<E>(va, k), o[k]);
                if (two)
                    o[k] = fma2(wb, pair_of<E>(vb, k), o[k]);
            }
        };
        const size_t step = (size_t)2 * P.H * D;
        const uint8_t *mask = P.mask ? P.mask + (size_t)bt * P.T : nullptr;
        int cached = 0, seen_all = 0;   // the sequence's entries in the cache; how many of this pass the token sees
        if constexpr (WIN != 0) {
            // entries of the cache that the tile kernel leaves to the rows: few sinks, and what only some windows reach
            const AttnWindow win(P, b);
            cached = win.n;
            if (P.staged && mask) {
                for (int j0 = 0; j0 < P.T; j0 += 32)
                    seen_all += __popc(__ballot_sync(0xffffffffu, j0 + lane < P.T && __ldg(mask + j0 + lane)));
            } else if (P.staged) {
                seen_all = t + 1;
            }
            const int back = P.window - seen_all;   // of the cache's last entries
            // [0, few) and [low, from)
            const int low = win.from > 0 ? max(P.sinks, win.n - max(min(back, win.n), 0)) : 0;
            const int some = win.few + max(win.from - low, 0);
            const uint8_t *scale = P.cscale ? P.cscale + (size_t)b * P.L * 2 * P.H + h : nullptr;
            const size_t at0 = (size_t)b * P.L * step + (size_t)h * D + sub * AT;
            auto fetch = [&](int i, RawRow<E> &k, RawRow<E> &v, float &fk, float &fv) {
                const int e = i < win.few ? i : low + i - win.few;
                const size_t at = at0 + (size_t)e * step;
                if (scale) {
                    const uint8_t *p = static_cast<const uint8_t *>(P.cache) + at;
                    k = load_codes<E>(p);
                    v = load_codes<E>(p + (size_t)P.H * D);
                    fk = fp8_factor(__ldg(scale + (size_t)e * 2 * P.H));
                    fv = fp8_factor(__ldg(scale + (size_t)e * 2 * P.H + P.H));
                } else {
                    const uint16_t *p = static_cast<const uint16_t *>(P.cache) + at;
                    k = load_row<E>(p);
                    v = load_row<E>(p + (size_t)P.H * D);
                    fk = fv = 1.0f;
                }
            };
            constexpr int SHARE = WIDE ? FW : 1;
            for (int i = WIDE ? warp : 0; i < some; i += 2 * SHARE) {
                RawRow<E> ka, va, kb, vb;
                float fka, fva, fkb, fvb;
                const bool two = i + SHARE < some;
                fetch(i, ka, va, fka, fva);
                fetch(two ? i + SHARE : i, kb, vb, fkb, fvb);
                attend(ka, va, fka, fva, kb, vb, fkb, fvb, two);
            }
        }
        if (P.staged) {
            // this pass's own
            const uint16_t *x = static_cast<const uint16_t *>(P.staged) + (size_t)b * P.T * step + (size_t)h * D + sub * AT;
            const int end = mask ? P.T : t + 1;
            int ahead = 0;   // that the token sees, ahead of j0
            for (int j0 = 0; j0 < end; j0 += 32) {
                const int j = j0 + lane;
                unsigned seen = __ballot_sync(0xffffffffu, j < end && (!mask || __ldg(mask + j)));
                if constexpr (WIN != 0) {
                    // by its place among all the token's entries
                    const int rank = ahead + __popc(seen & ((1u << lane) - 1));
                    ahead += __popc(seen);
                    seen &= __ballot_sync(0xffffffffu, rank >= seen_all - P.window || cached < P.sinks - rank);
                }
                if constexpr (WIDE != 0)
                    seen &= (0xffffffffu / ((1u << FW) - 1)) << warp;   // this warp's share
                while (seen) {
                    const int ja = __ffs(seen) - 1;
                    seen &= seen - 1;
                    const bool two = seen != 0;
                    const int jb = two ? __ffs(seen) - 1 : ja;
                    seen &= seen - 1;
                    const uint16_t *ea = x + (size_t)(j0 + ja) * step, *eb = x + (size_t)(j0 + jb) * step;
                    attend(load_row<E>(ea), load_row<E>(ea + (size_t)P.H * D), 1.0f, 1.0f, load_row<E>(eb),
                           load_row<E>(eb + (size_t)P.H * D), 1.0f, 1.0f, two);
                }
            }
        }
    }
    int code = bad ? 1 : 0;
    // of the tile kernel ahead: none, one for all pairs, or one for the prefix and one for the caches
    if (launches > 0) {
        asm volatile("griddepcontrol.wait;" ::: "memory");   // the tile kernel's results
        if (!bad) {
            // where this row's partial results are: over the prefix, then over its cache
            const int HS = P.H * W.own.tiles;
            // two lines: each kind of pair has its own; one: the prefix pairs come first on both's
            const int two_lines = launches == 2;
            const int2 before = P.L > 0 ? __ldcg(W.base + b) : make_int2(0, 0);
            // not read through the non-coherent path: the tile kernel has just written them
            const AttnLine line0 = *W.line, line1 = two_lines ? W.line[1] : line0;
            int cnt0 = 0, c0 = 0, pair0 = 0, grp0 = 0, row0 = 0, cnt1 = 0, c1 = 0, pair1 = 0, grp1 = 0, row1 = 0;
            if (W.ppairs) {
                const int wide = W.pre.tq * (1 + W.pre.two), tile = bt / wide, in = bt - tile * wide;
                pair0 = h * W.pre.tiles + tile;
                grp0 = in >= W.pre.tq;
                row0 = (in - grp0 * W.pre.tq) * P.G + g;
                const int at = pair0 * line0.pre.pair(W.pu);
                c0 = line0.owner(at);
                cnt0 = (line0.owner(at + line0.pre.begin(W.pu - 1)) - c0 + 1) << (1 - W.pre.two);
            }
            const int ub = WIN ? AttnWindow(P, b).units() : attn_units(len);
            if (ub > 0) {
                const int wide = W.own.tq * (1 + W.own.two), tile = t / wide, in = t - tile * wide;
                const int i = h * W.own.tiles + tile;
                const int at = line1.own + HS * line1.sequences(before.x, before.y) + i * line1.own_cost.pair(ub);
                pair1 = b * HS + i;
                grp1 = in >= W.own.tq;
                row1 = (in - grp1 * W.own.tq) * P.G + g;
                c1 = line1.owner(at);
                cnt1 = (line1.owner(at + line1.own_cost.begin(ub - 1)) - c1 + 1) << (1 - W.own.two);
            }
            const int all = cnt0 + cnt1;   // may differ between the warp's rows
            const int rows0 = W.pre.tq * P.G, rows1 = W.own.tq * P.G;
            const int column = sub * AT & ~7;
            const float *const v0 = W.o_p + row0 * 8 + sub * AT % 8, *const v1 = W.o_s + row1 * 8 + sub * AT % 8;
            for (int i0 = 0; __any_sync(0xffffffffu, i0 < all); i0 += STEP) {
                // each lane of a row looks up a partial result, then all of them read the values
                const int at_i = i0 + (WIDE ? sub * FW + warp : sub);
                const bool own = at_i >= cnt0;
                const int i = at_i - (own ? cnt0 : 0), two = own ? W.own.two : W.pre.two;
                float pm = -inf, pl = 0.0f;
                int part = 0;   // which partial result, and of which kind
                bool gave_up = false;
                if (at_i < all) {
                    // with one set of rows, a CTA has one of each group (an empty one if they were joined)
                    const int c = (own ? c1 : c0) + (two ? i : i >> 1);
                    const int gr = two ? (own ? grp1 : grp0) : i & 1;
                    part = (c + (own ? pair1 : pair0)) * 2 + gr;
                    const float2 ml = own ? __ldcg(W.ml_s + (size_t)part * rows1 + row1)
                                          : __ldcg(W.ml_p + (size_t)part * rows0 + row0);
                    part = part * 2 + own;
                    pm = ml.x;
                    pl = ml.y;
                    gave_up = __ldcg(W.stat + (own && two_lines ? AT_MAX_CTAS : 0) + c) != 0;
                }
                if (__any_sync(0xffffffffu, gave_up))
                    code = 7;
                float top = pm;
#pragma unroll
                for (int w = LPR / 2; w; w >>= 1)
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
                const float ref = rescale(top);
                // A partial result over no entries has no values.  One whose weight underflows is -0: its
                // values are read all the same, a NaN among them is the row's.  A sum that is NaN (every
                // score may be, which leaves pm = -inf) is the row's, too.
                float wt = 0.0f;
                if (pl != 0.0f) {
                    wt = pl == pl ? ex2a(pm - ref) : nan;
                    wt = wt == 0.0f ? -0.0f : wt;
                }
                float add = pl == 0.0f ? 0.0f : wt * pl;
#pragma unroll
                for (int w = LPR / 2; w; w >>= 1)
                    add += __shfl_xor_sync(0xffffffffu, add, w);
                l += add;
                // the partial results that some row of the warp has
                unsigned have = __ballot_sync(0xffffffffu, __float_as_uint(wt) != 0);
                if constexpr (WIDE == 0)
                    have = (have | have >> 8 | have >> 16 | have >> 24) & 0xffu;
                while (have) {
                    float wj[FLY], y[FLY][E];
#pragma unroll
                    for (int n = 0; n < FLY; ++n) {
                        const int j = have ? __ffs(have) - 1 : 0;
                        const float w = __shfl_sync(0xffffffffu, wt, j, LPR);
                        const int pj = __shfl_sync(0xffffffffu, part, j, LPR);
                        const int rows = pj & 1 ? rows1 : rows0;
                        const float *sj = (pj & 1 ? v1 : v0) + (size_t)(pj >> 1) * rows * D + column * rows;
                        wj[n] = have ? w : 0.0f;
                        have &= have - 1;
#pragma unroll
                        for (int k = 0; k < E; ++k)
                            y[n][k] = 0.0f;
                        if (__float_as_uint(wj[n]) != 0)
                            load_values<E>(sj, 8 * rows, y[n]);
                    }
#pragma unroll
                    for (int n = 0; n < FLY; ++n) {
                        const f2 ww = pk(wj[n], wj[n]);
#pragma unroll
                        for (int k = 0; k < NP; ++k)
                            o[k] = fma2(ww, pk(y[n][2 * k], y[n][2 * k + 1]), o[k]);
                    }
                }
            }
        }
    }
    if constexpr (WIDE != 0) {
        __shared__ float s_o[FW][D], s_m[FW], s_l[FW];
        __shared__ int s_code[FW];
#pragma unroll
        for (int k = 0; k < NP; ++k)
            upk(o[k], s_o[warp][sub * E + 2 * k], s_o[warp][sub * E + 2 * k + 1]);
        if (lane == 0) {
            s_m[warp] = m;
            s_l[warp] = l;
            s_code[warp] = code;
        }
        __syncthreads();
        const int d = threadIdx.x * 2;
        if (d >= D)
            return;
        m = -inf;
#pragma unroll
        for (int w = 0; w < FW; ++w) {
            m = fmaxf(m, s_m[w]);
            code = max(code, s_code[w]);
        }
        const float ref = m == -inf ? 0.0f : m;
        float x = 0.0f, y = 0.0f;
        l = 0.0f;
#pragma unroll
        for (int w = 0; w < FW; ++w) {
            const float f = ex2a(s_m[w] - ref);
            l = fmaf(s_l[w], f, l);
            x = fmaf(s_o[w][d], f, x);
            y = fmaf(s_o[w][d + 1], f, y);
        }
        const float inv = code ? nan : l == 0.0f ? 0.0f : 1.0f / l;
        *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(P.out) + r * D + d) = pack_bf16(x * inv, y * inv);
    } else {
        if (!real)
            return;
        const float inv = code ? nan : l == 0.0f ? 0.0f : 1.0f / l;
        uint16_t *out = static_cast<uint16_t *>(P.out) + r * D + sub * AT;
        uint32_t w[NP];
#pragma unroll
        for (int k = 0; k < NP; ++k) {
            float lo, hi;
            upk(o[k], lo, hi);
            w[k] = pack_bf16(lo * inv, hi * inv);
        }
#pragma unroll
        for (int k = 0; k < E / 8; ++k)
            *reinterpret_cast<uint4 *>(out + k * 64) = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
    }
    if (WIDE ? threadIdx.x == 0 : sub == 0) {
        if (code && P.status)
            atomicCAS(P.status, 0, code);
        if (P.lse)
            P.lse[r] = code ? nan : 0.6931471805599453f * (m + log2f(l));
    }
}

// Where a window begins that all tokens of a sequence share, under a mask: the token that sees the most
// entries of this pass has the shortest one over the cache.  A CTA per sequence, eight lanes to a token, whose
// loads do not wait for one another (32 masks of 61 x 61: 13.5 us with a warp to a token in turn).
__global__ void __launch_bounds__(512) va_window(const __grid_constant__ AttnParams P, int32_t *from)
{
    const int b = blockIdx.x;
    __shared__ int most;
    if (threadIdx.x == 0)
        most = 0;
    __syncthreads();
    int top = 0;
    for (int t0 = 0; t0 < P.T; t0 += 64) {
        const int t = t0 + threadIdx.x / 8;
        int seen = 0;
        if (t < P.T) {
            const uint8_t *mask = P.mask + ((size_t)b * P.T + t) * P.T;
#pragma unroll 8
            for (int j = threadIdx.x % 8; j < P.T; j += 8)
                seen += __ldg(mask + j) != 0;
        }
#pragma unroll
        for (int o = 4; o; o >>= 1)
            seen += __shfl_xor_sync(0xffffffffu, seen, o);
        top = max(top, seen);
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if (threadIdx.x % 32 == 0)
        atomicMax(&most, top);
    __syncthreads();
    if (threadIdx.x == 0) {
        int n = __ldg(P.len + b);
        n = n < 0 || n > P.L ? 0 : n;
        from[b] = n - max(min(P.window - most, n), 0);
    }
}

template <int D, int WIDE, int WIN>
cudaError_t finish(const AttnParams &P, const AttnWork &W, int launches, cudaStream_t stream)
{
    constexpr int FW = WIDE ? WIDE : 4;
    const int per_token = WIDE ? P.Hq : (P.Hq + FW * 4 - 1) / (FW * 4);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(P.B * P.T * per_token));
    cfg.blockDim = dim3(FW * 32);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = launches > 0 ? 1 : 0;   // behind the tile kernel; alone it starts like any other
    return cudaLaunchKernelEx(&cfg, va_finish<D, WIDE, WIN>, P, W, launches, per_token);
}

}  // namespace

bool attention_fits(int B, int T, int H, int G, int D, int P, int L)
{
    // units of the whole call, and every slot index, in 31 bits
    const AttnPlan a = attn_plan(B, T, H, G, D, P, L, false);
    return a.max_line < (1LL << 31) && (long long)B * H * a.own.tiles < (1LL << 30);
}

size_t attention_workspace(int B, int T, int H, int G, int D, int P, int L)
{
    const size_t a = attn_plan(B, T, H, G, D, P, L, false).total, b = attn_plan(B, T, H, G, D, P, L, true).total;
    return (a > b ? a : b) + WORK_ALIGN - 16;   // the caller's is 16-byte aligned
}

cudaError_t launch_attention(AttnParams P, bool quant, void *workspace, int sms, uint32_t spin_limit,
                             cudaStream_t stream, int *launches)
{
    *launches = 0;
    if (P.status) {
        const cudaError_t e = cudaMemsetAsync(P.status, 0, sizeof(int32_t), stream);
        if (e != cudaSuccess)
            return e;
    }
    const AttnPlan a = attn_plan(P.B, P.T, P.H, P.G, P.D, P.P, P.L, quant);
    char *w = reinterpret_cast<char *>(((uintptr_t)workspace + WORK_ALIGN - 1) & ~(uintptr_t)(WORK_ALIGN - 1));
    AttnWork W{};
    W.pre = a.pre;
    W.own = a.own;
    W.ppairs = a.ppairs;
    W.pu = a.pu;
    W.base = reinterpret_cast<int2 *>(w + a.base);
    W.line = reinterpret_cast<AttnLine *>(w + a.line);
    W.stat = reinterpret_cast<int32_t *>(w + a.stat);
    W.ml_p = reinterpret_cast<float2 *>(w + a.ml_p);
    W.o_p = reinterpret_cast<float *>(w + a.o_p);
    W.ml_s = reinterpret_cast<float2 *>(w + a.ml_s);
    W.o_s = reinterpret_cast<float *>(w + a.o_s);
    if (P.window > 0 && P.mask && P.L > 0) {
        int32_t *from = reinterpret_cast<int32_t *>(w + a.from);
        va_window<<<P.B, 512, 0, stream>>>(P, from);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess)
            return e;
        ++*launches;
        P.from = from;
    }
    // one CTA per SM, fewer where even full caches have fewer units
    const long long most = sms < AT_MAX_CTAS ? sms : AT_MAX_CTAS;
    int lines = 0;
    auto tiles = [&](const AttnParams &A, const AttnWork &V, bool q8, long long units) {
        const int ctas = (int)(units < most ? units : most);
        if (ctas == 0)
            return cudaSuccess;
        const cudaError_t e = launch_attn_tiles(A, V, q8, ctas, lines > 0, spin_limit, stream);
        if (e == cudaSuccess) {
            ++*launches;
            ++lines;
        }
        return e;
    };
    cudaError_t e;
    if (a.split) {
        KvQuantParams R{};
        R.cache = static_cast<uint8_t *>(const_cast<void *>(P.prefix));   // read only
        R.scale = const_cast<uint8_t *>(P.pscale);
        R.out = w + a.prefix;
        R.NL = R.B = 1;
        R.K = R.L = P.P;
        R.H = P.H;
        R.D = P.D;
        e = launch_kvq_read(R, false, stream);
        if (e != cudaSuccess)
            return e;
        ++*launches;
        AttnParams A = P;
        AttnWork V = W;
        A.prefix = w + a.prefix;
        A.L = 0;
        V.base = nullptr;
        e = tiles(A, V, false, (long long)a.ppairs * a.pu);
        if (e != cudaSuccess)
            return e;
        A = P;
        A.P = 0;
        V = W;
        V.ppairs = 0;
        V.stat += AT_MAX_CTAS;
        ++V.line;
        e = tiles(A, V, true, a.max_units - (long long)a.ppairs * a.pu);
    } else {
        e = tiles(P, W, quant, a.max_units);
    }
    if (e != cudaSuccess)
        return e;
    const long long rows = (long long)P.B * P.T * P.Hq;
    const int wide = rows <= WIDER_ROWS ? 16 : rows <= WIDE_ROWS ? 4 : 0;
    auto of = [&](auto win) {
        constexpr int WIN = decltype(win)::value;
        if (P.D == 128)
            return wide == 16 ? finish<128, 16, WIN>(P, W, lines, stream)
                              : wide ? finish<128, 4, WIN>(P, W, lines, stream) : finish<128, 0, WIN>(P, W, lines, stream);
        return wide == 16 ? finish<64, 16, WIN>(P, W, lines, stream)
                          : wide ? finish<64, 4, WIN>(P, W, lines, stream) : finish<64, 0, WIN>(P, W, lines, stream);
    };
    e = P.window > 0 ? of(std::integral_constant<int, 1>{}) : of(std::integral_constant<int, 0>{});
    if (e == cudaSuccess)
        ++*launches;
    return e;
}

}  // namespace sv
