// sv_filter.cuh -- filtered rows of logits (k_filter.cu): parameters, and the
// arithmetic of their weights.
//
// A row's tokens in descending order of the logit z (lowest index first among
// equals) have the weights w = e^((z - max) / T).  top-k keeps the first k;
// top-p, of those, a token if the weights ahead of it sum up to less than p
// times the sum of what top-k left; min-p keeps w >= min_p; the first stays in
// any case.  All three keep a head of the order, so what a row keeps is told by
// one number, its last token: the cut.
//
// Which token a head ends with, and which token a uniform falls on, turns on
// sums of up to V weights, and one token more or less changes a draw.  So the
// weights are held in 64-bit integers, in units of 2^-43 of the largest: their
// sums are exact, the same in every order, and depend on no split of the work.
// A weight itself is right to 2^-31.5 (and to half a unit).  (The total that top-p
// takes its share of, where it comes from a histogram: every 1 + q rounded to 2^-29
// and every bin down to a unit, so right to 2^-29.)  With sums of float pairs, 2^-24
// of the smaller halves, many equal weights summed up to 2^-27 off.  With float32
// throughout, 2^-24 of a weight, the head of a row of 128256 tokens ends one
// token off about once in a thousand rows.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

#include "sv_kernel.cuh"
#include "sv_params.h"

namespace sv {

// 2^(j / 64) as two floats, the second in units of 2^-33.
struct FilterTable {
    float2 t[64];
};
constexpr double filter_pow2(int j)
{
    const double y = j * (0.69314718055994530942 / 64.0);
    double sum = 1.0, term = 1.0;
    for (int n = 1; n < 24; ++n) {
        term *= y / n;
        sum += term;
    }
    return sum;
}
constexpr FilterTable filter_table()
{
    FilterTable t{};
    for (int j = 0; j < 64; ++j) {
        const double v = filter_pow2(j);
        t.t[j].x = (float)v;
        t.t[j].y = (float)((v - (double)(float)v) * 0x1p33);
    }
    return t;
}

// The weights of one row.  2^((x - m) c) = 2^(i / 64) (1 + q): the exponent is the
// sum of a multiple of 1/64 and a rest r, |r| <= 1/128, exact up to its last bit;
// 2^r - 1 = y + y^2/2 + y^3/6 with y = r ln 2, off by 2^-34.
//
// m is the largest logit, or 0 where that is so near that its token's weight comes
// to within 2^-10 octaves of 1: all weights of the row have the one factor 2^(m c) then.
struct FilterWeight {
    static constexpr float ROUND = 196608.0f;   // 1.5 2^17: steps of 1/64
    float m, c_hi, c_lo;
    float low;              // logits below have weights below 2^-43.75, 0.6 of a unit, and count as none
    const float2 *table;    // in shared memory
    FilterWeight() = default;
    __device__ __forceinline__ FilterWeight(float top, float hi, float lo, const float2 *t)
    {
        m = hi > 0.0f && fabsf(top) * hi < 0x1p-10f ? 0.0f : top;
        c_hi = hi, c_lo = lo, table = t;
        low = hi > 0.0f ? __fadd_ru(m, __fdiv_rn(-43.75f, hi)) : m;
    }
    // A logit at or above the row's largest
    __device__ __forceinline__ float highest() const { return m != 0.0f || c_hi == 0.0f ? m : __fdiv_ru(0x1p-10f, c_hi); }
    // Two logits at or above `low` (others come to nothing that may be used): the bits of i / 64 + ROUND, and 2^33 q.
    // What d = x - m has lost is `rest`, exactly.  SHORT, logits of 8 bits: x - (d + m), which is exact where m is
    // the larger one, and where x is, since it is less than 2^16 times m: a multiple of m's last bit, d has 25 bits
    // at most and d + m 24.  (Nearer to 0 than that, m is 0.)
    template <bool SHORT>
    __device__ __forceinline__ f2 split(f2 x, uint32_t &i0, uint32_t &i1) const
    {
        const f2 mm = pk(m, m), nm = pk(-m, -m), one = pk(-1.0f, -1.0f), ch = pk(c_hi, c_hi), cl = pk(c_lo, c_lo);
        const f2 round = pk(ROUND, ROUND);
        const f2 d = add2(x, nm);
        f2 rest;
        if constexpr (SHORT) {
            rest = fma2(add2(d, mm), one, x);
        } else {
            const f2 back = fma2(x, one, d);
            rest = add2(fma2(fma2(back, one, d), one, x), fma2(back, one, nm));
        }
        const f2 t = fma2(d, ch, round);
        f2 r = fma2(d, ch, fma2(t, one, round));
        r = fma2(d, cl, r);
        r = fma2(rest, ch, r);
        float a, b;
        upk(t, a, b);
        i0 = __float_as_uint(a);
        i1 = __float_as_uint(b);
        constexpr float a1 = 0.69314718f * 0x1p33f, a2 = 0.24022651f * 0x1p33f, a3 = 0.055504109f * 0x1p33f;
        return mul2(r, fma2(r, fma2(r, pk(a3, a3), pk(a2, a2)), pk(a1, a1)));
    }
    // i alone, for a logit at or above `low`
    __device__ __forceinline__ int place(float x) const
    {
        return __float_as_int(__fmaf_rn(__fadd_rn(x, -m), c_hi, ROUND)) - __float_as_int(ROUND);
    }
    // 2^(i / 64) (1 + q) in units, for a logit at or above `low` (another comes to nothing that may be used): 2^(i mod
    // 64 / 64) to half a unit, its correction in steps of 2^-33; then the rest of i as a shift, to half a unit
    __device__ __forceinline__ u64 units(uint32_t i, float q) const
    {
        const float2 e = table[i & 63];
        const int n = (int)(__float_as_uint(ROUND) - i + 63) >> 6;   // ROUND's bits end in 22 zeros
        u64 w;
        asm("shl.b64 %0, %1, %2;" : "=l"(w) : "l"(1ull), "r"(n - 1));   // half of what is shifted out; 0 if nothing is
        w += (u64)((__float_as_uint(e.x) & 0x7fffffu) | 0x800000u) * (1u << 20);
        w += (u64)((long long)__float2int_rn(fmaf(e.x, q, e.y)) * 1024);
        asm("shr.u64 %0, %1, %2;" : "=l"(w) : "l"(w), "r"(n));
        return w;
    }
    // in units; 0 below `low`
    __device__ __forceinline__ u64 operator()(float x) const
    {
        if (!(x >= low))
            return 0;
        uint32_t i, j;
        float q, r;
        upk(split<false>(pk(x, x), i, j), q, r);
        return units(i, q);
    }
    // The weights whose sum of 1 + q is v 2^-29 and whose i is -bin, in units
    __device__ __forceinline__ u64 of_bin(u64 v, int bin) const
    {
        const float2 e = table[-bin & 63];
        const u64 t = (u64)((__float_as_uint(e.x) & 0x7fffffu) | 0x800000u) * (1u << 20) +
                      (long long)__float2int_rn(e.y) * 1024;
        return __umul64hi(v << 15, t << 20) >> ((bin + 63) >> 6);   // v < 2^48
    }
};

// What a number in [0, 1) is of a sum, downward and upward: exact products, without the 64-bit floating-point unit
// (16 clocks of an SM to a warp's instruction).
__device__ __forceinline__ u64 share_down(float u, u64 sum) { return __umul64hi(sum, __float2ull_rz(u * 0x1p64f)); }
__device__ __forceinline__ u64 share_up(float u, u64 sum)
{
    const u64 f = __float2ull_rz(u * 0x1p64f);
    return __umul64hi(sum, f) + (sum * f != 0);
}
// w / Z in units of 2^-62, for w <= Z: the same number for the same w and Z.
struct FilterShare {
    u64 r;
    int e;
    FilterShare() = default;
    __device__ __forceinline__ explicit FilterShare(u64 Z)
    {
        e = __clzll((long long)Z);
        r = (u64)(0x1p126 / (double)(Z << e));
    }
    __device__ __forceinline__ u64 operator()(u64 w) const { return __umul64hi(w << e, r); }
};

// Floats in their order, as unsigned numbers; -0 counts as 0.
__device__ __forceinline__ uint32_t filter_key(float x)
{
    const uint32_t u = __float_as_uint(x + 0.0f);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float filter_value(uint32_t k)
{
    return __uint_as_float(k ^ (((uint32_t)((int32_t)~k >> 31)) | 0x80000000u));
}

}  // namespace sv
