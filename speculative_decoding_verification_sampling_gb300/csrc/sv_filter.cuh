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
// A weight itself is right to 2^-31.5 (and to half a unit).  With float32
// throughout, 2^-24 of a weight, the head of a row of 128256 tokens ends one
// token off about once in a thousand rows.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

#include "sv_params.h"

namespace sv {

typedef unsigned long long u64;

// One set of filters, an entry per sequence; nullptr: off (T: 1).
struct FilterSet {
    const float *T;
    const int32_t *k;
    const float *p;
    const float *least;
};

// What is kept of a row, for the kernel that verifies: the tokens with
// (z, index) at the cut or ahead of it.
struct FilterRow {
    float m, c_hi, c_lo;   // the largest logit; log2(e) / T as two floats
    float cut;             // kept: z > cut, or z == cut and index <= last
    uint32_t last;
    int32_t n;             // tokens kept, listed in the workspace; -1: not listed
    u64 Z;                 // their weights' sum
    int32_t code;          // 0, or a status
    int32_t pad[7];
};
static_assert(sizeof(FilterRow) == 64, "a row's record");

constexpr int FILTER_CAP = 2048;   // tokens of a row that are ranked together, and listed
constexpr int FILTER_MAX_V = 524288;

struct FilterParams {
    const void *logits;      // [B][rows][V]: sample: [B][K]; verify: the target's [B][K + 1]
    const void *draft;       // verify: [B][K][V]
    const float *uniforms;   // sample: [B][K]; verify: [B][K + 1][2]
    const int32_t *tokens;   // verify: [B][K]
    FilterSet f, df;         // of the logits, and of the draft
    int32_t *out_tokens, *out_len;
    float *out_prob;
    int32_t *status;
    FilterRow *rows;         // verify: [B][2K + 1], target rows first
    int32_t *list_x;         // verify: [B][K + 1][FILTER_CAP], in the row's order
    u64 *list_w;
    int B, K, V;
};

// 2^(j / 64) as two floats.
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
        t.t[j].y = (float)(v - (double)(float)v);
    }
    return t;
}

constexpr float FILTER_UNIT = 8796093022208.0f;   // 2^43

// The weights of one row.
struct FilterWeight {
    float m, c_hi, c_lo, least;   // `least`: a z - m from which on weights are nothing, 2^-120
    const float2 *table;          // in shared memory
    FilterWeight() = default;
    __device__ __forceinline__ FilterWeight(float m_, float hi, float lo, const float2 *t)
        : m(m_), c_hi(hi), c_lo(lo), least(hi > 0.0f ? -120.0f / hi : -3e38f), table(t)
    {
    }
    // 2^((x - m) c) = 2^(i / 64) (1 + q).  The exponent is the sum of a multiple of 1/64 and a rest r,
    // |r| <= 1/128, both exact up to the last bits of r: 2^r - 1 = y + y^2/2 + y^3/6 with y = r ln 2, off by
    // 2^-34.
    static constexpr float ROUND = 196608.0f;   // 1.5 2^17: steps of 1/64
    // SHORT: logits of 8 bits.  Their difference is exact where they lie within 2^16 of each other; where x is
    // the smaller one, what is lost is x - (d + m).  (Where m is, 2^-16 of the other logits: 2^-24 of them is lost.)
    template <bool SHORT>
    __device__ __forceinline__ int split(float x, float &q) const
    {
        float d = x - m;
        float rest;
        if constexpr (SHORT) {
            rest = x - (d + m);
        } else {
            const float back = d - x;
            rest = (x - (d - back)) + (-m - back);
        }
        rest = d > least ? rest : 0.0f;
        d = fmaxf(d, least);
        const float zh = __fmul_rn(d, c_hi);   // not to be fused with what follows
        float zl = fmaf(d, c_hi, -zh);
        zl = fmaf(d, c_lo, zl);
        zl = fmaf(rest, c_hi, zl);
        const float t = zh + ROUND;
        const float r = (zh - (t - ROUND)) + zl;
        q = r * fmaf(r, fmaf(r, 0.055504109f, 0.24022651f), 0.69314718f);
        return __float_as_int(t) - __float_as_int(ROUND);
    }
    // the same i alone
    __device__ __forceinline__ int place(float x) const
    {
        return __float_as_int(__fadd_rn(__fmul_rn(fmaxf(x - m, least), c_hi), ROUND)) - __float_as_int(ROUND);
    }
    // as two floats, of which the second is small
    template <bool SHORT>
    __device__ __forceinline__ float2 pair(float x) const
    {
        float q;
        const int i = split<SHORT>(x, q);
        const float2 e = table[i & 63];
        const float s = __int_as_float(((i >> 6) + 127) << 23);
        return make_float2(e.x * s, fmaf(e.x, q, e.y) * s);
    }
    // in units
    __device__ __forceinline__ u64 operator()(float x) const
    {
        const float2 w = pair<false>(x);
        return (u64)(__float2ll_rn(w.x * FILTER_UNIT) + __float2ll_rn(w.y * FILTER_UNIT));
    }
};

// A thread's sum of weights: the rounding errors of the larger halves go with the smaller ones, so the sum is
// right to 2^-24 of those.  `s` begins at the largest weight there is.
struct FilterSum {
    float s = 1.0f, c = 0.0f;
    __device__ __forceinline__ void add(float2 w)
    {
        const float t = s + w.x;
        c += (s - t) + w.x;
        c += w.y;
        s = t;
    }
    __device__ __forceinline__ u64 units() const
    {
        return (u64)(__float2ll_rn((s - 1.0f) * FILTER_UNIT) + __float2ll_rn(c * FILTER_UNIT));
    }
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
