// sv_attn.cuh -- work split and partial results of the verification attention,
// shared by the tile kernel (k_attn_tiles.cu), the kernel that finishes the
// rows (k_attn.cu) and the host.
//
// A "pair" is a set of query rows and the stretch of entries they all see:
//   - prefix pairs: one key/value head and a tile of (sequence, token) rows,
//     over the P prefix entries;
//   - sequence pairs: one sequence, one key/value head and a tile of its
//     tokens, over its own cache entries.
// A pair's entries come in units of 128.  The units of all pairs, prefix
// pairs first, form one line that is cut into equal lengths, one per CTA, so
// ragged lengths balance by themselves; with fewer units than CTAs, the first
// CTAs take one each and the others none, so no CTA in between is idle.  CTA c leaves one partial result per
// pair it touches: (c, pair) runs along a staircase, on which c + pair never
// repeats, so c + pair is its slot.
//
// An 8-bit prefix under many rows is read back to bfloat16 first: the products
// over it bound the call then, and the kernel for bfloat16 entries runs them at
// 1.4 times the rate of the one for codes (64 sequences of 32 tokens, 32 heads,
// 8192 entries: 190 us and 301 us), while reading back takes 6 bytes per
// element once. That breaks even at about 700 rows per key/value head. Prefix
// and caches are then two lines, of one launch each.
#pragma once
#include <cstdint>

#include "sv_params.h"

namespace sv {

constexpr int AT_ROWS = 128;      // query rows of a tile (one accumulator)
constexpr int AT_UNIT = 128;      // entries of a unit
constexpr int AT_MAX_CTAS = 192;  // CTAs that the workspace is sized for

// Tiles of one kind of pair: a tile holds tq tokens (tq * G <= 128 rows), an
// item one or two tiles (two: both halves of the kernel work on the same
// entries; one: they take turns).  With 8-bit entries and few rows, the rows lie
// in their tile `copies` times in long stretches, each copy for a part of the
// entries, and what they leave is joined (`join`).
struct AttnTiling {
    int tq, two, tiles, copies, join;
};
inline AttnTiling attn_tiling(long long tokens, int G, bool quant)
{
    AttnTiling t;
    const int cap = AT_ROWS / G;
    t.tq = (int)(tokens < cap ? tokens : cap);
    t.two = tokens > cap;
    const long long per = (long long)t.tq * (t.two ? 2 : 1);
    t.tiles = (int)((tokens + per - 1) / per);
    t.copies = !quant || t.two || t.tq * G > 64 ? 1 : t.tq * G > 32 ? 2 : 4;
    t.join = quant && !t.two;
    return t;
}

constexpr long long READ_BACK_ROWS = 1024;   // rows per key/value head from which an 8-bit prefix is read back

struct AttnPlan {
    AttnTiling pre, own;
    int split;           // an 8-bit prefix is read back, prefix and caches are lines of their own
    int ppairs;          // prefix pairs
    int pu;              // units of a prefix pair
    long long max_units; // with every sequence at its capacity
    // byte offsets into the workspace
    size_t base, stat, ml_p, o_p, ml_s, o_s, prefix, total;
};

inline AttnPlan attn_plan(int B, int T, int H, int G, int D, int P, int L, bool quant)
{
    AttnPlan a{};
    a.split = quant && P > 0 && (long long)B * T * G >= READ_BACK_ROWS;
    a.pre = attn_tiling((long long)B * T, G, quant);
    a.own = attn_tiling(T, G, quant);
    a.pu = (P + AT_UNIT - 1) / AT_UNIT;
    a.ppairs = P > 0 ? H * a.pre.tiles : 0;
    const long long spairs = L > 0 ? (long long)B * H * a.own.tiles : 0;
    a.max_units = (long long)a.ppairs * a.pu + spairs * ((L + AT_UNIT - 1) / AT_UNIT);
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t o = at;
        at = (at + bytes + 255) & ~(size_t)255;
        return o;
    };
    a.base = take(((size_t)B + 1) * 4);
    a.stat = take(2 * AT_MAX_CTAS * 4);
    const size_t rp = a.ppairs ? ((size_t)a.ppairs + AT_MAX_CTAS) * 2 * a.pre.tq * G : 0;
    const size_t rs = spairs ? ((size_t)spairs + AT_MAX_CTAS) * 2 * a.own.tq * G : 0;
    a.ml_p = take(rp * 8);
    a.o_p = take(rp * D * 4);
    a.ml_s = take(rs * 8);
    a.o_s = take(rs * D * 4);
    a.prefix = take(a.split ? (size_t)P * 2 * H * D * 2 : 0);
    a.total = at;
    return a;
}

// The line of U units over at most `ctas` CTAs: where CTA c starts (and c - 1
// ends), and which CTA works on unit u.
__device__ __forceinline__ int attn_start(int c, long long U, int ctas)
{
    const long long n = U < ctas ? U : ctas;
    return (int)(c < n ? c * U / n : U);
}
__device__ __forceinline__ int attn_owner(int u, long long U, int ctas)
{
    // the largest c with c U < (u + 1) n, from an estimate that is off by one at most
    const long long n = U < ctas ? U : ctas, x = ((long long)u + 1) * n;
    int c = (int)__fdividef((float)x, (float)U);
    c -= c * U >= x;
    c += (c + 1) * U < x;
    return c;
}

// Device view of the plan.
struct AttnWork {
    AttnTiling pre, own;
    int ppairs, pu;
    int32_t *base;   // [B + 1] units of the sequences before b (one pair's worth), then their total; nullptr: not here
    int32_t *stat;   // [CTAs] 0, or the code of a CTA that gave up
    float2 *ml_p, *ml_s;   // [slot][2][tq * G] reference exponent and sum of a partial row
    float *o_p, *o_s;      // [slot][2][tq * G][D] its weighted values
};

}  // namespace sv
