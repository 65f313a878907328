// sv_attn.cuh -- work split and partial results of the verification attention,
// shared by the tile kernel (k_attn_tiles.cu), the kernel that finishes the
// rows (k_attn.cu) and the host.
//
// A "pair" is a set of query rows and the stretch of entries they all see:
//   - prefix pairs: one key/value head and a tile of (sequence, token) rows,
//     over the P prefix entries;
//   - sequence pairs: one sequence, one key/value head and a tile of its
//     tokens, over its own cache entries.
// A pair's entries come in units of 128.  All pairs, prefix pairs first, form
// one line, on which a pair is as long as it takes: so much for each unit, and
// so much for the pair (Q, the first product, the results).  The line is cut
// into equal lengths, one per CTA, so ragged lengths balance by themselves; a
// CTA takes the units that begin in its length (the first one begins with the
// pair).  No length is shorter than the longest unit, so every CTA between a
// pair's first and its last has units of it.  Where there are fewer than
// SPREAD units per CTA, every unit counts 1 and a pair nothing: the call is
// short, and all the CTAs are better used than evenly loaded.
// CTA c leaves one partial result per pair it touches: (c, pair) runs along a
// staircase, on which c + pair never repeats, so c + pair is its slot.
//
// An 8-bit prefix under many rows is read back to bfloat16 first: the products
// over it bound the call then, and the kernel for bfloat16 entries runs them at
// 1.6 times the rate of the one for codes, while reading back takes 6 bytes per
// element once.  Whole calls, heads 32/8 x 128, read back and by codes: 64
// sequences of 32 tokens over 8192 entries, 290 us and 410 us; over 16384 entries
// and caches to 512, 1280 rows per key/value head, 134 us and 158 us, 1020 rows
// 117 us and 131 us, 640 rows 98 us and 105 us; over 8192, 1020 rows 88 us and
// 94 us, 520 rows 74 us and 73 us.  So it breaks even at about 600 rows, but from
// there to 1023 rows the codes stay, up to a tenth slower: their weights are
// float16, which is eight times as exact as bfloat16.  Prefix and caches are then
// two lines, of one launch each.
#pragma once
#include <cstdint>

#include "sv_params.h"

namespace sv {

constexpr int AT_ROWS = 128;      // query rows of a tile (one accumulator)
constexpr int AT_UNIT = 128;      // entries of a unit
constexpr int AT_MAX_CTAS = 192;  // CTAs that the workspace is sized for
constexpr int SPREAD = 4;

// Tiles of one kind of pair: a tile holds tq tokens (tq * G <= 128 rows), an
// item one or two tiles (two: both halves of the kernel work on the same
// entries; one: they take turns).  With 8-bit entries and few rows, the rows lie
// in their tile `copies` times in long stretches, each copy for a part of the
// entries, and what they leave is joined (`join`).  On the line, a unit is
// 1 << shift long, and a pair `over` more; 1 is about 0.45 us, measured: a unit
// of two tiles 1.8 us, its pair 3.6 us; a unit of one tile 1 us, its pair 1.8 us
// and up to 1.8 us more with the rows that are written (64 sequences of 32
// tokens, 8192 shared and 512 own entries, 32 heads: 278 us a call so, 359 us
// with 1 us a pair); with 8-bit entries a unit is taken for 0.9 us and a
// pair for 4 us (1.0 to 1.3 us a unit, where 1216 pairs of 8 to 32 units share the
// HBM).  Heads of 64 count the same; their units take 0.85 us in bfloat16 and 1 us
// in 8 bits.  At most 12: max_line.
struct AttnTiling {
    int tq, two, tiles, copies, join, shift, over;
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
    t.shift = t.two ? 2 : 1;
    t.over = t.two ? 8 : quant ? 9 : 4 + t.tq * G / 32;
    return t;
}

// Units of n >= 0 entries; n may lie just below 2^31.
__host__ __device__ constexpr int attn_units(int n) { return ((n - 1) >> 7) + 1; }
static_assert(AT_UNIT == 128 && attn_units(0) == 0 && attn_units(128) == 1 && attn_units(0x7fffffff) == 1 << 24, "units");

// A sliding window: of sequence b's cache entries, all its tokens see [0, sinks)
// and [from, n); what only some of them see, up to T - 1 entries ahead of `from`,
// the kernel that finishes the rows adds row by row, with their own bounds.  In
// units, the sinks come first, then the entries from `from` on, wherever that lies,
// so a window of 128 entries is one unit.  Few sinks under few rows are left to the
// other kernel as well: a unit of its own takes a pair 1 to 1.8 us of one SM, an entry
// of a row there 0.016 ns of the whole GPU (32 trees of 61 nodes, 64/8 heads, 16
// sinks: 179 us a call row by row, 139 us in units; 256 sequences of 5 tokens, 32/8
// heads, 4 sinks: 2048 units more are 13 us).
constexpr int FEW_SINKS = 640;   // times a pair's rows
struct AttnWindow {
    int n;      // entries of the sequence (0 where its length is out of range)
    int from;   // 0: every token sees all of them
    int sinks;  // in units; the others see to min(sinks, from)
    int few;    // row by row
    __device__ __forceinline__ AttnWindow(const AttnParams &A, int b)
    {
        n = __ldg(A.len + b);
        n = n < 0 || n > A.L ? 0 : n;
        // the last token sees T entries of this pass, itself included
        const int back = A.window - (A.staged ? A.T : 0);
        from = A.from ? A.from[b] : n - max(min(back, n), 0);
        from = from <= A.sinks ? 0 : from;
        const bool rows = A.sinks <= FEW_SINKS && A.sinks * min(A.T * A.G, 2 * AT_ROWS) <= FEW_SINKS;
        sinks = from > 0 && !rows ? A.sinks : 0;
        few = from > 0 && rows ? A.sinks : 0;
    }
    __device__ __forceinline__ int sink_units() const { return attn_units(sinks); }
    __device__ __forceinline__ int units() const { return attn_units(sinks) + attn_units(n - from); }
};

constexpr long long READ_BACK_ROWS = 1024;   // rows per key/value head from which an 8-bit prefix is read back

struct AttnPlan {
    AttnTiling pre, own;
    int split;           // an 8-bit prefix is read back, prefix and caches are lines of their own
    int ppairs;          // prefix pairs
    int pu;              // units of a prefix pair
    long long max_units, max_line;   // with every sequence at its capacity
    // byte offsets into the workspace
    size_t base, stat, line, from, ml_p, o_p, ml_s, o_s, prefix, total;
};

inline AttnPlan attn_plan(int B, int T, int H, int G, int D, int P, int L, bool quant)
{
    AttnPlan a{};
    a.split = quant && P > 0 && (long long)B * T * G >= READ_BACK_ROWS;
    a.pre = attn_tiling((long long)B * T, G, quant);
    a.own = attn_tiling(T, G, quant);
    a.pu = attn_units(P);
    a.ppairs = P > 0 ? H * a.pre.tiles : 0;
    const long long spairs = L > 0 ? (long long)B * H * a.own.tiles : 0;
    a.max_units = (long long)a.ppairs * a.pu + spairs * attn_units(L);
    a.max_line = 4 * a.max_units + 12 * (a.ppairs + spairs);
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t o = at;
        at = (at + bytes + 255) & ~(size_t)255;
        return o;
    };
    a.base = take((size_t)B * 8);
    a.stat = take(2 * AT_MAX_CTAS * 4);
    a.line = take(2 * 64);
    a.from = take((size_t)B * 4);
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

// What a kind of pair takes on the line.
struct AttnCost {
    int shift, over;
    __device__ __forceinline__ int pair(int units) const { return units > 0 ? (units << shift) + over : 0; }
    // where unit i begins in its pair; how many units begin ahead of x > 0
    __device__ __forceinline__ int begin(int i) const { return i == 0 ? 0 : (i << shift) + over; }
    __device__ __forceinline__ int ahead(int x) const
    {
        const int n = (x - over + (1 << shift) - 1) >> shift;
        return n > 1 ? n : 1;
    }
};

// A line, and its cut.
struct AttnLine {
    AttnCost pre, own_cost;
    long long length;
    int ctas;   // that share it
    int own;    // where the sequence pairs begin
    int total;  // one pair's worth of units of all sequences
    float rate; // ctas / length
    AttnLine() = default;
    // pu units and `ppairs` prefix pairs; HS pairs per sequence; `seqs` sequences with `units` in all
    __device__ __forceinline__ AttnLine(const AttnTiling &p, const AttnTiling &o, int ppairs, int pu, int HS, int units,
                                        int seqs, int most)
    {
        const long long all = (long long)ppairs * pu + (long long)HS * units;
        const bool brief = all < (long long)SPREAD * most;
        pre = brief ? AttnCost{0, 0} : AttnCost{p.shift, p.over};
        own_cost = brief ? AttnCost{0, 0} : AttnCost{o.shift, o.over};
        total = units;
        own = ppairs * pre.pair(pu);
        length = own + (long long)HS * sequences(units, seqs);
        // the longest unit is a first one
        const int a = ppairs > 0 ? pre.over + (1 << pre.shift) : 1, b = seqs > 0 ? own_cost.over + (1 << own_cost.shift) : 1;
        const long long n = length / (a > b ? a : b);
        ctas = (int)(n < most ? (n > 1 ? n : 1) : most);
        rate = __fdividef((float)ctas, (float)length);
    }
    // one pair's worth of `seqs` sequences with `units` in all
    __device__ __forceinline__ int sequences(int units, int seqs) const
    {
        return (units << own_cost.shift) + own_cost.over * seqs;
    }
    // where CTA c begins (and c - 1 ends)
    __device__ __forceinline__ int start(int c) const { return (int)(c < ctas ? c * length / ctas : length); }
    // which CTA has position x: the largest c with c length < (x + 1) ctas, from an estimate that is
    // off by one at most
    __device__ __forceinline__ int owner(int x) const
    {
        const long long y = ((long long)x + 1) * ctas;
        int c = (int)(((float)x + 1.0f) * rate);
        c -= c * length >= y;
        c += (c + 1) * length < y;
        return c;
    }
};

static_assert(sizeof(AttnLine) <= 64, "its place in the workspace");

// Device view of the plan.
struct AttnWork {
    AttnTiling pre, own;
    int ppairs, pu;
    int2 *base;      // [B] of the sequences before b: units (one pair's worth), how many have any; nullptr: not here
    struct AttnLine *line;   // this launch's, for the kernel that finishes the rows
    int32_t *stat;   // [CTAs] 0, or the code of a CTA that gave up
    float2 *ml_p, *ml_s;   // [slot][2][tq * G] reference exponent and sum of a partial row
    float *o_p, *o_s;      // [slot][2][D / 8][tq * G][8] its weighted values: rows side by side, as the threads that
                           // write them lie (with rows of D, 256 rows of results took 4 us; 1 us so)
};

}  // namespace sv
