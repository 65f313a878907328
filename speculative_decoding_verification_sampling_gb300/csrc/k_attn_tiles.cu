// k_attn_tiles.cu -- the verification attention over the shared prefix and the
// sequences' caches, on the tensor cores.
//
// For a tile of up to 128 query rows (the tokens and heads that read one
// key/value head) and 128 entries at a time:
//   S = Q K^T           tcgen05.mma, operands in shared memory, S in TMEM
//   P = 2^(c S - m)     one thread per row; P goes back to TMEM as bfloat16, over S
//   O = O + P V         tcgen05.mma, P from TMEM, V from shared memory, O in TMEM
// m is a reference exponent per row: it follows the row's maximum only once
// that has passed it by more than 8, so O is rescaled a few times per stretch
// and 2^(c S - m) stays below 2^8.  The sum l takes the unrounded weights.
// Rounding P to bfloat16 is what the tensor cores ask for when V is bfloat16:
// 2^-8 of each weight, in random directions, beside the output's own 2^-8.
//
// Two softmax groups of four warps keep the tensor cores busy during each
// other's exponentials.  Where the rows fill more than one tile, both groups
// work on the same entries (each K and V tile read once for 256 rows); where
// they do not, the groups take alternate units of the same rows and leave a
// partial result each.  A loader thread feeds a ring of K and V tiles with
// TMA; one warp issues every tcgen05.mma.
//
// Entries in 8 bits. What such a kernel has least of is shared-memory
// bandwidth: turning a tile of codes into 16-bit numbers reads and writes three
// times its bytes there. So K's codes go to the tensor cores as they are
// (kind::f8f6f4), and Q meets them as a sum of two e4m3 numbers: each row times
// a power of two that puts its largest element in (224, 448], then rounded, and
// the remainder rounded again. That is exact for elements down to 2^-10 of the
// row's largest, and off by 2^-18 of the largest at most. The scales of K's
// rows multiply the columns of S. V's codes become float16, by four warps, in
// the layout that TMA would have written, with scales relative to the unit's
// largest, which becomes 2^7: float16 holds a code times 2^s exactly for s in
// [-15, 7], and a head whose scale is more than 2^22 below loses its last bits
// (at 2^-40 of the unit's largest element); from 2^32 below on its factor is 0
// in float16, and so are its values (2^-32 of the largest). What the largest
// stands for, bv, goes back in exactly, into the exponent of the weights: O
// holds 2^(c S + bv - m) V with a reference m of its own, while l holds 2^(c S
// - n), n following the scores alone, so a unit counts in l whatever its
// values' scale is. A unit that is nothing beside m (2^-64 or less) is summed
// up relative to its own maximum; its P are 0 in float16 either way. The
// results leave with n alone: O times 2^(m - n). P is rounded to float16 here:
// by 2^-11 of a weight, but subnormal ones by 2^-25. So that these are far
// down, m stays 11 to 15 below the row's maximum (of c S + bv), and P may reach
// 2^15: 2^-11 holds for weights down to 2^-25 of the largest, and below that
// 2^-36 of it. A head of zeros, whose byte is 127, counts for nothing in its
// unit: an entry with most of a row's weight and zeros for values would push
// all the others down. With few rows, where HBM is the bound, one warp's pass
// over 128 scores per row and their scales is too long a chain: the rows then
// lie in their tile two or four times, and each warp of a group takes the
// columns that fall to its copy.
//
// Measured, 32 query and 8 key/value heads of 128: 64 sequences of 32 tokens over
// 8192 shared entries, 190 us, 1448 TFLOP/s (bound by the two groups' softmax, the
// tensor cores 62 % active); 64 of 5 tokens over 4096 own entries each, 174 us,
// 6.2 TB/s (HBM); 64 of 9 tokens over 8192 own 8-bit entries each, 265 us, 4.1
// TB/s (the chain of a unit, and the copies in flight beside tiles being
// converted); 256 of 5 tokens over 512 own 8-bit entries each, 117 us (9 us to a
// pair of four units: one warp's softmax over 128 columns is 1.8 us of each).
//
// The last unit of a stretch is ragged: scores past its end become -inf, and
// V's rows past it are zeroed in shared memory, since 0 * NaN would reach O.
#include <atomic>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "sv_attn.cuh"
#include "sv_cluster.cuh"
#include "sv_fp8.cuh"
#include "sv_launch.h"

namespace sv {
namespace {

// ------------------------------------------------------------------ PTX
__device__ __forceinline__ void tma_4d(uint32_t dst, const CUtensorMap *map, unsigned long long *bar, int x, int y,
                                       int z, int w)
{
    asm volatile("cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
                 "l"(map), "r"(saddr(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
                 : "memory");
}
__device__ __forceinline__ void tma_5d(uint32_t dst, const CUtensorMap *map, unsigned long long *bar, int x, int y,
                                       int z, int w, int v)
{
    asm volatile("cp.async.bulk.tensor.5d.shared::cta.global.tile.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst),
                 "l"(map), "r"(saddr(bar)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(v)
                 : "memory");
}

// Shared-memory operand, swizzled: the low word holds the start address and
// the leading offset, the high word the stride offset (eight rows), all in
// 16-byte units, descriptor version 1 and the swizzle code (2: rows of 128
// bytes, 4: of 64).  The issuing thread keeps to 32-bit additions on the low
// word: its own instructions are what the tensor cores wait for otherwise.
constexpr uint32_t DESC_128 = (1024u >> 4) | (1u << 14) | (2u << 29);
constexpr uint32_t DESC_64 = (512u >> 4) | (1u << 14) | (4u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lead)
{
    return ((addr & 0x3ffffu) >> 4) | ((lead >> 4) << 16);
}
// Instruction descriptor: A and B both bfloat16, float16 (kind::f16) or e4m3
// (kind::f8f6f4), float32 accumulator, M = 128.
enum MmaType { MMA_F16 = 0, MMA_E4M3 = 0, MMA_BF16 = 1 };
__host__ __device__ constexpr uint32_t mma_desc(int n, bool b_mn_major, MmaType type)
{
    return (1u << 4) | ((uint32_t)type << 7) | ((uint32_t)type << 10) | ((b_mn_major ? 1u : 0u) << 16) |
           ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc)
{
    asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d),
                 "r"(a), "r"(b), "r"(idesc), "r"(acc), "r"(DESC_128)
                 : "memory");
}
template <uint32_t B_HI>
__device__ __forceinline__ void mma_ss8(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc)
{
    asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %6};\n\t"
                 "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, %3, p;\n\t}" ::"r"(d),
                 "r"(a), "r"(b), "r"(idesc), "r"(acc), "r"(DESC_128), "r"(B_HI)
                 : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc)
{
    asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 db;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "mov.b64 db, {%2, %5};\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d),
                 "r"(a), "r"(b), "r"(idesc), "r"(acc), "r"(DESC_128)
                 : "memory");
}
__device__ __forceinline__ void mma_commit(unsigned long long *bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(saddr(bar))
                 : "memory");
}
// One lane of a converged warp, the same one every time.  A branch on it tells
// the compiler that one thread runs what follows, so that the operands of
// tcgen05.mma and TMA go to uniform registers directly.
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}
// A value that all lanes hold, made known as such.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }
__device__ __forceinline__ void mbar_arrive_n(unsigned long long *bar, uint32_t n)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(saddr(bar)), "r"(n) : "memory");
}
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void async_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

#define R4(f, i) f(i), f(i + 1), f(i + 2), f(i + 3)
#define R16(f, i) R4(f, i), R4(f, i + 4), R4(f, i + 8), R4(f, i + 12)
#define R32(f, i) R16(f, i), R16(f, i + 16)

// Columns of this warp's 32 lanes; the wait is part of the instruction block, so
// no use of x can be moved ahead of it.
__device__ __forceinline__ void tmem_ld(uint32_t addr, float (&x)[32])
{
#define OUT(i) "=f"(x[i])
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
                 "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
                 "tcgen05.wait::ld.sync.aligned;"
                 : R32(OUT, 0)
                 : "r"(addr)
                 : "memory");
#undef OUT
}
__device__ __forceinline__ void tmem_ld(uint32_t addr, float (&x)[128])
{
#define OUT(i) "=f"(x[i])
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
                 "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%128];\n\t"
                 "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
                 "{%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
                 "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%129];\n\t"
                 "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
                 "{%64, %65, %66, %67, %68, %69, %70, %71, %72, %73, %74, %75, %76, %77, %78, %79, "
                 "%80, %81, %82, %83, %84, %85, %86, %87, %88, %89, %90, %91, %92, %93, %94, %95}, [%130];\n\t"
                 "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
                 "{%96, %97, %98, %99, %100, %101, %102, %103, %104, %105, %106, %107, %108, %109, %110, %111, "
                 "%112, %113, %114, %115, %116, %117, %118, %119, %120, %121, %122, %123, %124, %125, %126, %127}, [%131];\n\t"
                 "tcgen05.wait::ld.sync.aligned;"
                 : R32(OUT, 0), R32(OUT, 32), R32(OUT, 64), R32(OUT, 96)
                 : "r"(addr), "r"(addr + 32), "r"(addr + 64), "r"(addr + 96)
                 : "memory");
#undef OUT
}
__device__ __forceinline__ void tmem_st(uint32_t addr, const uint32_t (&x)[16])
{
#define IN(i) "r"(x[i])
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::R16(IN, 0),
                 "r"(addr)
                 : "memory");
#undef IN
}
__device__ __forceinline__ void tmem_st(uint32_t addr, const uint32_t (&x)[32])
{
#define IN(i) "r"(x[i])
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
                 "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::R32(IN, 0),
                 "r"(addr)
                 : "memory");
#undef IN
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void store8(float *p, const float *x)
{
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(x[0]), "f"(x[1]), "f"(x[2]),
                 "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7])
                 : "memory");
}

// ------------------------------------------------------------------ layout
template <int D, bool Q8>
struct TileCfg {
    static constexpr uint32_t TILE = 128 * D * 2;            // a 16-bit tile: 128 rows of D, in blocks of 64 columns
    static constexpr uint32_t BLOCK = 128 * 128;             // one such block: 128 rows of 128 bytes
    static constexpr uint32_t RAW = 128 * D;                 // a tile of codes
    static constexpr uint32_t KT = Q8 ? RAW : TILE;          // K as the tensor cores read it
    static constexpr int NK = D == 128 ? 3 : 6;              // tiles in flight: K, V, V's codes
    static constexpr int NV = D == 128 ? 2 : Q8 ? 4 : 6;
    static constexpr int NR = Q8 ? (D == 128 ? 2 : 4) : 0;
    static constexpr uint32_t K0 = 2 * TILE, V0 = K0 + NK * KT, R0 = V0 + NV * TILE;   // behind two Q tiles
    static constexpr uint32_t TILES = R0 + NR * RAW;         // TileShared lies behind them
    static constexpr int THREADS = Q8 ? 512 : 384;
    // registers per thread: at launch, then of the softmax groups and of the
    // other warpgroups (their sum over the warpgroups stays within the launch's)
    static constexpr int REGS = Q8 ? 128 : 168, REGS_SOFT = Q8 ? 152 : 208, REGS_REST = Q8 ? 104 : 80;
    static_assert(2 * REGS_SOFT + (THREADS / 128 - 2) * REGS_REST <= THREADS / 128 * REGS, "register split");
};

constexpr int W_LOAD = 8, W_MMA = 9, W_SCALE = 10, W_CVT = 12;   // warps 0-7: softmax, two groups; 12-15: conversion
constexpr int FAC = 4;   // units whose scales are ready ahead

// A CTA's length of the line, and the pair in which it begins: where that is on
// the line, its sequence (-1: the prefix), head and tile.
struct Place {
    int from, to, pair, b, h, tile;
    AttnCost pre, own;
};

struct TileShared {
    unsigned long long q_full[2], q_empty[2], k_full[6], k_empty[6], v_full[6], v_empty[6], r_full[4], r_empty[4];
    unsigned long long s_full[2], p_ready[2], o_full[2], drain;
    unsigned long long q_ready[2], f_full[FAC], f_empty[FAC];   // 8-bit entries: Q in e4m3, a unit's scales
    uint32_t tmem;
    volatile int abort;
    int issued[3];   // copies, as the loader ends: Q, K, V (or its codes)
    Place start;
    unsigned long long sums[16];   // per warp
};
struct QuantShared : TileShared {
    alignas(16) float4 k_fac[FAC][AT_UNIT / 4];   // what a unit's rows of K stand for
    uint16_t v_fac[FAC][AT_UNIT];                 // float16 factors of its rows of V
    float v_unit[FAC];                            // log2 of what 1 stands for in its V
    uint8_t q_unit[2][AT_ROWS];                   // the scale bytes of Q's rows
    float2 nl[2][AT_ROWS];                        // n and l of both groups' rows, as an item is joined
};

constexpr uint32_t SMEM_MAX = 232448;
template <int D, bool Q8>
constexpr uint32_t tile_smem()
{
    constexpr uint32_t n = TileCfg<D, Q8>::TILES + (uint32_t)(Q8 ? sizeof(QuantShared) : sizeof(TileShared));
    static_assert(n <= SMEM_MAX, "shared memory of a CTA");
    return n;
}

struct TileParams {
    AttnParams A;
    AttnWork W;
    uint32_t spin_limit;
};

__device__ __forceinline__ int seq_units(const AttnParams &A, int b)
{
    const int n = __ldg(A.len + b);
    return n < 0 || n > A.L ? 0 : attn_units(n);
}

// Units from which a stretch of 8-bit entries with one set of rows uses copies of
// them and joins what the groups and copies leave (a fixed cost per stretch: 8 units
// each under 64 sequences of 5 tokens take 56 us without, 67 us with; 12 each 73 us
// and 75 us, 16 each 89 us either way; 64 each under 64 of 9, 265 us with, 304 us
// without).
constexpr int JOIN_UNITS = 12;

// One stretch of one pair, as a CTA works on it.
struct Item {
    int n;           // units
    int h, b;        // key/value head; sequence (-1: the prefix)
    int row0;        // first (sequence, token) row of the item's tiles
    int tokens;      // rows of that kind in the pair from row0 on
    int e0, left;    // first entry, entries from there to the end of the stretch
    int two;
    int copies;      // of the rows in a tile
    bool join;       // both groups' and all copies' results become one
    int slot;
};

// The items of one CTA, in order.  Every role walks them by itself.
struct Walk {
    const TileParams &P;
    Place at;
    int units;   // of the pair's stretch
    __device__ Walk(const TileParams &p, const Place &start) : P(p), at(start)
    {
        units = at.b < 0 ? P.W.pu : at.b < P.A.B ? seq_units(P.A, at.b) : 0;
    }
    __device__ bool next(Item &it)
    {
#pragma unroll 1
        while (at.pair < at.to) {
#pragma unroll 1
            while (units == 0)   // sequences without entries
                units = seq_units(P.A, ++at.b);
            const bool pre = at.b < 0;
            const AttnCost cost = pre ? at.pre : at.own;
            // the units that begin in this CTA's length
            const int u0 = at.from <= at.pair ? 0 : cost.ahead(at.from - at.pair);
            const int u1 = min(units, cost.ahead(at.to - at.pair));
            const AttnTiling &tl = pre ? P.W.pre : P.W.own;
            const int t0 = at.tile * (tl.tq << tl.two);
            it.h = at.h;
            it.b = at.b;
            it.two = tl.two;
            it.row0 = pre ? t0 : at.b * P.A.T + t0;
            it.tokens = (pre ? P.A.B * P.A.T : P.A.T) - t0;
            it.e0 = u0 * AT_UNIT;
            it.left = (pre ? P.A.P : __ldg(P.A.len + at.b)) - it.e0;
            it.slot = blockIdx.x + ((pre ? 0 : at.b * P.A.H) + at.h) * tl.tiles + at.tile;
            it.n = u1 - u0;
            it.join = tl.join && it.n >= JOIN_UNITS;
            it.copies = it.join ? tl.copies : 1;
            at.pair += cost.pair(units);
            if (++at.tile == tl.tiles) {
                at.tile = 0;
                if (++at.h == P.A.H) {
                    at.h = 0;
                    ++at.b;
                    units = at.b < P.A.B ? seq_units(P.A, at.b) : 0;
                }
            }
            if (it.n > 0)
                return true;
        }
        return false;
    }
};

// The K and V tiles of an item, in the order in which the tensor cores use
// them: the first K tile (with one set of rows the first two, one for each
// softmax group), then V 0, the next K, V 1, the next K, ...
struct TileRef {
    int unit, kind;   // kind 0: K, 1: V
};
__device__ __forceinline__ TileRef item_tile(const Item &it, int s)
{
    const int ahead = min(it.two ? 1 : 2, it.n), r = s - ahead, more = it.n - ahead;
    if (r < 0)
        return {s, 0};
    if (r < 2 * more)
        return (r & 1) ? TileRef{ahead + r / 2, 0} : TileRef{r / 2, 1};
    return {r - more, 1};
}

// A place in a ring of n slots and the parity of its current pass.
struct Ring {
    int slot = 0;
    uint32_t phase = 0;
    __device__ void next(int n)
    {
        if (++slot == n) {
            slot = 0;
            phase ^= 1;
        }
    }
};

// Bounded wait on a barrier of this CTA: false once the polls ran out or
// another role has given up.
__device__ __forceinline__ bool tile_wait(unsigned long long *bar, uint32_t parity, uint32_t limit, TileShared &sh)
{
#pragma unroll 1
    for (uint32_t it = 0;; ++it) {
        if (mbar_test(bar, parity))
            return true;
        if (it >= limit || sh.abort) {
            sh.abort = 1;
            return false;
        }
    }
}

// Whether the phase has completed, without waiting (a try_wait would suspend
// the thread for a while).
__device__ __forceinline__ bool mbar_poll(unsigned long long *bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok)
                 : "r"(saddr(bar)), "r"(parity)
                 : "memory");
    return ok != 0;
}

// The same for a whole warp: every lane waits, and all come to one answer.
__device__ __forceinline__ bool tile_wait_warp(unsigned long long *bar, uint32_t parity, uint32_t limit, TileShared &sh)
{
    return __all_sync(0xffffffffu, tile_wait(bar, parity, limit, sh));
}

// ------------------------------------------------------------------ roles
// The loader: one thread.  Q tiles as an item begins, then K and V tiles in
// the order in which the tensor cores use them.
template <int D, bool Q8>
__device__ void load_role(const TileParams &P, const CUtensorMap *mq_pre, const CUtensorMap *mq_own,
                          const CUtensorMap *m_pre, const CUtensorMap *m_own, TileShared &sh, uint32_t smem,
                          uint32_t limit)
{
    using C = TileCfg<D, Q8>;
    // V tiles, or their codes
    constexpr int NV = Q8 ? C::NR : C::NV;
    constexpr uint32_t V0 = Q8 ? C::R0 : C::V0, VT = Q8 ? C::RAW : C::TILE;
    unsigned long long *const vfull = Q8 ? sh.r_full : sh.v_full, *const vempty = Q8 ? sh.r_empty : sh.v_empty;
    Ring q, k, v;
    int nq = 0, nk = 0, nv = 0;   // copies issued
    Walk walk(P, sh.start);
    Item it, after;
    bool ok = true, more = walk.next(it), have_q = false;
#pragma unroll 1
    while (ok && more) {
        more = walk.next(after);
        bool early = false;
#pragma unroll 1
        for (int s = 0; ok && s < 2 * it.n; ++s) {
            // the item's Q, or the next item's as soon as its place is free (with one set of rows to both)
            const bool now = s == 0 && !have_q;
            if (now || (!early && more && !it.two && !after.two && mbar_poll(&sh.q_empty[q.slot], q.phase ^ 1))) {
                const Item &x = now ? it : after;
                const bool pre = x.b < 0;
                const CUtensorMap *mq = pre ? mq_pre : mq_own;
                const int tq = pre ? P.W.pre.tq : P.W.own.tq;
                early = !now;
#pragma unroll 1
                for (int g = 0; ok && g <= x.two; ++g) {
                    if (!(ok = tile_wait(&sh.q_empty[q.slot], q.phase ^ 1, limit, sh)))
                        break;
                    mbar_arrive_tx(&sh.q_full[q.slot], (uint32_t)x.copies * tq * P.A.G * D * 2);
#pragma unroll 1
                    for (int c = 0; c < D / 64 * x.copies; ++c) {
                        const int blk = c % (D / 64), copy = c / (D / 64);
                        tma_4d(smem + q.slot * C::TILE + blk * C::BLOCK + copy * (C::BLOCK / x.copies), mq,
                               &sh.q_full[q.slot], blk * 64, 0, x.h, x.row0 + g * tq);
                    }
                    q.next(2);
                    ++nq;
                }
            }
            const auto [j, kind] = item_tile(it, s);
            unsigned long long *const full = kind ? &vfull[v.slot] : &sh.k_full[k.slot];
            Ring &ring = kind ? v : k;
            if (!ok || !(ok = tile_wait(kind ? &vempty[v.slot] : &sh.k_empty[k.slot], ring.phase ^ 1, limit, sh)))
                break;
            const uint32_t dst = smem + (kind ? V0 + v.slot * VT : C::K0 + k.slot * C::KT);
            const int e = it.e0 + j * AT_UNIT;
            mbar_arrive_tx(full, VT);
#pragma unroll 1
            for (int x = 0; x < (Q8 ? 1 : D / 64); ++x) {
                if (it.b < 0)
                    tma_4d(dst + x * C::BLOCK, m_pre, full, x * 64, it.h, kind, e);
                else
                    tma_5d(dst + x * C::BLOCK, m_own, full, x * 64, it.h, kind, e, it.b);
            }
            if (kind) {
                v.next(NV);
                ++nv;
            } else {
                k.next(C::NK);
                ++nk;
            }
        }
        have_q = early;
        it = after;
    }
    sh.issued[0] = nq;
    sh.issued[1] = nk;
    sh.issued[2] = nv;
}

// The issuer of every tcgen05.mma: one warp, one elected lane issues.
template <int D, bool Q8>
__device__ void mma_role(const TileParams &P, TileShared &sh, uint8_t *tiles, uint32_t smem, uint32_t limit)
{
    using C = TileCfg<D, Q8>;
    constexpr uint32_t IS = mma_desc(128, false, Q8 ? MMA_E4M3 : MMA_BF16), IO = mma_desc(D, true, Q8 ? MMA_F16 : MMA_BF16);
    const int lane = threadIdx.x & 31;
    // with 8-bit entries one thread runs all of this; with others the warp does, and elects one to
    // issue, since it clears V's tail together
    auto wait = [&](unsigned long long *bar, uint32_t parity, uint32_t lim, TileShared &s) {
        return Q8 ? tile_wait(bar, parity, lim, s) : tile_wait_warp(bar, parity, lim, s);
    };
    auto lead = [] { return Q8 || elect_one(); };
    auto rejoin = [] {
        if (!Q8)
            __syncwarp();
    };
    const uint32_t tmem = Q8 ? sh.tmem : (uint32_t)uniform((int)sh.tmem);
    Ring q, kr, vr;
    uint32_t pphase = 0;   // a bit for each group
    bool ok = true;
    auto give = [&](unsigned long long *bar) {
        if (lead())
            mma_commit(bar);
        rejoin();
    };
    Walk walk(P, sh.start);
    Item it;
#pragma unroll 1
    while (ok && walk.next(it)) {
        if (!Q8) {
            it.n = uniform(it.n);
            it.two = uniform(it.two);
        }
        const int q0 = q.slot;
        for (int g = 0; ok && g <= it.two; ++g) {
            ok = wait(Q8 ? &sh.q_ready[q.slot] : &sh.q_full[q.slot], q.phase, limit, sh);
            q.next(2);
        }
        tc_after();
        int ks = 0, vs = 0;
        // S of group g and unit j; with K's next tile where it is the first to use it, and its last word on it
        auto scores = [&](int g, int j, bool takes, bool gives) {
            if (takes) {
                ks = kr.slot;
                ok = ok && wait(&sh.k_full[ks], kr.phase, limit, sh);
                kr.next(C::NK);
                tc_after();
            }
            if (ok && lead()) {
                const int qs = (q0 + (it.two ? g : 0)) & 1;
                const uint32_t a = desc_lo(smem + qs * C::TILE, 16), b = desc_lo(smem + C::K0 + ks * C::KT, 16);
                if constexpr (Q8) {
                    // two terms of Q: blocks of their own (D = 128), halves of a 128-byte row (D = 64)
                    constexpr uint32_t TERM = D == 128 ? C::BLOCK : 64;
#pragma unroll
                    for (int t = 0; t < 2; ++t)
#pragma unroll
                        for (int k = 0; k < D / 32; ++k)
                            mma_ss8<D == 128 ? DESC_128 : DESC_64>(tmem + g * 128, a + ((t * TERM + k * 32) >> 4),
                                                                   b + ((k * 32) >> 4), IS, t + k > 0);
                } else {
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint32_t at = ((k / 4) * C::BLOCK + (k % 4) * 32) >> 4;
                        mma_ss(tmem + g * 128, a + at, b + at, IS, k > 0);
                    }
                }
                mma_commit(&sh.s_full[g]);
                if (gives)
                    mma_commit(&sh.k_empty[ks]);
                if (!Q8 && j + 1 == it.n)   // the last product with this Q
                    mma_commit(&sh.q_empty[qs]);
            }
            rejoin();
        };
        // O of group g takes unit j
        auto values = [&](int g, int j, bool takes, bool gives) {
            if (takes) {
                vs = vr.slot;
                ok = ok && wait(&sh.v_full[vs], vr.phase, limit, sh);
                vr.next(C::NV);
                tc_after();
                const int nv = it.left - j * AT_UNIT;
                if (!Q8 && ok && nv < AT_UNIT) {
                    // V's rows past the stretch (the conversion from 8 bits leaves zeros there by itself)
#pragma unroll 1
                    for (int k = 0; k < D / 64; ++k)
#pragma unroll 1
                        for (int x = nv * 8 + lane; x < AT_UNIT * 8; x += 32)
                            *reinterpret_cast<uint4 *>(tiles + C::V0 + vs * C::TILE + k * C::BLOCK + x * 16) =
                                make_uint4(0, 0, 0, 0);
                    async_fence();
                    rejoin();
                }
            }
            // P of this group is in TMEM
            ok = ok && wait(&sh.p_ready[g], (g ? pphase >> 1 : pphase) & 1, limit, sh);
            pphase ^= 1u << g;
            tc_after();
            if (ok && lead()) {
                // V is read along its rows: blocks of 64 columns lie BLOCK apart, 16 rows are 2048 bytes
                const uint32_t b = desc_lo(smem + C::V0 + vs * C::TILE, C::BLOCK);
                const int step = it.two ? 1 : 2;
#pragma unroll
                for (int k = 0; k < AT_UNIT / 16; ++k)
                    mma_ts(tmem + 256 + g * D, tmem + g * 128 + k * 8, b + ((k * 2048) >> 4), IO, j >= step || k > 0);
                if (gives)
                    mma_commit(&sh.v_empty[vs]);
                if (j + step >= it.n)
                    mma_commit(&sh.o_full[g]);
            }
            rejoin();
        };
        // Two sets of rows: S0 S1, then for each unit P0 V, the next S0, P1 V, the next S1.
        if (it.two && !Q8) {
#pragma unroll 1
            for (int j = -1; ok && j < it.n; ++j) {
                const bool more = j + 1 < it.n;
                if (j >= 0)
                    values(0, j, true, false);
                if (more)
                    scores(0, j + 1, true, false);
                if (j >= 0)
                    values(1, j, false, true);
                if (more)
                    scores(1, j + 1, false, true);
            }
        } else {
            // one set: as its tiles come (or two, from the same few instructions)
#pragma unroll 1
            for (int i = 0; ok && i < it.n << (1 + it.two); ++i) {
                int g, j, kind;
                if (it.two) {
                    const int r = i - 2, u = r >> 2;
                    if (r < 0)
                        g = i, j = 0, kind = 0;
                    else if (u < it.n - 1)
                        g = (r >> 1) & 1, kind = 1 - (r & 1), j = u + 1 - kind;
                    else
                        g = r & 1, kind = 1, j = u;
                } else {
                    const TileRef x = item_tile(it, i);
                    g = x.unit & 1, j = x.unit, kind = x.kind;
                }
                if (kind)
                    values(g, j, !it.two || g == 0, !it.two || g == 1);
                else
                    scores(g, j, !it.two || g == 0, !it.two || g == 1);
            }
        }
        // 8-bit entries: the softmax groups have read the rows' scales, too
        if (Q8)
            for (int g = 0; ok && g <= it.two; ++g)
                give(&sh.q_empty[it.two ? (q0 + g) & 1 : q0]);
    }
}

// Where a role of the CTA has given up, and all of them have ended: waits for the
// copies and the products in flight, which the others may have issued without a
// wait of their own running out.  `warp`: this thread's.
template <int D, bool Q8>
__device__ void wind_down(TileShared &sh, int warp, uint32_t limit)
{
    using C = TileCfg<D, Q8>;
    constexpr int NV = Q8 ? C::NR : C::NV;
    if (warp == W_LOAD && elect_one()) {
        const int nq = sh.issued[0], nk = sh.issued[1], nv = sh.issued[2];
        unsigned long long *const vfull = Q8 ? sh.r_full : sh.v_full;
        for (int i = 1; i <= 2 && i <= nq; ++i)
            (void)ring_wait(&sh.q_full[(nq - i) % 2], ((nq - i) / 2) & 1, limit);
        for (int i = 1; i <= C::NK && i <= nk; ++i)
            (void)ring_wait(&sh.k_full[(nk - i) % C::NK], ((nk - i) / C::NK) & 1, limit);
        for (int i = 1; i <= NV && i <= nv; ++i)
            (void)ring_wait(&vfull[(nv - i) % NV], ((nv - i) / NV) & 1, limit);
    }
    if (warp == W_MMA && elect_one()) {   // the thread that issued them
        mma_commit(&sh.drain);
        (void)ring_wait(&sh.drain, 0, limit);
    }
    __syncthreads();
}

// Raises a row's reference exponent m to s where that has passed it by more than
// `slack`, and scales O and l down with it.
template <int D>
__device__ __forceinline__ void follow_maximum(uint32_t to, float s, float slack, bool first, bool real, float &m,
                                               float &l)
{
    const bool up = real && s > m + slack;
    if (!__any_sync(0xffffffffu, up))
        return;
    const float f = up ? ex2a(m - s) : 1.0f;   // 2^(-inf) = 0 the first time
    if (up) {
        m = s;
        l *= f;
    }
    if (first)
        return;
    // this group's last P V has completed: S after it has
#pragma unroll 1
    for (int k = 0; k < D; k += 32) {
        float o[32];
        uint32_t y[32];
        tmem_ld(to + k, o);
#pragma unroll
        for (int u = 0; u < 32; ++u)
            y[u] = __float_as_uint(o[u] * f);
        tmem_st(to + k, y);
    }
}

// One unit of a softmax group: this thread's row (`real`: it is one) of S, of
// which `nv` columns belong to the stretch, becomes its row of P.
template <int D>
__device__ __forceinline__ void softmax_unit(uint32_t ts, uint32_t to, int nv, float c, bool first, bool real,
                                             float &m, float &l)
{
    float x[AT_UNIT];
    tmem_ld(ts, x);
    if (nv < AT_UNIT) {
#pragma unroll
        for (int k = 0; k < AT_UNIT; ++k)
            x[k] = k < nv ? x[k] : -F_INF;
    }
    float top[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
    for (int k = 4; k < AT_UNIT; k += 4)
#pragma unroll
        for (int u = 0; u < 4; ++u)
            top[u] = fmaxf(top[u], x[k + u]);
    follow_maximum<D>(to, fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * c, 8.0f, first, real, m, l);
    const float ref = m == -F_INF ? 0.0f : m;
    const f2 cc = pk(c, c), nref = pk(-ref, -ref);
    f2 sum[2] = {pk(0.0f, 0.0f), pk(0.0f, 0.0f)};
    // P's 64 columns lie over those of S, which this thread has read
#pragma unroll
    for (int h = 0; h < AT_UNIT / 2; h += 32) {
        uint32_t p[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) {
            const f2 e = ex2x2(fma2(pk(x[2 * (h + k)], x[2 * (h + k) + 1]), cc, nref));
            sum[k & 1] = add2(sum[k & 1], e);
            float lo, hi;
            upk(e, lo, hi);
            p[k] = pack_bf16(lo, hi);
        }
        tmem_st(ts + h, p);
    }
    float lo, hi;
    upk(add2(sum[0], sum[1]), lo, hi);
    l += lo + hi;
    tmem_st_wait();
}

constexpr float FAR_BELOW = -3e38f;   // a score's reference where there is none yet; finite
constexpr float P_TOP = 11.0f, P_SLACK = 4.0f;   // float16: the largest P of a row lies in [2^11, 2^15] as m moves

// The same with 8-bit entries, over this copy's `nc` columns from `col` on (nv
// of them in the stretch): scores times the scales of their rows of K, V's unit
// in the exponent, P in float16; n and l are the row's maximum and its sum. In
// steps of 32 columns, twice over S: the loops are short on purpose, the warps
// of this kernel run six different programs and have to share the instruction
// cache.
template <int D>
__device__ __forceinline__ void softmax_unit8(uint32_t ts, uint32_t to, int col, int nc, int nv, float c, float bv,
                                              const float4 *k_fac, bool first, bool real, float &m, float &n,
                                              float &l)
{
    float x[32];
    auto load = [&](int k0) {
        tmem_ld(ts + col + k0, x);
#pragma unroll
        for (int k = 0; k < 32; k += 4) {
            const float4 y = k_fac[(k0 + k) / 4];
            upk(mul2(pk(x[k], x[k + 1]), pk(y.x, y.y)), x[k], x[k + 1]);
            upk(mul2(pk(x[k + 2], x[k + 3]), pk(y.z, y.w)), x[k + 2], x[k + 3]);
        }
        if (nv < k0 + 32) {
#pragma unroll
            for (int k = 0; k < 32; ++k)
                x[k] = k0 + k < nv ? x[k] : -F_INF;
        }
    };
    float top[4] = {-F_INF, -F_INF, -F_INF, -F_INF};
#pragma unroll 1
    for (int k0 = 0; k0 < nc; k0 += 32) {
        load(k0);
#pragma unroll
        for (int k = 0; k < 32; k += 4)
#pragma unroll
            for (int u = 0; u < 4; ++u)
                top[u] = fmaxf(top[u], x[k + u]);
    }
    const float most = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * c;
    float none = 0.0f;
    follow_maximum<D>(to, most + bv - P_TOP, P_SLACK, first, real, m, none);
    if (most > n + 8.0f) {
        l *= ex2a(n - most);
        n = most;
    }
    const float ref = fmaxf(fminf(m - bv, most + 64.0f), FAR_BELOW);   // finite, also where every score is -inf
    const f2 cc = pk(c, c), nref = pk(-ref, -ref);
    f2 sum[2] = {pk(0.0f, 0.0f), pk(0.0f, 0.0f)};
    uint32_t p[16];
    // a step's P lies over columns of S that this thread has read, or does not read at all
#pragma unroll 1
    for (int k0 = 0; k0 < nc; k0 += 32) {
        load(k0);
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const f2 e = ex2x2(fma2(pk(x[2 * k], x[2 * k + 1]), cc, nref));
            sum[k & 1] = add2(sum[k & 1], e);
            float lo, hi;
            upk(e, lo, hi);
            p[k] = pack_f16(lo, hi);
        }
        tmem_st(ts + (col + k0) / 2, p);
    }
    // nothing from the other copies' columns
#pragma unroll
    for (int k = 0; k < 16; ++k)
        p[k] = 0;
#pragma unroll 1
    for (int k0 = nc; k0 < AT_UNIT; k0 += 32)
        tmem_st(ts + ((col + k0) & (AT_UNIT - 1)) / 2, p);
    float lo, hi;
    upk(add2(sum[0], sum[1]), lo, hi);
    l = fmaf(lo + hi, ex2a(ref - n), l);
    tmem_st_wait();
}

// The eight softmax warps.  Warps that gave up keep coming here, item by item.
__device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// Joins the partial results of an item with one set of rows: both groups, and
// every copy, in chunks of columns by way of the item's Q tile, which nothing
// reads any more.  `half` is the root of the weight of this thread's part of its
// row, `any` whether its warp has values at all, `seen` whether its part does.
// dst: a partial result's values, of `rows` rows.
template <int D>
__device__ __forceinline__ void join_parts(uint8_t *scratch, uint32_t to, int part, int parts, int row, int have,
                                           bool any, bool seen, float half, float *dst, int rows)
{
    constexpr int CW = D / 4;        // columns of a chunk: 256 rows of them fill the Q tile
    constexpr int V = CW / 4;        // 16-byte vectors of a row's chunk
    const int tid = threadIdx.x;     // of 256
#pragma unroll 1
    for (int k = 0; k < 4; ++k) {
        float o[32];
        if (any)
            tmem_ld(to + k * CW, o);
        if (row < have) {
#pragma unroll
            for (int v = 0; v < V; ++v)
                *reinterpret_cast<float4 *>(scratch + ((part * have + row) * V + (v ^ (row % V))) * 16) =
                    !any || !seen ? make_float4(0.0f, 0.0f, 0.0f, 0.0f)
                                  : make_float4(o[4 * v] * half * half, o[4 * v + 1] * half * half,
                                                o[4 * v + 2] * half * half, o[4 * v + 3] * half * half);
        }
        softmax_sync();
#pragma unroll 1
        for (int i = tid; i < have * V; i += 256) {
            const int r = i / V, v = i % V;
            float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            for (int p = 0; p < parts; ++p) {
                const float4 z = *reinterpret_cast<const float4 *>(scratch + ((p * have + r) * V + (v ^ (r % V))) * 16);
                y.x += z.x, y.y += z.y, y.z += z.z, y.w += z.w;
            }
            *reinterpret_cast<float4 *>(dst + ((k * CW + v * 4) / 8 * rows + r) * 8 + v % 2 * 4) = y;
        }
        if (k == 3)
            async_fence();   // the tile is TMA's next
        softmax_sync();
    }
}

// Softmax of group g: a thread owns a row of the group's tile (a warp reaches
// only its own quarter of the TMEM lanes).
template <int D, bool Q8>
__device__ void softmax_role(const TileParams &P, QuantShared &sh, uint8_t *tiles, int g, uint32_t limit)
{
    using C = TileCfg<D, Q8>;
    const int lane = threadIdx.x & 31, w = (threadIdx.x / 32) & 3;
    const uint32_t lanes = (uint32_t)(w * 32) << 16;
    const uint32_t ts = sh.tmem + lanes + g * 128, to = sh.tmem + lanes + 256 + g * D;
    float c = P.A.c, bv = 0.0f;
    int unit = 0;   // of the CTA, as the item starts
    uint32_t sphase = 0, ophase = 0;
    bool ok = true;
    Ring q;
    Walk walk(P, sh.start);
    Item it;
    if (P.spin_limit < CL_PLAIN_POLLS && sh.start.from < sh.start.to) {
        // the first wait, in that many plain polls: a test's way to giving up
        ok = mbar_poll(&sh.s_full[g], 0);
        for (uint32_t k = 1; !ok && k < P.spin_limit; ++k)
            ok = mbar_poll(&sh.s_full[g], 0);
        if (!(ok = __all_sync(0xffffffffu, ok)))
            sh.abort = 1;
    }
#pragma unroll 1
    for (; walk.next(it); unit += it.n) {
        // the slot of this group's Q tile: the second of two, or the only one
        const int qs = it.two ? (q.slot + g) & 1 : q.slot;
        if (!it.two)
            q.next(2);
        const bool pre = it.b < 0;
        const int tq = pre ? P.W.pre.tq : P.W.own.tq, rows = tq * P.A.G;
        // this warp's copy of the rows, its columns and its row of the copy
        const int copies = Q8 ? it.copies : 1, quarters = 4 / copies, copy = w / quarters, col = copy * (AT_UNIT / copies);
        const int row = (w - copy * quarters) * 32 + lane;
        // rows of this group's tile that exist
        const int have = min(max(it.tokens - (it.two ? g * tq : 0), 0), tq) * P.A.G;
        const bool active = row - lane < have;
        const int cnt = it.two ? it.n : (it.n - g + 1) / 2;
        float m = -F_INF, n = FAR_BELOW, l = 0.0f;   // n: with 8-bit entries, l's reference
#pragma unroll 1
        for (int i = 0; ok && i < cnt; ++i) {
            const int j = it.two ? i : 2 * i + g, nv = it.left - j * AT_UNIT - col;
            if (!(ok = tile_wait_warp(&sh.s_full[g], sphase, limit, sh)))
                break;
            sphase ^= 1;
            tc_after();
            const int fs = (unit + j) % FAC;
            if (Q8 && !(ok = tile_wait_warp(&sh.f_full[fs], ((unit + j) / FAC) & 1, limit, sh)))
                break;
            if (active) {
                if constexpr (Q8) {
                    // written before Q was handed to the tensor cores that made S
                    if (i == 0)
                        c = P.A.c * fp8_factor(sh.q_unit[qs][w * 32 + lane]);
                    bv = sh.v_unit[fs];
                }
                if constexpr (Q8)
                    softmax_unit8<D>(ts, to, col, AT_UNIT / copies, nv, c, bv, sh.k_fac[fs] + col / 4, i == 0,
                                     row < have, m, n, l);
                else
                    softmax_unit<D>(ts, to, nv, c, i == 0, row < have, m, l);
            }
            tc_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&sh.p_ready[g]);
                if constexpr (Q8)   // eight arrivals: both groups read the unit's scales, or one does for both
                    mbar_arrive_n(&sh.f_empty[fs], it.two ? 1 : 2);
            }
        }
        if (ok && cnt > 0) {
            if ((ok = tile_wait_warp(&sh.o_full[g], ophase, limit, sh))) {
                ophase ^= 1;
                tc_after();
            }
        }
        float2 *const ml = pre ? P.W.ml_p : P.W.ml_s;
        float *const o_all = pre ? P.W.o_p : P.W.o_s;
        if (Q8 && it.join) {
            const size_t at = (size_t)it.slot * 2 * rows;
            sh.nl[g][w * 32 + lane] = make_float2(n, l);
            softmax_sync();
            float top = FAR_BELOW, sum = 0.0f;
#pragma unroll 1
            for (int p = 0; p < 2 * copies; ++p)
                top = fmaxf(top, sh.nl[p & 1][(p >> 1) * (AT_ROWS / copies) + row].x);
#pragma unroll 1
            for (int p = 0; p < 2 * copies; ++p) {
                const float2 y = sh.nl[p & 1][(p >> 1) * (AT_ROWS / copies) + row];
                sum = fmaf(y.y, ex2a(y.x - top), sum);
            }
            if (g == 0 && copy == 0 && row < have) {
                ml[at + row] = make_float2(top, sum);
                ml[at + rows + row] = make_float2(-F_INF, 0.0f);
            }
            join_parts<D>(tiles + qs * C::TILE, to, copy * 2 + g, 2 * copies, row, have, ok && cnt > 0 && active,
                          l != 0.0f, ex2a(0.5f * (m - top)), o_all + at * D, rows);
            if (ok && threadIdx.x == 0)
                mbar_arrive(&sh.q_empty[qs]);
        } else {
            const size_t at = ((size_t)it.slot * 2 + g) * rows;
            // in range: m - n lies in [-122, 117], as bv does in [-107, 120]
            const float to_n = Q8 ? ex2a(m - n) : 1.0f;
            if (row < have)
                ml[at + row] = make_float2(Q8 ? n : m, l);
            if (ok && cnt > 0 && active) {
#pragma unroll 1
                for (int k = 0; k < D; k += 32) {
                    float o[32];
                    tmem_ld(to + k, o);
                    if constexpr (Q8) {
#pragma unroll
                        for (int u = 0; u < 32; u += 2)
                            upk(mul2(pk(o[u], o[u + 1]), pk(to_n, to_n)), o[u], o[u + 1]);
                    }
                    if (row < have) {
#pragma unroll
                        for (int u = 0; u < 32; u += 8)
                            store8(o_all + at * D + ((k + u) / 8 * rows + row) * 8, o + u);
                    }
                }
            }
            if (Q8 && ok && w == 0 && lane == 0 && (it.two || g == 0))
                mbar_arrive(&sh.q_empty[qs]);
        }
        tc_before();
    }
}

// Scale bytes of four heads, 32 entries apart: those that are 127 and whose codes
// are all zeros (of either sign) become 0.  Rarely called, and kept out of line for
// that: inlined, it took the calls around it from 381 us to 426 us (128 sequences
// of 9 tokens to 8192 own entries), by its place in the instruction cache alone.
template <int D>
__device__ __noinline__ uint32_t without_zeros(uint32_t bytes, const uint8_t *codes, size_t step)
{
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
        const uint8_t *p = codes + i * step;
        bool none = (bytes >> (8 * i) & 255) == 127;
#pragma unroll 1
        for (int k = 0; none && k < D; k += 16) {
            const uint4 c = __ldg(reinterpret_cast<const uint4 *>(p + k));
            none = ((c.x | c.y | c.z | c.w) & 0x7f7f7f7fu) == 0;
        }
        if (none)
            bytes &= ~(255u << (8 * i));
    }
    __syncwarp();
    return bytes;
}

// 8-bit entries: one warp turns the units' scale bytes into factors, up to FAC
// units ahead; the bytes of later units are asked into the caches meanwhile.
template <int D>
__device__ __forceinline__ void scale_role(const TileParams &P, QuantShared &sh, uint32_t limit)
{
    const int lane = threadIdx.x & 31;
    const int stride = 2 * P.A.H;   // bytes from an entry to the next
    Walk walk(P, sh.start);
    Item it;
    Ring r;
#pragma unroll 1
    while (walk.next(it)) {
        const size_t e0 = (it.b < 0 ? 0 : (size_t)it.b * P.A.L) + it.e0;
        const uint8_t *sc = (it.b < 0 ? P.A.pscale : P.A.cscale) + e0 * stride + it.h;
        // the values' codes of its first entry
        const uint8_t *codes = static_cast<const uint8_t *>(it.b < 0 ? P.A.prefix : P.A.cache) +
                               (e0 * stride + P.A.H + it.h) * D;
        int asked = 0;
#pragma unroll 1
        for (int j = 0; j < it.n; ++j) {
#pragma unroll 1
            for (; asked < min(it.n, j + 2 * FAC); ++asked)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (asked * AT_UNIT + i * 32 + lane < it.left)
                        asm volatile("prefetch.global.L2 [%0];" ::"l"(sc + (size_t)(asked * AT_UNIT + i * 32 + lane) * stride));
            const int nv = it.left - j * AT_UNIT;
            uint32_t kb[4], vb[4], top;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                kb[i] = vb[i] = 0;
                if (i * 32 + lane < nv) {
                    const uint8_t *p = sc + (size_t)(j * AT_UNIT + i * 32 + lane) * stride;
                    kb[i] = __ldg(p);
                    vb[i] = __ldg(p + P.A.H);
                }
            }
            // V's are relative to the largest, no lower than 2^-100
            auto largest = [&] {
                top = 27;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    top = max(top, vb[i] == 255 ? 0u : vb[i]);
                top = __reduce_max_sync(0xffffffffu, top);
            };
            largest();
            if (top == 127) {   // heads of zeros do not count
                const uint32_t left = without_zeros<D>(vb[0] | vb[1] << 8 | vb[2] << 16 | vb[3] << 24,
                                                       codes + (size_t)(j * AT_UNIT + lane) * stride * D,
                                                       (size_t)32 * stride * D);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    vb[i] = left >> (8 * i) & 255;
                largest();
            }
            if (!tile_wait_warp(&sh.f_empty[r.slot], r.phase ^ 1, limit, sh))
                return;
            float *kf = reinterpret_cast<float *>(sh.k_fac[r.slot]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                kf[i * 32 + lane] = fp8_factor(kb[i]);
                const int e = (int)vb[i] - (int)top + 7 + 127;   // 2^(byte - top + 7)
                const float f = vb[i] == 255 ? __int_as_float(0x7fc00000) : __int_as_float(max(e, 0) << 23);
                sh.v_fac[r.slot][i * 32 + lane] = (uint16_t)pack_f16(f, 0.0f);
            }
            if (lane == 0)
                sh.v_unit[r.slot] = (float)((int)top - 7 - 127);
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&sh.f_full[r.slot]);
            r.next(FAC);
        }
    }
}

// 8-bit entries: Q to two e4m3 terms, V's codes to float16; warp w of the four
// takes rows 32 w .. 32 w + 31 of each tile of codes.  What runs rarely is kept short
// (four rows of Q at a time, the tail's zeros in a loop): the roles share the
// instruction cache, and with eight rows of Q at a time and the tail unrolled 64
// sequences of 9 tokens over 8192 own entries took 312 us where they took 261 us so.
template <int D>
__device__ void convert_role(const TileParams &P, QuantShared &sh, uint8_t *tiles, uint32_t limit)
{
    using C = TileCfg<D, true>;
    const int lane = threadIdx.x & 31, w = (threadIdx.x / 32) & 3;
    Ring r, s, q;
    Walk walk(P, sh.start);
    Item it;
    int unit = 0;   // of the CTA, as the item starts

    // A Q tile, in place, eight lanes to a row and four rows at a time: both terms of a row go
    // where the row was (D = 128: its two 128-byte pieces; D = 64: the two halves of its one).
    auto convert_q = [&](const Item &x) {
        if (!tile_wait_warp(&sh.q_full[q.slot], q.phase, limit, sh))
            return false;
        uint8_t *tile = tiles + q.slot * C::TILE;
        // four rows to a warp in turn, so that few rows keep all four busy
        const int rows = (x.b < 0 ? P.W.pre.tq : P.W.own.tq) * P.A.G, each = AT_ROWS / x.copies - 1;
#pragma unroll 1
        for (int r0 = w * 4; r0 < AT_ROWS; r0 += 16) {
            if ((r0 & each) >= rows)
                continue;
            const int row = r0 + lane / 8, c = (lane % 8) ^ (row & 7);
            uint8_t *at = tile + row * 128;
            uint4 v[D / 64];
            uint32_t top = 0;
#pragma unroll
            for (int k = 0; k < D / 64; ++k) {
                v[k] = *reinterpret_cast<const uint4 *>(at + k * C::BLOCK + (lane % 8) * 16);
                top = __vmaxu2(top, __vmaxu2(__vmaxu2(v[k].x & 0x7fff7fffu, v[k].y & 0x7fff7fffu),
                                             __vmaxu2(v[k].z & 0x7fff7fffu, v[k].w & 0x7fff7fffu)));
            }
            top = max(top & 0xffffu, top >> 16);
#pragma unroll
            for (int o = 4; o; o >>= 1)
                top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
            __syncwarp();   // every lane has its part of the rows
            // this lane's chunk of eight columns: half c & 1 of a term's 16-byte chunk 4 k + c / 2
            float inv;
            const uint32_t byte = fp8_scale(top << 16, inv);
#pragma unroll
            for (int k = 0; k < D / 64; ++k) {
                const uint32_t in[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
                uint32_t t0[2], t1[2];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    float y[4], z[4];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        y[2 * e] = __uint_as_float(in[2 * u + e] << 16) * inv;
                        y[2 * e + 1] = __uint_as_float(in[2 * u + e] & 0xffff0000u) * inv;
                    }
                    t0[u] = pack_e4m3(y[0], y[1], y[2], y[3]);
                    unpack_e4m3(t0[u], z);
                    t1[u] = pack_e4m3(y[0] - z[0], y[1] - z[1], y[2] - z[2], y[3] - z[3]);   // exact differences
                }
                const int chunk = 4 * k + c / 2, half = (c & 1) * 8;
                const uint32_t o0 = ((chunk ^ (row & 7)) << 4) + half;
                const uint32_t o1 = D == 128 ? C::BLOCK + o0 : (((chunk + 4) ^ (row & 7)) << 4) + half;
                *reinterpret_cast<uint2 *>(at + o0) = make_uint2(t0[0], t0[1]);
                *reinterpret_cast<uint2 *>(at + o1) = make_uint2(t1[0], t1[1]);
            }
            if (lane % 8 == 0)
                sh.q_unit[q.slot][row] = (uint8_t)byte;
        }
        async_fence();
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&sh.q_ready[q.slot]);
        q.next(2);
        return true;
    };

    // A tile of codes, 16 of a row per lane and pass.  A row's 16 codes become two 16-byte chunks
    // of the swizzled 16-bit layout (chunk c of row r at c ^ (r & 7)); the codes are swizzled the
    // same way (D = 64: at c ^ (r / 2 & 3)).  Eight lanes take four chunks of the rows r and r ^ 5:
    // their bit 2 keeps the loads, their bit 0 the stores apart, so neither meets a bank conflict.
    constexpr int PASSES = D / 16, STEP = D == 128 ? 2 : 1;   // passes; of them over the same eight rows
    const int c2 = lane & 3, blk = D == 128 ? (lane >> 3) & 1 : 0, hi = D == 128 ? lane >> 4 : lane >> 3;
    uint32_t src0[STEP], dst0[STEP];
    int row0[STEP];
#pragma unroll
    for (int k = 0; k < STEP; ++k) {
        const int r7 = (D == 128 ? 2 * k + hi : hi) ^ ((lane >> 2 & 1) * 5);
        row0[k] = w * 32 + r7;
        src0[k] = row0[k] * D + (D == 128 ? ((blk * 4 + c2) ^ r7) : (c2 ^ (r7 >> 1 & 3))) * 16;
        dst0[k] = blk * C::BLOCK + row0[k] * 128 + ((2 * c2) ^ r7) * 16;
    }
    auto convert = [&](const uint8_t *src, uint8_t *dst, const uint16_t *fac, int valid) {
        // every load ahead of the stores: the compiler cannot tell that they do not alias
        uint4 v[PASSES];
        uint32_t f[PASSES];
#pragma unroll
        for (int p = 0; p < PASSES; ++p) {
            const int k = p % STEP, o = p / STEP * 8;
            v[p] = *reinterpret_cast<const uint4 *>(src + src0[k] + o * D);
            f[p] = fac[row0[k] + o];
        }
#pragma unroll
        for (int p = 0; p < PASSES; ++p) {
            const int k = p % STEP, o = p / STEP * 8;
            const uint32_t ff = f[p] * 0x10001u;
            uint4 a, b;
            scale_e4m3(v[p].x, ff, a.x, a.y);
            scale_e4m3(v[p].y, ff, a.z, a.w);
            scale_e4m3(v[p].z, ff, b.x, b.y);
            scale_e4m3(v[p].w, ff, b.z, b.w);
            *reinterpret_cast<uint4 *>(dst + dst0[k] + o * 128) = a;
            *reinterpret_cast<uint4 *>(dst + (dst0[k] ^ 16) + o * 128) = b;
        }
        if (valid < AT_UNIT) {
            // the rows past the stretch
#pragma unroll 1
            for (int o = 0; o < PASSES / STEP * 8; o += 8)
#pragma unroll
                for (int k = 0; k < STEP; ++k) {
                    if (row0[k] + o < valid)
                        continue;
                    *reinterpret_cast<uint4 *>(dst + dst0[k] + o * 128) = make_uint4(0, 0, 0, 0);
                    *reinterpret_cast<uint4 *>(dst + (dst0[k] ^ 16) + o * 128) = make_uint4(0, 0, 0, 0);
                }
        }
    };

    Item after;
    bool more = walk.next(it), ready = false;
#pragma unroll 1
    while (more) {
        more = walk.next(after);
        bool early = false;
#pragma unroll 1
        for (int j = 0; j < it.n; ++j) {
            // the item's Q, or (one set of rows to both) the next item's as soon as it is there
            int todo = j == 0 && !ready ? it.two + 1 : 0;
            const bool now = todo > 0;
            if (!now && more && !early && !it.two && !after.two &&
                __all_sync(0xffffffffu, mbar_poll(&sh.q_full[q.slot], q.phase))) {
                todo = 1;
                early = true;
            }
#pragma unroll 1
            for (; todo; --todo)
                if (!convert_q(now ? it : after))
                    return;
            const int fs = (unit + j) % FAC;
            if (!(tile_wait_warp(&sh.f_full[fs], ((unit + j) / FAC) & 1, limit, sh) &&
                  tile_wait_warp(&sh.r_full[r.slot], r.phase, limit, sh) &&
                  tile_wait_warp(&sh.v_empty[s.slot], s.phase ^ 1, limit, sh)))
                return;
            convert(tiles + C::R0 + r.slot * C::RAW, tiles + C::V0 + s.slot * C::TILE, sh.v_fac[fs],
                    it.left - j * AT_UNIT);
            async_fence();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&sh.v_full[s.slot]);
                mbar_arrive(&sh.r_empty[r.slot]);
                mbar_arrive(&sh.f_empty[fs]);
            }
            r.next(C::NR);
            s.next(C::NV);
        }
        unit += it.n;
        ready = early;
        it = after;
    }
}

template <int D, bool Q8>
__global__ void __launch_bounds__(TileCfg<D, Q8>::THREADS, 1)
    va_tiles(const __grid_constant__ CUtensorMap mq_pre, const __grid_constant__ CUtensorMap mq_own,
             const __grid_constant__ CUtensorMap m_pre, const __grid_constant__ CUtensorMap m_own,
             const __grid_constant__ TileParams P)
{
    using C = TileCfg<D, Q8>;
    // no static shared memory: the tiles start on a 1024-byte boundary, as their swizzle asks
    extern __shared__ __align__(1024) uint8_t tiles[];
    QuantShared &sh = *reinterpret_cast<QuantShared *>(tiles + C::TILES);   // the TileShared of it without 8-bit entries
    pdl_trigger();
    const int tid = threadIdx.x, warp = tid / 32;
    const uint32_t smem = saddr(tiles);
    // Polls, of about 0.1 us.  A spin limit below CL_PLAIN_POLLS reaches the softmax's first wait for
    // scores alone.
    const uint32_t limit = P.spin_limit > OWN_WAIT_MIN ? P.spin_limit : OWN_WAIT_MIN;

    // ---- where this CTA's length begins: sums over runs of sequences, then the run.  Units in the
    // low word, sequences that have any in the high one.
    typedef unsigned long long u64;
    const int B = P.A.B, run = (B + C::THREADS - 1) / C::THREADS;
    u64 sum = 0;
    for (int b = tid * run; b < min(B, (tid + 1) * run); ++b) {
        const int u = seq_units(P.A, b);
        sum += (u64)u | (u64)(u > 0) << 32;
    }
    u64 upto = sum;   // inclusive scan in the warp
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 y = __shfl_up_sync(0xffffffffu, upto, o);
        upto += tid % 32 >= o ? y : 0;
    }
    if (tid % 32 == 31)
        sh.sums[warp] = upto;
    if (tid == 0) {
        sh.abort = 0;
        for (int k = 0; k < 2; ++k) {
            mbar_init(&sh.q_full[k], 1);
            mbar_init(&sh.q_empty[k], Q8 ? 2 : 1);   // the tensor cores, and the softmax warps' last use
            mbar_init(&sh.q_ready[k], 4);
            mbar_init(&sh.s_full[k], 1);
            mbar_init(&sh.p_ready[k], 4);
            mbar_init(&sh.o_full[k], 1);
        }
        for (int k = 0; k < C::NK; ++k) {
            mbar_init(&sh.k_full[k], 1);
            mbar_init(&sh.k_empty[k], 1);
        }
        for (int k = 0; k < C::NV; ++k) {
            mbar_init(&sh.v_full[k], Q8 ? 4 : 1);
            mbar_init(&sh.v_empty[k], 1);
        }
        for (int k = 0; k < C::NR; ++k) {
            mbar_init(&sh.r_full[k], 1);
            mbar_init(&sh.r_empty[k], 4);
        }
        for (int k = 0; k < FAC; ++k) {
            mbar_init(&sh.f_full[k], 1);
            mbar_init(&sh.f_empty[k], 12);   // eight of the softmax warps, four of the converting ones
        }
        mbar_init(&sh.drain, 1);
        asm volatile("fence.mbarrier_init.release.cluster;\n\tfence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == W_MMA) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(saddr(&sh.tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_before();
    __syncthreads();
    tc_after();
    {
        u64 before = 0, total = 0;
#pragma unroll 1
        for (int k = 0; k < C::THREADS / 32; ++k) {
            before += k < warp ? sh.sums[k] : 0;
            total += sh.sums[k];
        }
        const int HS = P.A.H * P.W.own.tiles;
        const AttnLine line(P.W.pre, P.W.own, P.W.ppairs, P.W.pu, HS, (int)total, (int)(total >> 32), gridDim.x);
        const int from = line.start(blockIdx.x), to = line.start(blockIdx.x + 1);
        if (tid == 0 && from < line.own) {
            const int one = line.pre.pair(P.W.pu), p = from / one;
            sh.start = Place{from, to, p * one, -1, p / P.W.pre.tiles, p % P.W.pre.tiles, line.pre, line.own_cost};
        } else if (tid == 0 && from == to) {
            sh.start = Place{from, to, to, B, 0, 0, line.pre, line.own_cost};   // nothing here
        }
        u64 at = before + upto - sum;   // of the sequences before this thread's run
#pragma unroll 1
        for (int b = tid * run; b < min(B, (tid + 1) * run); ++b) {
            const int u = seq_units(P.A, b);
            if (blockIdx.x == 0 && P.W.base)
                P.W.base[b] = make_int2((int)at, (int)(at >> 32));
            const int lo = line.own + HS * line.sequences((int)at, (int)(at >> 32)), one = line.own_cost.pair(u);
            if (from < to && from >= lo && from < lo + one * HS) {
                const int p = (from - lo) / one;
                sh.start = Place{from, to, lo + p * one, b, p / P.W.own.tiles, p % P.W.own.tiles, line.pre, line.own_cost};
            }
            at += (u64)u | (u64)(u > 0) << 32;
        }
        if (blockIdx.x == 0 && tid == 0)
            *P.W.line = line;
    }
    __syncthreads();

    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::REGS_SOFT));
        softmax_role<D, Q8>(P, sh, tiles, warp / 4, limit);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REGS_REST));
        if (warp == W_LOAD) {
            if (elect_one())
                load_role<D, Q8>(P, &mq_pre, &mq_own, &m_pre, &m_own, sh, smem, limit);
        } else if (warp == W_MMA) {
            if (!Q8 || elect_one())
                mma_role<D, Q8>(P, sh, tiles, smem, limit);
        } else if (Q8 && warp == W_SCALE) {
            scale_role<D>(P, sh, limit);
        } else if (Q8 && warp >= W_CVT) {
            convert_role<D>(P, sh, tiles, limit);
        }
    }
    __syncwarp();
    tc_before();
    __syncthreads();
    if (sh.abort)
        wind_down<D, Q8>(sh, warp, limit);
    tc_after();
    if (warp == W_MMA)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(sh.tmem) : "memory");
    if (tid == 0)
        P.W.stat[blockIdx.x] = sh.abort ? (int)ST_TIMEOUT : 0;
    pdl_wait();   // behind another launch of this kernel: whoever waits for this one waits for both
}

// ------------------------------------------------------------------ host
using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                 const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled()
{
    static const EncodeTiled fn = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) !=
                cudaSuccess ||
            r != cudaDriverEntryPointSuccess)
            return (EncodeTiled) nullptr;
        return (EncodeTiled)f;
    }();
    return fn;
}

// A map over a row-major array of `rank` dimensions (innermost first); boxes
// of bfloat16 are 64 wide, boxes of codes a whole head: rows of 128 bytes, or of
// 64, swizzled as the tensor cores read them.
bool make_map(CUtensorMap *map, bool codes, const void *base, int rank, const cuuint64_t *dim, const cuuint32_t *box)
{
    cuuint64_t stride[4];
    cuuint64_t bytes = codes ? 1 : 2;
    for (int k = 0; k + 1 < rank; ++k) {
        bytes *= dim[k];
        stride[k] = bytes;
    }
    const cuuint32_t one[5] = {1, 1, 1, 1, 1};
    return encode_tiled()(map, codes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank,
                          const_cast<void *>(base), dim, stride, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          codes && box[0] < 128 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool Q8>
cudaError_t launch_tiles(const TileParams &P, int grid, bool second, cudaStream_t stream)
{
    using C = TileCfg<D, Q8>;
    if (!encode_tiled())
        return cudaErrorNotSupported;
    const AttnParams &A = P.A;
    CUtensorMap mq_pre, mq_own, m_pre, m_own;
    // q as [token row][Hkv][G][D]
    const cuuint64_t dq[4] = {D, (cuuint64_t)A.G, (cuuint64_t)A.H, (cuuint64_t)A.B * A.T};
    const cuuint32_t bp[4] = {64, (cuuint32_t)A.G, 1, (cuuint32_t)P.W.pre.tq};
    const cuuint32_t bo[4] = {64, (cuuint32_t)A.G, 1, (cuuint32_t)P.W.own.tq};
    const cuuint32_t wide = Q8 ? D : 64;
    const cuuint64_t dp[4] = {D, (cuuint64_t)A.H, 2, (cuuint64_t)A.P};
    const cuuint64_t dc[5] = {D, (cuuint64_t)A.H, 2, (cuuint64_t)A.L, (cuuint64_t)A.B};
    const cuuint32_t box[5] = {wide, 1, 1, AT_UNIT, 1};
    if ((A.P > 0 && (!make_map(&mq_pre, false, A.q, 4, dq, bp) || !make_map(&m_pre, Q8, A.prefix, 4, dp, box))) ||
        (A.L > 0 && (!make_map(&mq_own, false, A.q, 4, dq, bo) || !make_map(&m_own, Q8, A.cache, 5, dc, box))))
        return cudaErrorInvalidValue;
    // an absent prefix or cache has no units: its maps are never used
    if (A.P == 0)
        mq_pre = mq_own, m_pre = m_own;
    if (A.L == 0)
        mq_own = mq_pre, m_own = m_pre;
    // the shared memory a launch may ask for, raised once per device
    static std::atomic<uint64_t> raised{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(raised.load(std::memory_order_relaxed) & bit)) {
        e = cudaFuncSetAttribute(va_tiles<D, Q8>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)tile_smem<D, Q8>());
        if (e != cudaSuccess)
            return e;
        raised.fetch_or(bit, std::memory_order_relaxed);
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = tile_smem<D, Q8>();
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = second ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, va_tiles<D, Q8>, mq_pre, mq_own, m_pre, m_own, P);
}

}  // namespace

// `second`: behind the launch for the prefix, as whose CTAs finish it may begin
// (it needs nothing of it).
cudaError_t launch_attn_tiles(const AttnParams &A, const AttnWork &W, bool quant, int grid, bool second,
                              uint32_t spin_limit, cudaStream_t stream)
{
    TileParams P{A, W, spin_limit};
    if (A.D == 128)
        return quant ? launch_tiles<128, true>(P, grid, second, stream) : launch_tiles<128, false>(P, grid, second, stream);
    return quant ? launch_tiles<64, true>(P, grid, second, stream) : launch_tiles<64, false>(P, grid, second, stream);
}

}  // namespace sv
