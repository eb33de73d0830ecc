// fa_paged.cuh -- attention of a few new rows over the paged key/value cache, split over the
// cache's length and joined (sm_103a): the kernels of fa_paged_sm103.cu (all entries) and
// fa_paged_range_sm103.cu (RANGED: a window with sinks, or the entries from a given one on).
//
// Formulas, per sequence, KV head and query row r of its head group: s_j = c q_r . k_j over the
// row's slots j, m = max s, p_j = e^{s_j - m} / l with l = sum e^{s_j - m}, o = sum p_j v_j,
// lse = m + ln l; with accumulate, weight_j += sum_r p_j.  Everything below is in log2 units.
//
// What bounds it: K and V are read once, 4 d bytes an entry in bf16, and M = Hq / Hkv * Tq rows use
// them: M flops a byte, far below the device's ratio for M up to 64.  So the design is about
// keeping loads in flight and spreading them evenly:
//   * The batch's tiles of 64 or 128 entries (all sequences and KV heads in a row) are cut into equal
//     shares, one per CTA, whatever the lengths: a share begins and ends anywhere, so at most its
//     first and last unit (a sequence's KV head) are partial, and a partial state (m, l,
//     sum e^{s - m} v) goes to one of the CTA's two workspace slots.  A second kernel joins the slots
//     of each unit in order (the same bits on every run).  Short tables, and batches whose units are
//     as even as shares would be, are taken a unit a CTA, and nothing is left to join.
//   * One warp fills a ring of tiles by TMA, a box per page (all 128-byte column chunks of its
//     rows at once, swizzled); page numbers are read one tile ahead.
//   * Four warps compute with m16n8k16 products out of registers (ldmatrix): a warp owns up to 16 query
//     rows and a quarter, half or all of a tile's entries (1, 2 or 4 row tiles).  Up to 8 rows the
//     operands change places, K and V^T being the 16 rows and the queries the 8 columns: half the
//     products and half the accumulators do, which e4m3 needs most, two entries of which come with the bytes of
//     one (16 sequences of 1001 to 65536, d 64 55.5 -> 53.6 us; 160 units of 2048 to 4096, d 256 65 -> 52).
//     The tensor cores of the fifth generation want 128 rows a product: with up to 16 rows, the usual
//     case, they would run nearly empty, and their accumulators would have to come back for the
//     softmax, where the warp-level products leave S in the registers that P V takes.  At 64 rows
//     the bound are the math warps, two a scheduler, with the product pipe 46 % busy (see below).
//   * P enters its product as two bf16 numbers (its leading 8 bits and the rest), so its error is
//     2^-17 and not 2^-9, which would be as large as the output's own rounding.  e4m3 codes become
//     f16 exactly; there P is scaled by 2^15, which keeps probabilities down to 2^-29 in f16's normal
//     range, with 11 bits, and a row of q by the power of two that puts its largest value next to
//     f16's end: bf16's 8 bits are exact down to 2^-31 of that value.
//
// Measured: 8 sequences of 32768 entries, 32 KV heads, d 128 (4.3 GB) 598 us, 7.2 TB/s; 64 sequences of 200 to
// 8000, 8 KV heads (1.1 GB) 164 us, 6.6 TB/s; 17 entries of one sequence 3.7 us.  Of the second, 3 us pass
// before the first load, 3 to 4 with the join, and the CTAs end within 10 % of one another, with the
// issue slots a fifth busy.  By rows (160 units of 2048 to 4096, d 128): 46, 47, 52, 62 and 103 us
// with 4, 8, 16, 32 and 64; e4m3, twice as long: 48, 50, 55, 87 and 159, its codes being converted by
// every row tile.
#pragma once

#include <algorithm>
#include <cfloat>
#include <climits>

#include <cuda_fp16.h>

#include "fa_common.cuh"
#include "fa_internal.h"
#include "fa_pdl.cuh"

namespace fa {
namespace {

// Device status words of the file's kernels: [0] a wait that ran out, [1] an index out of range.  Two, because
// indexes are checked first, and a timeout, after which nothing of the call is valid, must not be lost to one.
__device__ int g_paged_status[2];

constexpr int kStatusBadIndex = 5;
constexpr int kMathWarps = 4;
constexpr int kThreads = 32 * (kMathWarps + 1);
constexpr int kSMs = 152;        // the grid is made for the GB300's; results depend on it, not on the device
constexpr int kMaxRows = 64;     // query rows of a head group that one CTA takes at a time
constexpr float kPShift = 15.f;  // e4m3: probabilities are scaled by 2^15

enum PagedSite : int { SITE_PAGED_FULL = 1, SITE_PAGED_EMPTY = 2 };

// ROWS: query rows of a CTA.  With 16 and more a warp's products have 16 query rows and 8 entries (or
// features); with 8 they are turned round (TURNED): 16 entries, or features, and 8 query rows, half as many.
template <int D, bool FP8, int ROWS>
struct Cfg {
    static constexpr bool TURNED = ROWS == 8;
    static constexpr int RT = TURNED ? 1 : ROWS / 16;              // row tiles
    static constexpr int ELEM = FP8 ? 1 : 2;
    static constexpr int ROWB = D * ELEM;                          // bytes of an entry's K or V row
    static constexpr int CB = ROWB < 128 ? ROWB : 128;             // bytes of a column chunk
    static constexpr int KT = ROWB <= 128 ? 128 : 64;              // entries a tile
    static constexpr int TILE = KT * ROWB;                         // K or V of a tile
    static constexpr int STAGE = 2 * TILE;
    static constexpr int GW = KT / 16 * RT / kMathWarps;           // groups of 16 entries a warp has of a tile
    static constexpr int GP = GW % 2 == 0 && D <= 128 ? 2 : 1;     // groups it takes at once
    static constexpr int QPITCH = D * 2 + 16;                      // bytes of a query row in shared memory
    static constexpr int MR = 512 / D;                             // rows of a row tile merged at a time
    static constexpr int OPITCH = D + 4;                           // floats of a merge row
    static constexpr int NQ = ROWS * QPITCH, NO = RT < kMathWarps ? kMathWarps * MR * OPITCH * 4 : 0, NML = kMathWarps * 16 * 8;
    static constexpr int SMALL = 1024 + NQ + NO + NML + RT * 16 * 4 + 24 * 12 + 64;
    // as many CTAs an SM as the accumulators leave registers for and the ring has room; the
    // ring takes what is left
    static constexpr int CTAS = D == 256 ? 1 : FP8 && D == 64 && RT == 1 ? 3 : 2;
    static constexpr int FIT = ((CTAS == 3 ? 75 : CTAS == 2 ? 113 : 227) * 1024 - SMALL) / STAGE;
    static constexpr int NST = FIT < 12 ? FIT : 12;
    static_assert(NST >= 2, "shared memory");
    // Stages in use where every SM has its CTAs: with 64 KB a CTA under way the memory is busy, and
    // more only queues (64 sequences, d 128 and 64: 164.9 and 164.4 us with two stages, 167.5 and 170.7
    // with three); where the products take longer the third hides them (e4m3 d 128: 101 against 107).
    static constexpr int DEPTH = !FP8 && D <= 128 && RT == 1 ? 2 : NST;
    static constexpr int OFF_Q = NST * STAGE;
    static constexpr int OFF_O = OFF_Q + NQ;
    static constexpr int OFF_ML = OFF_O + NO;
    static constexpr int OFF_RS = OFF_ML + NML;                    // scale of each row's scores
    static constexpr int OFF_BAR = OFF_RS + RT * 16 * 4;           // full[NST], empty[NST]
    static constexpr int OFF_OK = OFF_BAR + 16 * NST;              // per stage: which 16-entry groups are there
    static constexpr int OFF_MISC = (OFF_OK + 4 * NST + 15) / 16 * 16;   // abort flag
    static constexpr int SMEM = OFF_MISC + 16 + 1024;
    static_assert(SMEM <= 227 * 1024, "shared memory");
};

struct PagedArgs {
    const __nv_bfloat16 *q;
    __nv_bfloat16 *o;
    float *lse, *weight;
    const float *ks, *vs;
    const int *block_table, *lens;
    const int *first_pages;   // not RANGED: every sequence's first n_first pages, in place of the table's
    float *part;     // [2 grid][rows][D] then m, l [rows]
    long long *where;   // [0] the share, [1 + b] the first tile of sequence b (not of an empty one)
    float *scores;   // [sequence][KV head][row][cap]
    int B, Hq, Hkv, G, Tq, M, rows, RB, causal, num_pages, max_pages, ps_shift, cap, grid, whole, may_whole, kt;
    int n_first;
    // RANGED.  left >= 0: row t, at position p = lens - Tq + t, sees slots from p - left, and those below
    // sinks.  left < 0: slots from base.
    int left, sinks, base, span;   // span: slots that a unit sees, at most
    float *o32;   // RANGED: o goes here in fp32, or null
    int withhold;   // test builds: the arrive that is left out
    float scale_log2;
    uint64_t timeout_ns;
};

// ------------------------------------------------------------------ instructions
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
template <bool HALF>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if constexpr (HALF)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                     "{%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                     "{%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// An 8 x 8 block of 16-bit values, two of a row a lane, turned round.
__device__ __forceinline__ uint32_t turn8x8(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
// Two e4m3 codes (in the low or high half of x) as two f16.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t x)
{
    uint32_t y;
    asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi)
{
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
// Bytes that a phase waits for, without the arrive (test builds).
__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ uint64_t policy_evict_normal()
{
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
    return p;
}
__device__ __forceinline__ void st_shared_zero16(uint32_t addr)
{
    asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(addr), "r"(0) : "memory");
}
__device__ __forceinline__ void math_sync()   // the math warps meet, each one whole
{
    __syncwarp();
    asm volatile("bar.sync 1, %0;" ::"n"(32 * kMathWarps) : "memory");
}
__device__ __forceinline__ float quad_max(float x)
{
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
    return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
}

// The product of three positive factors, the largest and the smallest first, so that no part of it
// leaves fp32's range where the whole does not.  What is too small becomes the smallest normal number: a
// factor of 0 would make a NaN of a masked entry's -inf, and 2^32 times it is still nothing as a score.  In
// the same way what is too large stays finite, for sums of 0.  A NaN of b, the cache's scale, stays one (the
// minima and maxima drop it).
__device__ __forceinline__ float score_scale(float a, float b, float c)
{
    const float hi = fmaxf(a, b), lo = fminf(a, b);
    const float x = fmaxf(hi, c) * fminf(lo, c) * fmaxf(lo, fminf(hi, c));
    return isnan(b) ? b : fminf(fmaxf(x, FLT_MIN), FLT_MAX);
}

// ------------------------------------------------------------------ shares
__device__ __forceinline__ int length_in_range(const PagedArgs &a, int len)
{
    if (len < 0 || len > a.cap) {
        atomicCAS(&g_paged_status[1], 0, kStatusBadIndex);
        return 0;
    }
    return len;
}
__device__ __forceinline__ int length_of(const PagedArgs &a, int b) { return length_in_range(a, a.lens[b]); }

// RANGED: the slots of a sequence of len entries that any row sees are those below sinks and those from `from`
// to len - 1.  Its tiles are numbered without those between: the sinks' first, then the others.
struct Visible {
    int from, sinks;
    int ns, skip;   // tiles of the sinks in front of the window's, and tiles left out behind them
    int nt;
};
__device__ __forceinline__ Visible visible_of(const PagedArgs &a, int len)
{
    Visible v;
    v.from = a.left >= 0 ? max(0, len - a.Tq - a.left) : min(a.base, len);
    v.sinks = min(a.sinks, len);
    const int first = v.from / a.kt;
    v.ns = min((v.sinks + a.kt - 1) / a.kt, first);
    v.skip = first - v.ns;
    v.nt = v.ns + (v.from < len ? (len + a.kt - 1) / a.kt - first : 0);
    return v;
}
template <bool RANGED>
__device__ __forceinline__ int tiles_in(const PagedArgs &a, int len)
{
    if constexpr (RANGED)
        return visible_of(a, len).nt;
    else
        return (len + a.kt - 1) / a.kt;
}
template <bool RANGED>
__device__ __forceinline__ int tiles_of(const PagedArgs &a, int b)
{
    return tiles_in<RANGED>(a, length_of(a, b));
}

// The sequence of up to 64 that comes `rank`-th by its tiles, most first and equal ones in order: lane i has the tiles
// of sequences i and 32 + i, x and y; `most` is the largest.
__device__ __forceinline__ int longest_first(int rank, int n, int x, int y, int most)
{
    const int lane = (int)lane_id();
    x = lane < n ? x : -1;
    y = 32 + lane < n ? y : -1;
    int lo = 0, hi = most;   // the tiles of the one sought: the largest t that more than `rank` sequences reach
    while (lo < hi) {
        const int t = (lo + hi + 1) >> 1;
        if (__popc(__ballot_sync(0xffffffffu, x >= t)) + __popc(__ballot_sync(0xffffffffu, y >= t)) > rank)
            lo = t;
        else
            hi = t - 1;
    }
    rank -= __popc(__ballot_sync(0xffffffffu, x > lo)) + __popc(__ballot_sync(0xffffffffu, y > lo));
    const uint32_t ex = __ballot_sync(0xffffffffu, x == lo), ey = __ballot_sync(0xffffffffu, y == lo);
    const int nx = __popc(ex);
    return rank < nx ? __fns(ex, 0, rank + 1) : 32 + __fns(ey, 0, rank - nx + 1);
}

// Tiles a CTA takes of the batch's `total`: equal shares, but at least 128 entries, below which
// the joining costs more than they do.
template <typename I>
__device__ __forceinline__ I share_of(const PagedArgs &a, I total)
{
    const I c = (total + a.grid - 1) / a.grid;
    const int least = a.kt < 128 ? 128 / a.kt : 1;
    return c < least ? least : c;
}

// A CTA's place in the batch's tiles: sequence b, unit ul (row block, KV head) in it, tile.
struct Place {
    int b, ul, tile, nt;
    long long left;   // tiles still to do
};

__device__ __forceinline__ long long warp_scan(long long x)   // sum over the lanes up to this one
{
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, off);
        if ((int)lane_id() >= off)
            x += y;
    }
    return x;
}

// Finds the CTA's place; p.left: its tiles, 0 if there is nothing for it.  Every warp does it for
// itself: the loads of the others are in the same cache lines, and a block-wide sum would cost
// barriers at a time when nothing is under way.
// whole: every unit is one CTA's, because there are enough CTAs and the longest unit is at most a
// quarter, or 7 tiles (4 with three CTAs an SM, where one by itself gains less), longer than an equal share,
// and not twice as long: a CTA whose neighbours have ended gets more
// of the bandwidth, and there are no second units to start and nothing to join.  us whole and in shares, by
// tiles of the longest unit / of a share: 296 units, d 128, 16/9 21.8 and 29.9, 18/16 29.6 and 32.4, 27/17 33.6 and
// 33.4, 63/33 63.8 and 57.9; 256 units, 64/54 82.9 and 87.5; 120 units, 18/7 20.7 and 18.0; 8 units, 4/2 7.6
// and 7.9, 6/2 9.0 and 8.0; e4m3, 296 units, 9/9 19.8 and 25.0, 200 units, 12/6 21.5 and 20.2; 144 units, d 256,
// 21/16 30.8 and 31.6, 63/46 77.8 and 72.3; 240 units, e4m3 d 64, 16/9 27.2 and 22.8, 296 units, 9/6 18.2 and 19.5.
template <bool RANGED>
__device__ __forceinline__ Place place_of(const PagedArgs &a, long long &share, long long &t0, bool &whole)
{
    const int per = a.Hkv * a.RB, lane = (int)lane_id();
    const int nt0 = lane < a.B ? tiles_of<RANGED>(a, lane) : 0;
    const long long inc0 = warp_scan((long long)nt0 * per);
    long long total = __shfl_sync(0xffffffffu, inc0, 31);
    int longest = nt0;
    if (a.B > 32) {
        long long x = 0;
#pragma unroll 4
        for (int b = 32 + lane; b < a.B; b += 32) {
            const int nt = tiles_of<RANGED>(a, b);
            x += nt;
            longest = max(longest, nt);
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1)
            x += __shfl_xor_sync(0xffffffffu, x, off);
        total += x * per;
    }
    longest = __reduce_max_sync(0xffffffffu, longest);
    share = total < INT_MAX ? share_of(a, (int)total) : share_of(a, total);
    Place p{a.B, 0, 0, 0, 0};
    const long long more = max(share >> 2, a.grid > 2 * kSMs ? 4ll : 7ll), most = (share * 13 >> 4) + 1;
    if (a.may_whole && longest <= share + min(more, most)) {
        whole = true;
        if ((int)blockIdx.x < a.B * per) {
            p.b = (int)blockIdx.x / per;
            p.ul = (int)blockIdx.x - p.b * per;
            // Not all start at once: the longest first, unless most are about as long.  us in order of length and of the
            // batch, 8 KV heads of 128: 64 sequences of 20 to 700 entries 25.8 and 28.0, 48 of 10 to 3000 under a window
            // of 1501 43.1 and 49.9, 64 of 100 to 2000 under one of 701 39.4 and 37.5.  More sequences, two units for every
            // place, do not gain (ranks for up to 128: 76 of 20 to 700 31.9 and 30.7, 70 of 10 to 3000 64.6 and 62.1), and four
            // lengths a lane cost the others 1 us
            if (RANGED && a.B <= 64 && a.B * per > a.grid && 5 * total < 4ll * longest * a.B * per)
                p.b = longest_first(p.b, a.B, nt0, 32 + lane < a.B ? tiles_of<RANGED>(a, 32 + lane) : 0, longest);
            p.left = p.nt = tiles_of<RANGED>(a, p.b);
        }
        return p;
    }
    t0 = share * blockIdx.x;
    if (t0 >= total)
        return p;
    p.left = min(share, total - t0);
    long long base = 0, inc = inc0;
    int nt = nt0;
    for (int b0 = 0; b0 < a.B; b0 += 32) {
        if (b0 > 0) {
            nt = b0 + lane < a.B ? tiles_of<RANGED>(a, b0 + lane) : 0;
            inc = warp_scan((long long)nt * per);
        }
        const uint32_t past = __ballot_sync(0xffffffffu, base + inc > t0);
        if (past) {
            const int src = __ffs(past) - 1;
            const long long end = base + __shfl_sync(0xffffffffu, inc, src);
            p.nt = __shfl_sync(0xffffffffu, nt, src);
            p.b = b0 + src;
            const long long in = t0 - (end - (long long)p.nt * per);
            p.ul = in < INT_MAX ? (int)in / p.nt : (int)(in / p.nt);
            p.tile = (int)(in - (long long)p.ul * p.nt);
            return p;
        }
        base += __shfl_sync(0xffffffffu, inc, 31);
    }
    p.left = 0;   // lengths that change under the call: nothing out of range is read
    return p;
}

// Tiles of the current unit that belong to this CTA; and on to the next unit.
__device__ __forceinline__ int segment(const Place &p) { return (int)min((long long)(p.nt - p.tile), p.left); }
template <bool RANGED>
__device__ __forceinline__ void next_unit(const PagedArgs &a, Place &p, int done)
{
    p.left -= done;
    p.tile = 0;
    if (p.left > 0 && ++p.ul == a.Hkv * a.RB) {
        p.ul = 0;
        do {
            if (++p.b >= a.B) {
                p.left = 0;
                return;
            }
            p.nt = tiles_of<RANGED>(a, p.b);
        } while (p.nt == 0);
    }
}

// sum + the probabilities 2^{s - lse} of four neighbouring entries over nrows rows of stored scores
// (which reach to the end of the last group of 16 entries); `last`: adds them to the weights at
// `at`, of which `left` or more are entries.
__device__ __forceinline__ float4 add_weights(const PagedArgs &a, long long at, int left, const float *sp, int nrows,
                                              const float *row_lse, float4 sum, bool last)
{
#pragma unroll 4
    for (int r = 0; r < nrows; ++r) {
        const float4 s = *reinterpret_cast<const float4 *>(sp + (long long)r * a.cap);
        const float y = row_lse[r];
        sum.x += ex2_approx(s.x - y);
        sum.y += ex2_approx(s.y - y);
        sum.z += ex2_approx(s.z - y);
        sum.w += ex2_approx(s.w - y);
    }
    if (!last)
        return sum;
    float *w = a.weight + at;
    if (left >= 4) {
        float4 x = *reinterpret_cast<const float4 *>(w);
        x.x += sum.x, x.y += sum.y, x.z += sum.z, x.w += sum.w;
        *reinterpret_cast<float4 *>(w) = x;
    } else {
        w[0] += sum.x;
        if (left > 1)
            w[1] += sum.y;
        if (left > 2)
            w[2] += sum.z;
    }
    return sum;
}

// ------------------------------------------------------------------ attention
template <int D, bool FP8, int ROWS, bool RANGED>
__global__ void __launch_bounds__(kThreads, Cfg<D, FP8, ROWS>::CTAS)
    paged_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                 const __grid_constant__ PagedArgs a)
{
    using C = Cfg<D, FP8, ROWS>;
    constexpr bool TURNED = C::TURNED;
    constexpr int RT = C::RT;
    constexpr int KW = kMathWarps / RT;             // warps that share a row tile's entries
    constexpr int KSTEPS = D / 16;                  // products along the head width, per 8 entries
    constexpr bool QREG = TURNED || (D <= 64 && !(FP8 && RT == 1));   // query fragments stay in registers
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t sbase = (raw + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (sbase - raw);
    const uint32_t bar0 = sbase + C::OFF_BAR;
    volatile uint32_t *there = reinterpret_cast<volatile uint32_t *>(smem + C::OFF_OK);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::OFF_MISC);
    const int lane = (int)lane_id(), warp = (int)warp_id();
    const WaitCtx ctx{abort_flag, &g_paged_status[0], a.timeout_ns};
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::NST; ++s) {
            mbar_init(bar0 + 8u * s, 1);
            mbar_init(bar0 + 8u * (C::NST + s), kMathWarps);
        }
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
    }
    pdl_wait();
    Place p;
    long long share = 0, t0 = 0;
    bool whole = a.whole;
    if (whole) {   // one unit a CTA, however long
        const int per = a.Hkv * a.RB, b = (int)blockIdx.x / per;
        const int nt = tiles_of<RANGED>(a, b);
        p = Place{b, (int)blockIdx.x - b * per, 0, nt, nt};
    } else {
        p = place_of<RANGED>(a, share, t0, whole);
        if (threadIdx.x == 0 && blockIdx.x == 0)
            a.where[0] = whole ? 0 : share;
        if (p.left == 0 && !(whole && p.b < a.B))
            return;   // the whole CTA
    }
    const long long mine_all = p.left;   // tiles of this CTA
    // Stages in use.  Long whole units that run in step do better with fewer, unless their pages are small (256
    // units, d 128: 32768 entries 594 us with two and 605 with three, 16384 299 and 305, in pages of 16 305 and
    // 301; 4096 82.1 and 80.1)
    const uint32_t depth = whole && (a.ps_shift < 6 || p.nt < 256) ? C::NST : C::DEPTH;
    __syncthreads();   // the barriers are there
    // rows of a page in one box, and boxes of a tile
    const int bp_shift = a.ps_shift < 6 ? a.ps_shift : 6, boxes = C::KT >> bp_shift;

    if (warp == kMathWarps) {
        // ---------------------------------------------------------- loads: lane 2 i is K of box i, 2 i + 1 V
        const bool mine = lane < 2 * boxes;
        const CUtensorMap *map = (lane & 1) ? &tm_v : &tm_k;
        const int box = lane >> 1;
        const uint32_t dst = (uint32_t)((lane & 1) * C::TILE + (box << bp_shift) * C::ROWB);
        const uint32_t box_bytes = (uint32_t)(C::ROWB << bp_shift);
        // K and V are read once, unless several row blocks read them: they leave the L2 to what is written
        // and read again (e4m3 d 64 58.5 -> 57.1 us, with stored scores 30.3 -> 28.2)
        const uint64_t policy = a.RB == 1 ? policy_evict_first() : policy_evict_normal();
        uint32_t n = 0, st = 0, round = 0;   // tiles so far; the stage of the next one, and its round
        bool ok = true;
        while (ok && p.left > 0) {
            const int len = length_of(a, p.b), h = p.ul % a.Hkv, cnt = segment(p);
            const int *table = a.block_table + (long long)p.b * a.max_pages;
            const Visible vis = RANGED ? visible_of(a, len) : Visible{};
            auto slot_of = [&](int tile) {   // of this lane's box
                if constexpr (RANGED)
                    tile += tile < vis.ns ? 0 : vis.skip;
                return tile * C::KT + (box << bp_shift);
            };
            // whether any row sees one of n slots from `slot` on; pages that no row sees may have been given back
            auto seen = [&](int slot, int n) { return slot < len && (!RANGED || slot + n > vis.from || slot < vis.sinks); };
            auto page_at = [&](int tile) {   // -1: nothing there
                const int slot = slot_of(tile);
                if (!mine || !seen(slot, 1 << bp_shift))
                    return -1;
                const int i = slot >> a.ps_shift;
                return !RANGED && i < a.n_first ? a.first_pages[i] : table[i];
            };
            int page = page_at(p.tile);
            for (int i = 0; i < cnt; ++i, ++n) {
                const int tile = p.tile + i, slot = slot_of(tile);
                const int next = i + 1 < cnt ? page_at(tile + 1) : -1;
                // A math warp that has given up releases its stages unread, after raising the abort flag: such a
                // stage is not filled again, so that each full barrier's phase is that of its last fill
                if (round > 0 && (!mbar_wait_warp(bar0 + 8u * (C::NST + st), (round - 1) & 1u, ctx, SITE_PAGED_EMPTY) ||
                                  __any_sync(0xffffffffu, *abort_flag))) {
                    ok = false;
                    break;
                }
                const bool inside = mine && seen(slot, 1 << bp_shift), good = inside && page >= 0 && page < a.num_pages;
                if (inside && !good)
                    atomicCAS(&g_paged_status[1], 0, kStatusBadIndex);
                // groups of 16 entries whose page is there and that begin in front of the length
                uint32_t groups = 0;
                if (good && !(lane & 1))
                    for (int g = 0; g < (1 << bp_shift) / 16; ++g)
                        if (seen(slot + 16 * g, 16))
                            groups |= 1u << ((box << bp_shift) / 16 + g);
                groups = __reduce_or_sync(0xffffffffu, groups);
                const uint32_t loads = __popc(__ballot_sync(0xffffffffu, good));
                if (lane == 0) {
                    there[st] = groups;
#if FA_TEST_WITHHOLD
                    const bool hold = a.withhold == (RANGED ? WITHHOLD_RANGE_FULL : WITHHOLD_PAGED_FULL) && blockIdx.x == 0 && n == 0;
#else
                    constexpr bool hold = false;
#endif
                    if (hold)
                        mbar_expect_tx(bar0 + 8u * st, loads * box_bytes);
                    else
                        mbar_arrive_expect_tx(bar0 + 8u * st, loads * box_bytes);
                }
                __syncwarp();
                if (good)
                    tma_load_4d_hint(sbase + st * C::STAGE + dst, map, bar0 + 8u * st, 0, slot & ((1 << a.ps_shift) - 1), 0,
                                     page * a.Hkv + h, policy);
                page = next;
                if (++st == depth) {
                    st = 0;
                    ++round;
                }
            }
            if (ok)
                next_unit<RANGED>(a, p, cnt);
        }
        // Every copy lands before the CTA exits, whoever gave up: the math warps may have done so after the
        // last copy was issued
        for (uint32_t s = n < depth ? 0 : n - depth; s < n; ++s)
            mbar_wait_drain(bar0 + 8u * (s % depth), (s / depth) & 1u);
    } else {
        // ---------------------------------------------------------- math
        const int rt = warp % RT, kw = warp / RT, c4 = lane & 3, r0 = lane >> 2;
        // the rows' scales; once they are read, the place of the rows' lse
        const float *rs = reinterpret_cast<const float *>(smem + C::OFF_RS);
        float *row_lse = reinterpret_cast<float *>(smem + C::OFF_RS);
        float2 *ml = reinterpret_cast<float2 *>(smem + C::OFF_ML);
        float *ob = reinterpret_cast<float *>(smem + C::OFF_O);
        constexpr int GP = C::GP;
        // where a lane reads in a group's rows (ldmatrix): K in (entries, 16-byte units) order, V in
        // (units, entries) order; unit u of a row lies at u ^ its swizzle
        const int krow = (lane & 7) + ((lane >> 4) << 3), vrow = lane & 15;
        auto swizzle_of = [](int row) { return C::CB == 128 ? row & 7 : (row >> 1) & 3; };
        const uint32_t k_lane = (uint32_t)(krow * C::CB), k_unit = (uint32_t)((((lane >> 3) & 1) ^ swizzle_of(krow)) << 4);
        const uint32_t v_lane = (uint32_t)(vrow * C::CB), v_unit = (uint32_t)(((lane >> 4) ^ swizzle_of(vrow)) << 4);
        const uint32_t q_lane = sbase + C::OFF_Q + (rt * 16 + (lane & 15)) * C::QPITCH + (lane >> 4) * 16;
        // The unit's query rows: a warp's share of them into registers, from there to shared memory as
        // bf16, or as f16 over the row's power of two with features in the order in which the codes of
        // four neighbours come out of a register.
        constexpr int QROWS = ROWS / kMathWarps;
        uint32_t qw[QROWS][D / 64];
        float qks = 1.f;
        auto fetch_q = [&](const Place &at) {
            const int h = at.ul % a.Hkv, row0 = at.ul / a.Hkv * a.rows, nrows = min(a.rows, a.M - row0);
            const __nv_bfloat16 *q = a.q + (((long long)at.b * a.Hq + h * a.G) * a.Tq + row0) * D;
#pragma unroll
            for (int j = 0; j < QROWS; ++j) {
                const int r = warp + kMathWarps * j;
#pragma unroll
                for (int i = 0; i < D / 64; ++i)
                    qw[j][i] = r < nrows ? reinterpret_cast<const uint32_t *>(q + (long long)r * D)[i * 32 + lane] : 0u;
            }
            if constexpr (FP8)
                qks = a.ks[h];
        };
        auto put_q = [&]() {
#pragma unroll
            for (int j = 0; j < QROWS; ++j) {
                const int r = warp + kMathWarps * j;
                uint8_t *qr = smem + C::OFF_Q + r * C::QPITCH;
                float scale = a.scale_log2;
                if constexpr (FP8) {
                    float big = 0.f;
#pragma unroll
                    for (int i = 0; i < D / 64; ++i)
                        big = fmax3(big, fabsf(__uint_as_float(qw[j][i] << 16)), fabsf(__uint_as_float(qw[j][i] & 0xFFFF0000u)));
#pragma unroll
                    for (int off = 16; off > 0; off >>= 1)
                        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, off));
                    // a power of two, `down`, brings the row's largest value into [2^14, 2^15) (as far as 2^127
                    // does): what a bf16 value of 2^-31 of it or more holds stays whole, below that a multiple of
                    // 2^-38 of it; sums of d products with codes stay below 2^15 448 d < 2^32.  Zeros and
                    // infinities stay
                    const int x = (int)(__float_as_uint(big) >> 23), de = x == 255 || big == 0.f ? 127 : min(268 - x, 254);
                    const float down = __uint_as_float((uint32_t)de << 23);
                    scale = score_scale(scale, qks, 1.f / down);
#pragma unroll
                    for (int i = 0; i < D / 64; ++i) {
                        const int f = i * 64 + 2 * lane, c = (f & 15) >> 2;   // features f, f + 1
                        const int at = (f & ~15) + 2 * c + ((f & 2) ? 8 : 0);
                        reinterpret_cast<uint32_t *>(qr)[at / 2] =
                            pack_f16x2(__uint_as_float(qw[j][i] << 16) * down, __uint_as_float(qw[j][i] & 0xFFFF0000u) * down);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < D / 64; ++i)
                        reinterpret_cast<uint32_t *>(qr)[i * 32 + lane] = qw[j][i];
                }
                if (lane == 0)
                    reinterpret_cast<float *>(smem + C::OFF_RS)[r] = scale;
            }
        };
        uint32_t st = 0, round = 0;   // the next tile's stage, and its round
        bool ok = true;
        // All CTAs are there, and the join's blocks take nothing from them (0.2 to 0.4 us); where no join
        // follows, the next call's do (240 units of 512 14.1 us instead of 13.2)
        // (own entries behind a shared prefix: its kernel's CTAs take the SMs that are done, and wait there)
        if ((whole && !a.whole) || (RANGED && a.o32))
            pdl_launch();
        if (RT == 1 && p.left > 0)
            fetch_q(p);
        if (p.left == 0) {   // whole units: an empty sequence
            const int h = p.ul % a.Hkv, row0 = p.ul / a.Hkv * a.rows, nrows = min(a.rows, a.M - row0);
            const long long grow = ((long long)p.b * a.Hq + h * a.G) * a.Tq + row0;
            if (RANGED && a.o32) {
                for (int e = threadIdx.x; e < nrows * (D / 4); e += 32 * kMathWarps)
                    reinterpret_cast<float4 *>(a.o32 + grow * D)[e] = make_float4(0.f, 0.f, 0.f, 0.f);
            } else {
                for (int e = threadIdx.x; e < nrows * (D / 8); e += 32 * kMathWarps)
                    reinterpret_cast<uint4 *>(a.o + grow * D)[e] = make_uint4(0, 0, 0, 0);
            }
            for (int r = threadIdx.x; r < nrows; r += 32 * kMathWarps)
                a.lse[grow + r] = -INFINITY;
        }
        while (p.left > 0) {
            const int len = length_of(a, p.b), h = p.ul % a.Hkv, rb = p.ul / a.Hkv, cnt = segment(p);
            if (threadIdx.x == 0 && p.tile == 0 && p.ul == 0 && !whole)
                a.where[1 + p.b] = t0 + (mine_all - p.left);
            const int row0 = rb * a.rows, nrows = min(a.rows, a.M - row0);
            const long long grow = ((long long)p.b * a.Hq + h * a.G) * a.Tq + row0;   // first row of q and o
            if constexpr (RT > 1)
                fetch_q(p);
            put_q();
            math_sync();
            uint32_t qf[QREG ? (TURNED ? KSTEPS / 2 : KSTEPS) : 1][4];   // turned: of two steps
            if constexpr (TURNED) {
#pragma unroll
                for (int k = 0; k < KSTEPS / 2; ++k)
                    ldsm4(qf[k], sbase + C::OFF_Q + (lane & 7) * C::QPITCH + (lane >> 3) * 16 + k * 64);
            } else if constexpr (QREG) {
#pragma unroll
                for (int k = 0; k < KSTEPS; ++k)
                    ldsm4(qf[k], q_lane + k * 32);
            }
            // the thread's two rows, and the slots that they see; a row past the last sees what the others may
            const int la = TURNED ? 2 * c4 : rt * 16 + r0, lz = la + (TURNED ? 1 : 8), ra = row0 + la, rz = row0 + lz;
            const float sc0 = rs[la], sc1 = rs[lz];
            const int all = a.causal ? len - a.Tq + 1 : len;   // slots that every row sees
            const int lim0 = a.causal && ra < a.M ? len - a.Tq + ra % a.Tq + 1 : len;
            const int lim1 = a.causal && rz < a.M ? len - a.Tq + rz % a.Tq + 1 : len;
            // RANGED: the first slot that either row sees besides the sinks, the latest of those of all rows
            const Visible vis = RANGED ? visible_of(a, len) : Visible{};
            const int low0 = RANGED && a.left >= 0 && ra < a.M ? max(0, len - a.Tq + ra % a.Tq - a.left) : vis.from;
            const int low1 = RANGED && a.left >= 0 && rz < a.M ? max(0, len - a.Tq + rz % a.Tq - a.left) : vis.from;
            const int low = RANGED && a.left >= 0 ? max(0, len - 1 - a.left) : vis.from;
            const bool st0 = a.scores && la < nrows, st1 = a.scores && lz < nrows;
            float *sp = a.scores ? a.scores + (((long long)p.b * a.Hkv + h) * a.M + ra) * a.cap : nullptr;

            auto sees0 = [&](int key) { return key < lim0 && (!RANGED || key >= low0 || key < vis.sinks); };
            auto sees1 = [&](int key) { return key < lim1 && (!RANGED || key >= low1 || key < vis.sinks); };
            auto put_scores = [&](int key, float x, float y, float z, float w) {   // of 8 entries, both rows
                if constexpr (TURNED) {   // x, y: entry r0; z, w: entry r0 + 8
                    if (st0)
                        sp[key + r0] = x, sp[key + r0 + 8] = z;
                    if (st1)
                        sp[(long long)a.cap + key + r0] = y, sp[(long long)a.cap + key + r0 + 8] = w;
                    return;
                }
                if (st0)
                    *reinterpret_cast<float2 *>(sp + key + 2 * c4) = make_float2(x, y);
                if (st1)
                    *reinterpret_cast<float2 *>(sp + 8ll * a.cap + key + 2 * c4) = make_float2(z, w);
            };

            constexpr int OT = D / (TURNED ? 16 : 8);   // accumulators: of 16 or 8 features
            float o[OT][4];
#pragma unroll
            for (int i = 0; i < OT; ++i)
                o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
            float m0 = -INFINITY, m1 = -INFINITY, l0[2] = {0.f, 0.f}, l1[2] = {0.f, 0.f};

            for (int i = 0; i < cnt; ++i) {
                if (ok && !mbar_wait_warp(bar0 + 8u * st, round & 1u, ctx, SITE_PAGED_FULL))
                    ok = false;   // the CTA gives up: no more is computed or written, and its warps still meet
                const uint32_t groups = ok ? there[st] : 0u;
#pragma unroll 1
                for (int j = 0; j < C::GW; j += GP) {
                    const int tile = RANGED && p.tile + i >= vis.ns ? p.tile + i + vis.skip : p.tile + i;
                    const int g = kw * C::GW + j, key0 = tile * C::KT + g * 16;
                    const uint32_t have = (groups >> g) & ((1u << GP) - 1u);
                    if (have == 0) {
                        if (ok && a.scores)   // pages out of range: masked
                            for (int t = 0; t < 2 * GP && key0 + 8 * (t & ~1) < len; t += TURNED ? 2 : 1)
                                put_scores(key0 + 8 * t, -INFINITY, -INFINITY, -INFINITY, -INFINITY);
                        continue;
                    }
                    // a group's rows lie in one box: [chunk][row in box][CB bytes], swizzled
                    const uint32_t chunk = (uint32_t)(C::CB << bp_shift);
                    uint32_t base[GP];
#pragma unroll
                    for (int u = 0; u < GP; ++u) {
                        const int at = (g + u) * 16;
                        base[u] = sbase + st * C::STAGE + (uint32_t)((at >> bp_shift << bp_shift) * C::ROWB +
                                                                     (at & ((1 << bp_shift) - 1)) * C::CB);
                    }
                    const bool clear = have == (1u << GP) - 1u && key0 + 16 * GP <= all &&
                                       (!RANGED || key0 >= low || key0 + 16 * GP <= vis.sinks);
                    // Entries behind the length (and groups that are not there) hold anything, and 0 times a
                    // NaN is one: their V rows become 0 before P V
                    auto zero_behind = [&]() {
                        if (clear)
                            return;
#pragma unroll
                        for (int u = 0; u < GP; ++u) {
                            const int first = (have >> u) & 1u ? len - (key0 + 16 * u) : 0, row = lane & 15;
                            const int slot = key0 + 16 * u + row;   // RANGED: nor do rows in front of the window matter
                            if (row >= first || (RANGED && slot < vis.from && slot >= vis.sinks))
                                for (int x = lane >> 4; x < C::ROWB / 16; x += 2)
                                    st_shared_zero16(base[u] + C::TILE + row * C::CB + (x / (C::CB / 16)) * chunk +
                                                     (x % (C::CB / 16)) * 16);
                        }
                        // written through the generic proxy, and next by TMA
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        __syncwarp();
                    };
                    if constexpr (TURNED) {
                        // ---- S^T = K Q^T: 16 entries x 8 rows a group, in two accumulators
                        float s[GP][2][4];
#pragma unroll
                        for (int u = 0; u < GP; ++u)
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                s[u][0][x] = s[u][1][x] = 0.f;
#pragma unroll
                        for (int k = 0; k < KSTEPS; k += 2) {
                            const uint32_t(&qk)[4] = qf[k / 2];
#pragma unroll
                            for (int u = 0; u < GP; ++u) {
                                uint32_t kf[4];
                                if constexpr (!FP8) {   // a 16-byte unit is 8 features
#pragma unroll
                                    for (int w = 0; w < 2; ++w) {
                                        const int kk = k + w;
                                        ldsm4(kf, base[u] + k_lane + (kk / (C::CB / 32)) * chunk + (k_unit ^ ((kk % (C::CB / 32)) << 5)));
                                        mma16816<false>(s[u][w], {kf[0], kf[2], kf[1], kf[3]}, qk[2 * w], qk[2 * w + 1]);
                                    }
                                } else {   // 16 features
                                    ldsm4(kf, base[u] + k_lane + (k / (C::CB / 16)) * chunk + (k_unit ^ ((k % (C::CB / 16)) << 4)));
                                    mma16816<true>(s[u][0], {e4m3x2_to_f16x2(kf[0]), e4m3x2_to_f16x2(kf[2]),
                                                             e4m3x2_to_f16x2(kf[0] >> 16), e4m3x2_to_f16x2(kf[2] >> 16)}, qk[0], qk[1]);
                                    mma16816<true>(s[u][1], {e4m3x2_to_f16x2(kf[1]), e4m3x2_to_f16x2(kf[3]),
                                                             e4m3x2_to_f16x2(kf[1] >> 16), e4m3x2_to_f16x2(kf[3] >> 16)}, qk[2], qk[3]);
                                }
                            }
                        }
                        // t: (entry, first row), (entry, second), (entry + 8, first), (entry + 8, second)
                        float t[GP][4];
#pragma unroll
                        for (int u = 0; u < GP; ++u) {
                            fadd2(t[u][0], t[u][1], s[u][0][0], s[u][0][1], s[u][1][0], s[u][1][1]);
                            fadd2(t[u][2], t[u][3], s[u][0][2], s[u][0][3], s[u][1][2], s[u][1][3]);
                        }
                        if (!clear) {
#pragma unroll
                            for (int u = 0; u < GP; ++u) {
                                const bool in = (have >> u) & 1u;
                                const int key = key0 + 16 * u + r0;
                                t[u][0] = in && sees0(key) ? t[u][0] : -INFINITY;
                                t[u][1] = in && sees1(key) ? t[u][1] : -INFINITY;
                                t[u][2] = in && sees0(key + 8) ? t[u][2] : -INFINITY;
                                t[u][3] = in && sees1(key + 8) ? t[u][3] : -INFINITY;
                            }
                        }
                        if (a.scores) {
#pragma unroll
                            for (int u = 0; u < GP; ++u)
                                if (key0 + 16 * u < len)
                                    put_scores(key0 + 16 * u, t[u][0] * sc0, t[u][1] * sc1, t[u][2] * sc0, t[u][3] * sc1);
                        }
                        // ---- online softmax; the rows' maxima are put together only when one of them grows
                        constexpr float SH = FP8 ? kPShift : 0.f;
                        float x0 = fmaxf(t[0][0], t[0][2]), x1 = fmaxf(t[0][1], t[0][3]);
                        if constexpr (GP == 2) {
                            x0 = fmax3(x0, t[1][0], t[1][2]);
                            x1 = fmax3(x1, t[1][1], t[1][3]);
                        }
                        float n0 = x0 * sc0 - SH, n1 = x1 * sc1 - SH;
                        if (__any_sync(0xffffffffu, n0 > m0 || n1 > m1)) {
#pragma unroll
                            for (int off = 4; off < 32; off <<= 1) {
                                n0 = fmaxf(n0, __shfl_xor_sync(0xffffffffu, n0, off));
                                n1 = fmaxf(n1, __shfl_xor_sync(0xffffffffu, n1, off));
                            }
                            n0 = fmaxf(n0, m0);
                            n1 = fmaxf(n1, m1);
                            const float f0 = ex2_approx(m0 - (n0 == -INFINITY ? 0.f : n0));
                            const float f1 = ex2_approx(m1 - (n1 == -INFINITY ? 0.f : n1));
                            l0[0] *= f0;
                            l1[0] *= f1;
#pragma unroll
                            for (int d = 0; d < OT; ++d) {
                                o[d][0] *= f0;
                                o[d][1] *= f1;
                                o[d][2] *= f0;
                                o[d][3] *= f1;
                            }
                            m0 = n0;
                            m1 = n1;
                        }
                        const float b0 = m0 == -INFINITY ? 0.f : m0, b1 = m1 == -INFINITY ? 0.f : m1;
#pragma unroll
                        for (int u = 0; u < GP; ++u)
#pragma unroll
                            for (int x = 0; x < 4; x += 2) {
                                ffma2(t[u][x], t[u][x + 1], t[u][x], t[u][x + 1], sc0, sc1, -b0, -b1);
                                t[u][x] = ex2_approx(t[u][x]);
                                t[u][x + 1] = ex2_approx(t[u][x + 1]);
                                fadd2(l0[0], l1[0], l0[0], l1[0], t[u][x], t[u][x + 1]);
                            }
                        zero_behind();
                        // ---- O^T += V^T P^T, group by group; P's 8 x 8 blocks (entries, rows) turned round
#pragma unroll
                        for (int u = 0; u < GP; ++u) {
                            const uint32_t vbase = base[u] + C::TILE + v_lane;
                            if constexpr (!FP8) {
                                uint32_t hi[2], lo[2];
#pragma unroll
                                for (int x = 0; x < 2; ++x) {
                                    const float pa = t[u][2 * x], pb = t[u][2 * x + 1];
                                    const uint32_t h = pack_bf16x2(pa, pb);
                                    hi[x] = turn8x8(h);
                                    lo[x] = turn8x8(pack_bf16x2(pa - __uint_as_float(h << 16), pb - __uint_as_float(h & 0xFFFF0000u)));
                                }
#pragma unroll
                                for (int d = 0; d < D / 16; ++d) {
                                    uint32_t vf[4];
                                    ldsm4_t(vf, vbase + (d / (C::CB / 32)) * chunk + (v_unit ^ ((d % (C::CB / 32)) << 5)));
                                    mma16816<false>(o[d], {vf[0], vf[2], vf[1], vf[3]}, hi[0], hi[1]);
                                    mma16816<false>(o[d], {vf[0], vf[2], vf[1], vf[3]}, lo[0], lo[1]);
                                }
                            } else {
                                const uint32_t p0 = turn8x8(pack_f16x2(t[u][0], t[u][1])), p1 = turn8x8(pack_f16x2(t[u][2], t[u][3]));
#pragma unroll
                                for (int d = 0; d < D / 32; ++d) {   // two 16-byte units: 32 features
                                    uint32_t vf[4];
                                    ldsm4_t(vf, vbase + (d / (C::CB / 32)) * chunk + (v_unit ^ ((d % (C::CB / 32)) << 5)));
#pragma unroll
                                    for (int w = 0; w < 2; ++w) {
                                        // a register holds features (f, f + 1) of entries 2 c and 2 c + 1: pair the entries;
                                        // even features are the product's first 8 rows, odd ones the others
                                        const uint32_t x = __byte_perm(vf[2 * w], 0, 0x3120), y = __byte_perm(vf[2 * w + 1], 0, 0x3120);
                                        mma16816<true>(o[2 * d + w], {e4m3x2_to_f16x2(x), e4m3x2_to_f16x2(x >> 16),
                                                                      e4m3x2_to_f16x2(y), e4m3x2_to_f16x2(y >> 16)}, p0, p1);
                                    }
                                }
                            }
                        }
                        continue;
                    } else {
                        // ---- S = Q K^T: 16 rows x 16 entries a group; a single group has two accumulators for
                        // each 8 entries, so that four products are always under way
                        float s[4][4];
#pragma unroll
                        for (int t = 0; t < 4; ++t)
                            s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.f;
#pragma unroll
                        for (int k = 0; k < KSTEPS; k += FP8 ? 2 : 1) {
                            uint32_t qa[4], qb[4];
                            if constexpr (QREG) {
#pragma unroll
                                for (int x = 0; x < 4; ++x) {
                                    qa[x] = qf[k][x];
                                    qb[x] = qf[FP8 ? k + 1 : k][x];
                                }
                            } else {
                                ldsm4(qa, q_lane + k * 32);
                                if constexpr (FP8)
                                    ldsm4(qb, q_lane + k * 32 + 32);
                            }
#pragma unroll
                            for (int u = 0; u < GP; ++u) {
                                uint32_t kf[4];
                                if constexpr (!FP8) {   // a 16-byte unit is 8 features
                                    ldsm4(kf, base[u] + k_lane + (k / (C::CB / 32)) * chunk + (k_unit ^ ((k % (C::CB / 32)) << 5)));
                                    const int z = GP == 2 ? 2 * u : (k & 1) * 2;
                                    mma16816<false>(s[z], qa, kf[0], kf[1]);
                                    mma16816<false>(s[z + 1], qa, kf[2], kf[3]);
                                } else {   // 16 features
                                    ldsm4(kf, base[u] + k_lane + (k / (C::CB / 16)) * chunk + (k_unit ^ ((k % (C::CB / 16)) << 4)));
                                    const int z = GP == 2 ? 2 * u : 2;
                                    mma16816<true>(s[2 * u], qa, e4m3x2_to_f16x2(kf[0]), e4m3x2_to_f16x2(kf[0] >> 16));
                                    mma16816<true>(s[2 * u + 1], qa, e4m3x2_to_f16x2(kf[2]), e4m3x2_to_f16x2(kf[2] >> 16));
                                    mma16816<true>(s[z], qb, e4m3x2_to_f16x2(kf[1]), e4m3x2_to_f16x2(kf[1] >> 16));
                                    mma16816<true>(s[z + 1], qb, e4m3x2_to_f16x2(kf[3]), e4m3x2_to_f16x2(kf[3] >> 16));
                                }
                            }
                        }
                        if constexpr (GP == 1) {
#pragma unroll
                            for (int x = 0; x < 4; ++x) {
                                s[0][x] += s[2][x];
                                s[1][x] += s[3][x];
                            }
                        }
                        if (!clear) {
#pragma unroll
                            for (int t = 0; t < 2 * GP; ++t) {
                                const bool in = (have >> (t >> 1)) & 1u;
                                const int key = key0 + 8 * t + 2 * c4;
                                s[t][0] = in && sees0(key) ? s[t][0] : -INFINITY;
                                s[t][1] = in && sees0(key + 1) ? s[t][1] : -INFINITY;
                                s[t][2] = in && sees1(key) ? s[t][2] : -INFINITY;
                                s[t][3] = in && sees1(key + 1) ? s[t][3] : -INFINITY;
                            }
                        }
                        if (a.scores) {
#pragma unroll
                            for (int t = 0; t < 2 * GP; ++t)
                                if (key0 + 8 * (t & ~1) < len)
                                    put_scores(key0 + 8 * t, s[t][0] * sc0, s[t][1] * sc0, s[t][2] * sc1, s[t][3] * sc1);
                        }
                        // ---- online softmax
                        constexpr float SH = FP8 ? kPShift : 0.f;
                        float x0 = fmaxf(fmax3(s[0][0], s[0][1], s[1][0]), s[1][1]);
                        float x1 = fmaxf(fmax3(s[0][2], s[0][3], s[1][2]), s[1][3]);
                        if constexpr (GP == 2) {
                            x0 = fmax3(fmax3(x0, s[2][0], s[2][1]), s[3][0], s[3][1]);
                            x1 = fmax3(fmax3(x1, s[2][2], s[2][3]), s[3][2], s[3][3]);
                        }
                        const float n0 = fmaxf(m0, quad_max(x0) * sc0 - SH), n1 = fmaxf(m1, quad_max(x1) * sc1 - SH);
                        const float b0 = n0 == -INFINITY ? 0.f : n0, b1 = n1 == -INFINITY ? 0.f : n1;
                        if (__any_sync(0xffffffffu, n0 > m0 || n1 > m1)) {
                            const float f0 = ex2_approx(m0 - b0), f1 = ex2_approx(m1 - b1);
                            l0[0] *= f0, l0[1] *= f0;
                            l1[0] *= f1, l1[1] *= f1;
#pragma unroll
                            for (int d = 0; d < D / 8; ++d) {
                                o[d][0] *= f0;
                                o[d][1] *= f0;
                                o[d][2] *= f1;
                                o[d][3] *= f1;
                            }
                            m0 = n0;
                            m1 = n1;
                        }
#pragma unroll
                        for (int t = 0; t < 2 * GP; ++t) {
                            ffma2(s[t][0], s[t][1], s[t][0], s[t][1], sc0, sc0, -b0, -b0);
                            ffma2(s[t][2], s[t][3], s[t][2], s[t][3], sc1, sc1, -b1, -b1);
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                s[t][x] = ex2_approx(s[t][x]);
                            fadd2(l0[0], l0[1], l0[0], l0[1], s[t][0], s[t][1]);
                            fadd2(l1[0], l1[1], l1[0], l1[1], s[t][2], s[t][3]);
                        }
                        zero_behind();
#pragma unroll
                        for (int u = 0; u < GP; ++u) {
                            const uint32_t vbase = base[u] + C::TILE + v_lane;
                            const float(&pu)[4] = s[2 * u], (&pw)[4] = s[2 * u + 1];
                            if constexpr (!FP8) {
                                uint32_t hi[4], lo[4];
#pragma unroll
                                for (int x = 0; x < 4; ++x) {
                                    const float pa = x < 2 ? pu[x * 2] : pw[(x - 2) * 2], pb = x < 2 ? pu[x * 2 + 1] : pw[(x - 2) * 2 + 1];
                                    hi[x] = pack_bf16x2(pa, pb);
                                    lo[x] = pack_bf16x2(pa - __uint_as_float(hi[x] << 16), pb - __uint_as_float(hi[x] & 0xFFFF0000u));
                                }
#pragma unroll
                                for (int d = 0; d < D / 16; ++d) {
                                    uint32_t vf[4];
                                    ldsm4_t(vf, vbase + (d / (C::CB / 32)) * chunk + (v_unit ^ ((d % (C::CB / 32)) << 5)));
                                    mma16816<false>(o[2 * d], hi, vf[0], vf[1]);
                                    mma16816<false>(o[2 * d + 1], hi, vf[2], vf[3]);
                                    mma16816<false>(o[2 * d], lo, vf[0], vf[1]);
                                    mma16816<false>(o[2 * d + 1], lo, vf[2], vf[3]);
                                }
                            } else {
                                uint32_t pf[4];
#pragma unroll
                                for (int x = 0; x < 4; ++x)
                                    pf[x] = x < 2 ? pack_f16x2(pu[x * 2], pu[x * 2 + 1]) : pack_f16x2(pw[(x - 2) * 2], pw[(x - 2) * 2 + 1]);
#pragma unroll
                                for (int d = 0; d < D / 32; ++d) {   // two 16-byte units: 32 features
                                    uint32_t vf[4];
                                    ldsm4_t(vf, vbase + (d / (C::CB / 32)) * chunk + (v_unit ^ ((d % (C::CB / 32)) << 5)));
#pragma unroll
                                    for (int w = 0; w < 2; ++w) {
                                        // a register holds features (f, f + 1) of entries 2 c and 2 c + 1: pair the entries
                                        const uint32_t x = __byte_perm(vf[2 * w], 0, 0x3120), y = __byte_perm(vf[2 * w + 1], 0, 0x3120);
                                        mma16816<true>(o[4 * d + 2 * w], pf, e4m3x2_to_f16x2(x), e4m3x2_to_f16x2(y));
                                        mma16816<true>(o[4 * d + 2 * w + 1], pf, e4m3x2_to_f16x2(x >> 16), e4m3x2_to_f16x2(y >> 16));
                                    }
                                }
                            }
                        }
                    }
                }
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bar0 + 8u * (C::NST + st));
                if (++st == depth) {
                    st = 0;
                    ++round;
                }
            }

            // the join's blocks may come now: earlier they would take registers that CTAs of the next
            // call want
            pdl_launch();
            // the next unit's query rows, under way while this one is put together
            Place next = p;
            next_unit<RANGED>(a, next, cnt);
            if (RT == 1 && next.left > 0)
                fetch_q(next);
            // ---- the warps' states of each row tile together, then out, MR rows of each at a time
            float s0 = l0[0] + l0[1], s1 = l1[0] + l1[1];
#pragma unroll
            for (int off = TURNED ? 4 : 1; off < (TURNED ? 32 : 4); off <<= 1) {
                s0 += __shfl_xor_sync(0xffffffffu, s0, off);
                s1 += __shfl_xor_sync(0xffffffffu, s1, off);
            }
            const bool first_lane = TURNED ? r0 == 0 : c4 == 0;   // of those that have the same rows
            if (first_lane) {
                ml[kw * RT * 16 + la] = make_float2(m0, s0);
                ml[kw * RT * 16 + lz] = make_float2(m1, s1);
            }
            math_sync();
            const bool entire = p.tile == 0 && cnt == p.nt;   // all of the unit
            const long long slot = 2ll * blockIdx.x + (p.left == mine_all ? 0 : 1);
            float *part = a.part + slot * a.rows * (D + 2);
            const float vs = FP8 ? a.vs[h] : 1.f;
            // the factor of this warp's sums in a row's output (or, scaled by vs, in its partial state); one
            // warp of the row tile writes the row's statistics
            auto factor = [&](int row, float m) {
                float t = -INFINITY, l = 0.f;
#pragma unroll
                for (int w = 0; w < KW; ++w)
                    t = fmaxf(t, ml[w * RT * 16 + row].x);
                const float z = t == -INFINITY ? 0.f : t;
#pragma unroll
                for (int w = 0; w < KW; ++w) {
                    const float2 y = ml[w * RT * 16 + row];
                    l = fmaf(y.y, ex2_approx(y.x - z), l);
                }
                if (kw == 0 && first_lane && row < nrows && ok) {
                    if (entire) {
                        const float y = t + log2f(l);   // -inf if l is 0
                        a.lse[grow + row] = l == 0.f ? -INFINITY : y * 0.69314718055994530942f;
                        row_lse[row] = l == 0.f ? 0.f : y;   // a row that saw nothing has no finite score either
                    } else {
                        part[(long long)a.rows * D + row] = t;
                        part[(long long)a.rows * (D + 1) + row] = l;
                    }
                }
                return ex2_approx(m - z) * (entire ? (l == 0.f ? 0.f : vs / l) : vs);
            };
            const float f0 = factor(la, m0), f1 = factor(lz, m1);
            if constexpr (KW == 1) {   // a row is one warp's: out of its registers
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int row = rt * 16 + r0 + 8 * half;
                    if (row >= nrows || !ok)
                        continue;
                    const float f = half ? f1 : f0;
                    uint32_t *dst = reinterpret_cast<uint32_t *>(a.o + (grow + row) * D) + (FP8 ? 2 * c4 : c4);
                    // 8-byte stores: a slot of `rows` (D + 2) floats is a multiple of 8 bytes
                    const bool wide = RANGED && entire && a.o32;
                    float2 *pd = reinterpret_cast<float2 *>(wide ? a.o32 + (grow + row) * D : part + (long long)row * D) + (FP8 ? 2 * c4 : c4);
#pragma unroll
                    for (int x = 0; x < D / 8; x += 2) {
                        const float a0 = o[x][2 * half] * f, a1 = o[x][2 * half + 1] * f;
                        const float b0 = o[x + 1][2 * half] * f, b1 = o[x + 1][2 * half + 1] * f;
                        if constexpr (!FP8) {
                            if (entire && !wide) {
                                dst[4 * x] = pack_bf16x2(a0, a1);
                                dst[4 * x + 4] = pack_bf16x2(b0, b1);
                            } else {
                                pd[4 * x] = make_float2(a0, a1);
                                pd[4 * x + 4] = make_float2(b0, b1);
                            }
                        } else {   // even and odd features of a 16-feature unit
                            if (entire && !wide) {
                                *reinterpret_cast<uint2 *>(dst + 4 * x) = make_uint2(pack_bf16x2(a0, b0), pack_bf16x2(a1, b1));
                            } else {
                                pd[4 * x] = make_float2(a0, b0);
                                pd[4 * x + 1] = make_float2(a1, b1);
                            }
                        }
                    }
                }
                math_sync();   // before the next unit's rows and states
            } else {
                constexpr int MR = C::MR;
#pragma unroll 1
                for (int first = 0; first < min(16, nrows); first += MR) {
                    if (TURNED && la / MR == first / MR) {
                        float *mine = ob + (kw * MR + la % MR) * C::OPITCH;
#pragma unroll
                        for (int x = 0; x < OT; ++x) {
                            if constexpr (!FP8) {
                                mine[16 * x + r0] = o[x][0] * f0;
                                mine[16 * x + 8 + r0] = o[x][2] * f0;
                                mine[C::OPITCH + 16 * x + r0] = o[x][1] * f1;
                                mine[C::OPITCH + 16 * x + 8 + r0] = o[x][3] * f1;
                            } else {
                                *reinterpret_cast<float2 *>(mine + 16 * x + 2 * r0) = make_float2(o[x][0] * f0, o[x][2] * f0);
                                *reinterpret_cast<float2 *>(mine + C::OPITCH + 16 * x + 2 * r0) = make_float2(o[x][1] * f1, o[x][3] * f1);
                            }
                        }
                    }
                    if (!TURNED && r0 / MR == (first & 7) / MR) {
                        float *mine = ob + (warp * MR + r0 % MR) * C::OPITCH;
                        const bool low = first < 8;
                        const float f = low ? f0 : f1;
#pragma unroll
                        for (int x = 0; x < (TURNED ? 0 : D / 8); x += 2) {
                            const float a0 = (low ? o[x][0] : o[x][2]) * f, a1 = (low ? o[x][1] : o[x][3]) * f;
                            const float b0 = (low ? o[x + 1][0] : o[x + 1][2]) * f, b1 = (low ? o[x + 1][1] : o[x + 1][3]) * f;
                            if constexpr (!FP8) {
                                *reinterpret_cast<float2 *>(mine + 8 * x + 2 * c4) = make_float2(a0, a1);
                                *reinterpret_cast<float2 *>(mine + 8 * x + 8 + 2 * c4) = make_float2(b0, b1);
                            } else {
                                *reinterpret_cast<float4 *>(mine + 8 * x + 4 * c4) = make_float4(a0, b0, a1, b1);
                            }
                        }
                    }
                    math_sync();
#pragma unroll
                    for (int e = 0; e < RT; ++e) {   // four features of one row a thread: RT * MR rows of D
                        const int at = e * 128 + (int)threadIdx.x, k = at / (D / 4), col = (at % (D / 4)) * 4;
                        const int rt_ = k / MR, row = rt_ * 16 + first + k % MR;
                        if (row >= nrows || !ok)
                            continue;
                        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                        for (int w = 0; w < KW; ++w) {
                            const float4 y = *reinterpret_cast<const float4 *>(ob + ((w * RT + rt_) * MR + k % MR) * C::OPITCH + col);
                            x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
                        }
                        const bool wide = RANGED && entire && a.o32;
                        if (entire && !wide) {
                            *reinterpret_cast<uint2 *>(a.o + (grow + row) * D + col) =
                                make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
                        } else {
                            float2 *dst = reinterpret_cast<float2 *>((wide ? a.o32 + (grow + row) * D : part + (long long)row * D) + col);
                            dst[0] = make_float2(x.x, x.y);
                            dst[1] = make_float2(x.z, x.w);
                        }
                    }
                    math_sync();
                }
            }
            // ---- one CTA has the whole unit, its scores too: weight_j += sum over the rows of
            // p_j = 2^{s_j - lse}, four neighbours a thread
            if (whole && a.scores && ok)
                for (int j = 4 * (int)threadIdx.x; j < len; j += 4 * 32 * kMathWarps)
                    add_weights(a, ((long long)p.b * a.Hkv + h) * a.cap + j, len - j,
                                a.scores + ((long long)p.b * a.Hkv + h) * a.M * a.cap + j, nrows, row_lse,
                                make_float4(0.f, 0.f, 0.f, 0.f), true);
            p = next;
        }
    }
}

// ------------------------------------------------------------------ join
// Where a unit's states are: CTAs c0 .. c1, the first one's in slot s0, the others' in their
// first slots.  c0 == c1: the whole unit was one CTA's and its o and lse are written.
struct Parts {
    int c0, c1;
    long long s0;
    bool none;   // no entry at all
};

// (SHORT: by 32-bit divisions where they do.)
template <bool SHORT = false>
__device__ __forceinline__ Parts parts_of(long long share, long long first, int ul, int nt)   // a.where[0], [1 + b]
{
    Parts p{0, 0, 0, nt == 0};
    if (nt > 0) {
        const long long t = first + (long long)ul * nt;
        if (SHORT && ((t + nt) | share) >> 32 == 0) {
            p.c0 = (int)((uint32_t)t / (uint32_t)share);
            p.c1 = (int)((uint32_t)(t + nt - 1) / (uint32_t)share);
        } else {
            p.c0 = (int)(t / share);
            p.c1 = (int)((t + nt - 1) / share);
        }
        p.s0 = 2ll * p.c0 + (t == p.c0 * share ? 0 : 1);
    }
    return p;
}

// The first blocks: o and lse of rpb rows of a unit whose entries were split (or of a sequence
// without any).  Blocks from there: kWeightRun entries' weights of one (sequence, KV head).
// The states of a row are read by D / 2 threads a state, two features each, so that several are
// under way at once.
constexpr int kJoinThreads = 128, kWeightRun = 4 * kJoinThreads;
constexpr int kMaxCtas = 3 * kSMs, kMaxParts = kMaxCtas;

template <int D>
__global__ void __launch_bounds__(kJoinThreads, 8) paged_join_kernel(const __grid_constant__ PagedArgs a, int wchunks, int rpb)
{
    __shared__ float wt[kMaxParts], row_lse[kMaxRows], sums[kJoinThreads * 2], red[8];
    const int tid = threadIdx.x, per = a.Hkv * a.RB;
    const int bpu = (a.rows + rpb - 1) / rpb;   // blocks a unit
    const long long rows_total = (long long)a.B * per * bpu, blk = blockIdx.x;
    const long long stride = (long long)a.rows * (D + 2);
    pdl_launch();
    const bool joins = blk < rows_total;
    const long long unit = joins ? blk / bpu : (blk - rows_total) / wchunks;   // or, for weights, (sequence, KV head)
    const int b = (int)(unit / (joins ? per : a.Hkv)), ul = (int)(unit - (long long)b * (joins ? per : a.Hkv)), h = ul % a.Hkv;
    // The lengths may be read in front of the wait: this kernel is launched when every CTA of the
    // attention is past its own wait (or after the kernel before this one has ended).  All that it wrote is read behind
    // the wait, in two steps: the place, then everything of the states at once (loads that wait for one
    // another cost 0.7 us each).
    const int len = length_in_range(a, __ldcg(a.lens + b)), nt = tiles_in<false>(a, len);
    pdl_wait();
    const long long share = a.where[0], place = a.where[1 + b];
    if (a.may_whole && share == 0)
        return;   // whole units: nothing is left to do
    if (joins) {
        const int first = (int)(blk - unit * bpu) * rpb, rb = ul / a.Hkv;
        const Parts p = parts_of(share, place, ul, nt);
        if (!p.none && p.c0 == p.c1)
            return;
        for (int row = first; row < min(first + rpb, min(a.rows, a.M - rb * a.rows)); ++row) {
            const long long grow = ((long long)b * a.Hq + h * a.G) * a.Tq + rb * a.rows + row;
            auto slot = [&](int i) { return a.part + (i == 0 ? p.s0 : 2ll * (p.c0 + i)) * stride; };
            const int n = p.none ? 0 : p.c1 - p.c0 + 1;
            constexpr int GROUPS = 2 * kJoinThreads / D;   // states under way
            constexpr int PER = (kMaxParts + kJoinThreads - 1) / kJoinThreads, AHEAD = 8;
            const int g = tid / (D / 2), f = 2 * (tid % (D / 2));
            float mi[PER], li[PER];
            float2 y[AHEAD];
#pragma unroll
            for (int u = 0; u < PER; ++u) {
                const int i = tid + u * kJoinThreads;
                mi[u] = i < n ? slot(i)[(long long)a.rows * D + row] : -INFINITY;
                li[u] = i < n ? slot(i)[(long long)a.rows * (D + 1) + row] : 0.f;
            }
#pragma unroll
            for (int u = 0; u < AHEAD; ++u) {
                const int i = g + u * GROUPS;
                y[u] = i < n ? *reinterpret_cast<const float2 *>(slot(i) + (long long)row * D + f) : make_float2(0.f, 0.f);
            }
            // the states' maxima, then their weights
            float m = -INFINITY, l = 0.f;
#pragma unroll
            for (int u = 0; u < PER; ++u)
                m = fmaxf(m, mi[u]);
#pragma unroll
            for (int off = 16; off > 0; off >>= 1)
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
            if (lane_id() == 0)
                red[warp_id()] = m;
            __syncthreads();
            m = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
#pragma unroll
            for (int u = 0; u < PER; ++u) {
                const int i = tid + u * kJoinThreads;
                const float w = mi[u] == -INFINITY ? 0.f : ex2_approx(mi[u] - m);
                l = fmaf(w, li[u], l);
                if (i < n)
                    wt[i] = w;
            }
#pragma unroll
            for (int off = 16; off > 0; off >>= 1)
                l += __shfl_xor_sync(0xffffffffu, l, off);
            if (lane_id() == 0)
                red[4 + warp_id()] = l;
            __syncthreads();
            l = (red[4] + red[5]) + (red[6] + red[7]);
            float2 x = make_float2(0.f, 0.f);
#pragma unroll
            for (int u = 0; u < AHEAD; ++u) {
                const int i = g + u * GROUPS;
                const float w = i < n ? wt[i] : 0.f;
                x.x = fmaf(w, y[u].x, x.x);
                x.y = fmaf(w, y[u].y, x.y);
            }
#pragma unroll 8
            for (int i = g + AHEAD * GROUPS; i < n; i += GROUPS) {
                const float2 z = *reinterpret_cast<const float2 *>(slot(i) + (long long)row * D + f);
                x.x = fmaf(wt[i], z.x, x.x);
                x.y = fmaf(wt[i], z.y, x.y);
            }
            reinterpret_cast<float2 *>(sums)[tid] = x;
            __syncthreads();
            if (g == 0) {
#pragma unroll
                for (int w = 1; w < GROUPS; ++w) {
                    const float2 z = reinterpret_cast<const float2 *>(sums)[w * (D / 2) + tid];
                    x.x += z.x;
                    x.y += z.y;
                }
                const float k = l == 0.f ? 0.f : 1.f / l;
                *reinterpret_cast<uint32_t *>(a.o + grow * D + f) = pack_bf16x2(x.x * k, x.y * k);
                if (tid == 0)
                    a.lse[grow] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994530942f;
            }
            __syncthreads();   // before the next row's states
        }
        return;
    }
    // ---- weight_j += sum over the rows of p_j = 2^{s_j - lse}, four neighbours a thread
    const long long uh = unit;
    const int j = (int)(blk - rows_total - uh * wchunks) * kWeightRun + 4 * tid;
    if (j - 4 * tid >= len)
        return;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int rb = 0; rb < a.RB; ++rb) {
        const Parts p = parts_of(share, place, rb * a.Hkv + h, nt);
        const int row0 = rb * a.rows, nrows = min(a.rows, a.M - row0);
        for (int r = tid; r < nrows; r += kJoinThreads) {
            float y;
            if (p.c0 == p.c1) {
                y = a.lse[((long long)b * a.Hq + h * a.G) * a.Tq + row0 + r] * 1.4426950408889634f;
            } else {
                float m = -INFINITY, l = 0.f;
                const int n = p.c1 - p.c0 + 1;
                auto slot = [&](int i) { return a.part + (i == 0 ? p.s0 : 2ll * (p.c0 + i)) * stride + (long long)a.rows * D + r; };
#pragma unroll 4
                for (int i = 0; i < n; ++i) {   // online, so that both loads of a state go together
                    const float mi = *slot(i), li = slot(i)[a.rows], t = fmaxf(m, mi), z = t == -INFINITY ? 0.f : t;
                    l = l * ex2_approx(m - z) + li * ex2_approx(mi - z);
                    m = t;
                }
                y = l == 0.f ? -INFINITY : m + log2f(l);
            }
            // a row that saw nothing has no finite score either: 2^{-inf - 0}
            row_lse[r] = y == -INFINITY ? 0.f : y;
        }
        __syncthreads();
        if (j < len)
            sum = add_weights(a, uh * a.cap + j, len - j, a.scores + (uh * a.M + row0) * a.cap + j, nrows, row_lse, sum,
                              rb == a.RB - 1);
        __syncthreads();
    }
}

// RANGED: a warp a row, which has few states; the first AHEAD of them are read whole at once, behind the place and
// nothing else.
template <int D>
__global__ void __launch_bounds__(kJoinThreads) range_join_kernel(const __grid_constant__ PagedArgs a)
{
    constexpr int F = D / 32, AHEAD = 4;
    pdl_launch();
    const int lane = (int)lane_id();
    const uint32_t row = blockIdx.x * (kJoinThreads / 32) + warp_id();   // (b Hq + head) Tq + t
    const bool here = row < (uint32_t)(a.B * a.Hq * a.Tq);
    const uint32_t bh = row / (uint32_t)a.Tq, b32 = bh / (uint32_t)a.Hq;
    const int t = (int)(row - bh * (uint32_t)a.Tq), head = (int)(bh - b32 * (uint32_t)a.Hq), b = (int)b32;
    const int h = head / a.G, i = (head - h * a.G) * a.Tq + t, rb = i / a.rows, ri = i - rb * a.rows;
    // the lengths in front of the wait, as in paged_join_kernel
    const int len = here ? length_in_range(a, __ldcg(a.lens + b)) : 0, nt = here ? tiles_in<true>(a, len) : 0;
    pdl_wait();
    if (!here)
        return;
    const long long share = __ldcg(a.where), place = __ldcg(a.where + 1 + b);
    if (a.may_whole && share == 0)
        return;   // whole units: nothing is left to do
    const Parts p = parts_of<true>(share, place, rb * a.Hkv + h, nt);
    if (!p.none && p.c0 == p.c1)
        return;
    const long long stride = (long long)a.rows * (D + 2);
    const int n = p.none ? 0 : p.c1 - p.c0 + 1;
    auto slot = [&](int s) { return a.part + (s == 0 ? p.s0 : 2ll * (p.c0 + s)) * stride; };
    auto state = [&](int s) {
        return s < n ? make_float2(__ldcg(slot(s) + (long long)a.rows * D + ri), __ldcg(slot(s) + (long long)a.rows * (D + 1) + ri))
                     : make_float2(-INFINITY, 0.f);
    };
    float y[AHEAD][F];
    float2 st[AHEAD];
#pragma unroll
    for (int s = 0; s < AHEAD; ++s) {
        st[s] = state(s);
#pragma unroll
        for (int f = 0; f < F; f += 2) {
            const float2 z = s < n ? __ldcg(reinterpret_cast<const float2 *>(slot(s) + (long long)ri * D + lane * F + f)) : make_float2(0.f, 0.f);
            y[s][f] = z.x, y[s][f + 1] = z.y;
        }
    }
    float m = -INFINITY, l = 0.f, x[F];
    for (int s = lane; s < n; s += 32)
        m = fmaxf(m, state(s).x);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
#pragma unroll
    for (int f = 0; f < F; ++f)
        x[f] = 0.f;
#pragma unroll
    for (int s = 0; s < AHEAD; ++s) {
        const float w = st[s].x == -INFINITY ? 0.f : ex2_approx(st[s].x - m);
        l = fmaf(w, st[s].y, l);
#pragma unroll
        for (int f = 0; f < F; ++f)
            x[f] = fmaf(w, y[s][f], x[f]);
    }
#pragma unroll 4
    for (int s = AHEAD; s < n; ++s) {
        const float2 z = state(s);
        const float w = z.x == -INFINITY ? 0.f : ex2_approx(z.x - m);
        l = fmaf(w, z.y, l);
#pragma unroll
        for (int f = 0; f < F; f += 2) {
            const float2 u = __ldcg(reinterpret_cast<const float2 *>(slot(s) + (long long)ri * D + lane * F + f));
            x[f] = fmaf(w, u.x, x[f]);
            x[f + 1] = fmaf(w, u.y, x[f + 1]);
        }
    }
    const float k = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int f = 0; f < F; f += 2)
        *reinterpret_cast<uint32_t *>(a.o + (long long)row * D + lane * F + f) = pack_bf16x2(x[f] * k, x[f + 1] * k);
    if (lane == 0)
        a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994530942f;
}

// ------------------------------------------------------------------ host
size_t round256(size_t x) { return (x + 255) & ~(size_t)255; }

int rows_of(int M) { return M < kMaxRows ? M : kMaxRows; }
int tile_rows(int M) { return M <= 8 ? 8 : M <= 16 ? 16 : M <= 32 ? 32 : 64; }   // of the instance


// Tables of up to this many slots (half at d 256): one CTA a unit and no join.  8 units of 256, 512 and
// 1024 entries, d 64: 4.7, 6.7 and 10.4 us against 7.2, 7.2 and 7.2 in shares; d 128: 6.0, 8.5 and 14.0
// against 7.9, 8.0 and 8.0; d 256: 7.5, 11.5 and 19.3 against 8.7, 8.7 and 8.9.  240 units of 512, d 128: 13.2
// against 20.1.
constexpr int kWholeSlots = 512;

size_t where_bytes(int B) { return round256((size_t)(B + 1) * sizeof(long long)); }
size_t part_bytes(int M, int d) { return round256((size_t)2 * kMaxCtas * rows_of(M) * (d + 2) * sizeof(float)); }

// K or V pool as [page, KV head][column chunk][row][CB bytes]; a box is all chunks of a page's
// rows (64 at most).
int encode_pool(CUtensorMap *map, const void *base, const fa_kv_cache &c, int box_rows)
{
    const bool f8 = c.dtype == FA_E4M3;
    const int elem = f8 ? 1 : 2, rowb = c.d * elem, cb = rowb < 128 ? rowb : 128;
    const uint64_t dims[4] = {(uint64_t)(cb / elem), (uint64_t)c.page_size, (uint64_t)(rowb / cb),
                              (uint64_t)c.num_pages * c.Hkv};
    const uint64_t strides[3] = {(uint64_t)rowb, (uint64_t)cb, (uint64_t)c.page_size * rowb};
    const uint32_t box[4] = {(uint32_t)(cb / elem), (uint32_t)box_rows, (uint32_t)(rowb / cb), 1};
    return encode_tmap(map, base, f8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, dims, strides,
                       box, cb == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
}

template <int D, bool FP8, int ROWS, bool RANGED>
int launch_main(const CUtensorMap &tk, const CUtensorMap &tv, const PagedArgs &a, int grid, cudaStream_t s)
{
    using C = Cfg<D, FP8, ROWS>;
    if (const int st = allow_smem<paged_kernel<D, FP8, ROWS, RANGED>>(C::SMEM); st != OK)
        return st;
    return launch_overlapped(paged_kernel<D, FP8, ROWS, RANGED>, dim3((unsigned)grid), kThreads, C::SMEM, 0, true, s, tk, tv, a);
}

template <int D, bool RANGED>
int paged_run(const fa_kv_cache &c, PagedArgs &a, cudaStream_t s)
{
    const bool f8 = c.dtype == FA_E4M3;
    const int rows = tile_rows(a.M);
    a.kt = f8 ? Cfg<D, true, 8>::KT : Cfg<D, false, 8>::KT;
    const int ctas = rows == 8    ? (f8 ? Cfg<D, true, 8>::CTAS : Cfg<D, false, 8>::CTAS)
                     : rows == 16 ? (f8 ? Cfg<D, true, 16>::CTAS : Cfg<D, false, 16>::CTAS)
                                  : f8 ? Cfg<D, true, 32>::CTAS : Cfg<D, false, 32>::CTAS;
    a.grid = kSMs * ctas;
    // tiles, at most: those of a window begin and end anywhere, and so do the sinks'
    const long long most = (long long)a.B * a.Hkv * a.RB * std::min((a.cap + a.kt - 1) / a.kt, RANGED ? a.span / a.kt + 3 : INT_MAX);
    // RANGED: up to two whole units for each CTA at a time, taken as others end.  us whole and in shares, 8 KV heads of
    // 128: 64 sequences of 20 to 700 entries 26.8 and 35.1 (a share of many short units has many starts), of 360 23.6 and
    // 24.6, of 1024 48.9 and 49.9, of 100 to 2000 under a window of 700 34.4 and 38.4; with more units a CTA
    // shares are better: 96 of 20 to 3000 107.9 and 103.3, 128 of 512 58.2 and 49.5, 200 of 300 69.6 and 53.2
    a.may_whole = a.may_whole && most > 0 && (long long)a.B * a.Hkv * a.RB <= (RANGED ? 2 : 1) * a.grid;
    int st = OK;
    if (most > 0) {
        CUtensorMap tk, tv;
        const int box = c.page_size < 64 ? c.page_size : 64;
        if ((st = encode_pool(&tk, c.k, c, box)) != OK || (st = encode_pool(&tv, c.v, c, box)) != OK)
            return st;
        const long long units = (long long)a.B * a.Hkv * a.RB;
        if (a.whole && units > INT_MAX)
            return ERR_UNSUPPORTED;
        const int grid = (int)(a.whole || (RANGED && a.may_whole && units > a.grid) ? units : most < a.grid ? most : a.grid);
        if (f8)
            st = rows == 8    ? launch_main<D, true, 8, RANGED>(tk, tv, a, grid, s)
                 : rows == 16 ? launch_main<D, true, 16, RANGED>(tk, tv, a, grid, s)
                 : rows == 32 ? launch_main<D, true, 32, RANGED>(tk, tv, a, grid, s)
                              : launch_main<D, true, 64, RANGED>(tk, tv, a, grid, s);
        else
            st = rows == 8    ? launch_main<D, false, 8, RANGED>(tk, tv, a, grid, s)
                 : rows == 16 ? launch_main<D, false, 16, RANGED>(tk, tv, a, grid, s)
                 : rows == 32 ? launch_main<D, false, 32, RANGED>(tk, tv, a, grid, s)
                              : launch_main<D, false, 64, RANGED>(tk, tv, a, grid, s);
        if (st != OK)
            return st;
    }
    if ((a.whole && most > 0) || (RANGED && a.o32))
        return OK;
    if constexpr (RANGED) {
        const long long blocks = ((long long)a.B * a.Hq * a.Tq + kJoinThreads / 32 - 1) / (kJoinThreads / 32);
        if (blocks > INT_MAX)
            return ERR_UNSUPPORTED;
        return launch_overlapped(range_join_kernel<D>, dim3((unsigned)blocks), kJoinThreads, 0, 0, most > 0, s, a);
    } else {
        const int wchunks = a.scores ? (a.cap + kWeightRun - 1) / kWeightRun : 0;
        // rows a block: one, unless that makes more blocks than the device holds at a time
        const long long units = (long long)a.B * a.Hkv * a.RB, held = 8 * kSMs;
        const int rpb = (int)std::min<long long>(a.rows, (units * a.rows + held - 1) / held);
        const long long blocks = units * ((a.rows + rpb - 1) / rpb) + (long long)a.B * a.Hkv * wchunks;
        if (blocks > INT_MAX)
            return ERR_UNSUPPORTED;
        return launch_overlapped(paged_join_kernel<D>, dim3((unsigned)blocks), kJoinThreads, 0, 0, most > 0, s, a, wchunks, rpb);
    }
}

// The arguments that both files' launches share.
PagedArgs paged_args(const fa_kv_cache &c, const void *q, void *o, float *lse, int Hq, int Tq, int causal, float scale, void *workspace)
{
    PagedArgs a{};
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.o = static_cast<__nv_bfloat16 *>(o);
    a.lse = lse;
    a.weight = c.weight;
    a.ks = c.k_scale;
    a.vs = c.v_scale;
    a.block_table = c.block_table;
    a.lens = c.lens;
    a.B = c.B;
    a.Hq = Hq;
    a.Hkv = c.Hkv;
    a.G = Hq / c.Hkv;
    a.Tq = Tq;
    a.M = a.G * Tq;
    a.rows = rows_of(a.M);
    a.RB = (a.M + a.rows - 1) / a.rows;
    a.causal = causal;
    a.num_pages = c.num_pages;
    a.max_pages = c.max_pages;
    a.ps_shift = 0;
    while ((1 << a.ps_shift) < c.page_size)
        ++a.ps_shift;
    a.cap = c.num_pages > 0 ? c.max_pages * c.page_size : 0;   // no pages: every length above 0 is out of range
    a.span = a.cap;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    a.where = reinterpret_cast<long long *>(ws);
    a.part = reinterpret_cast<float *>(ws + where_bytes(c.B));
    a.scale_log2 = std::min(scale * 1.4426950408889634f, FLT_MAX);   // finite, for sums of 0
    a.timeout_ns = wait_timeout_ns();
    a.withhold = WITHHOLD_NONE;
    return a;
}

// The file's status word (a timeout before an index out of range), read and cleared.
int paged_words_fetch_clear(cudaStream_t s, int *host_word)
{
    int word[2] = {0, 0};
    if (cudaMemcpyFromSymbolAsync(word, g_paged_status, sizeof(word), 0, cudaMemcpyDeviceToHost, s) != cudaSuccess ||
        cudaStreamSynchronize(s) != cudaSuccess)
        return ERR_CUDA;
    *host_word = word[0] ? word[0] : word[1];
    const int zero[2] = {0, 0};
    if (*host_word != 0 &&
        (cudaMemcpyToSymbolAsync(g_paged_status, zero, sizeof(zero), 0, cudaMemcpyHostToDevice, s) != cudaSuccess ||
         cudaStreamSynchronize(s) != cudaSuccess))
        return ERR_CUDA;
    return OK;
}

}  // namespace
}  // namespace fa
