// fa_prefix_sm103.cu -- attention of a batch over a prefix that all its sequences share, computed once for
// the rows of all of them, and joined with each sequence's own entries (sm_103a).
//
// Formulas, per KV head: the B G Tq query rows of its head group in all sequences are the rows of one matrix Q, the
// prefix's entries the rows of K and V.  S = Q K^T, and per row the online softmax's state over a run of entries:
// m = max c s, l = sum e^{c s - m}, O~ = sum e^{c s - m} v.  States of several runs, and that of the
// sequence's own entries (fa_paged_range_sm103.cu: o and lse, that is m = lse, l = 1, O~ = o), join as
// o = sum_i e^{m_i - M} O~_i / L, L = sum_i e^{m_i - M} l_i, lse = M + ln L.  Everything below is in log2 units.
//
// What bounds it: each entry's 4 d bytes (bf16) serve B G Tq rows at 4 d flops each, so that with 128 rows a KV
// head the tensor cores and the memory take about the same time, and with more the products do.  So they
// are tcgen05 products of 128 query rows by a tile of entries, with S and O~ in tensor memory:
//   * A CTA has one KV head's 128 (d 256) or 256 rows, in one or two query tiles, and one run of the
//     prefix's tiles of 128 entries (64 at d 256).  The runs are as many as fill the SMs.
//   * Warp 0 loads K and V tiles by TMA, a box for each page and 64 features, into 128-byte swizzled
//     tiles; pages that are not there, and what lies behind the prefix, come as zeros (a box behind the
//     pool's end).  One thread per query tile issues the products, S of tile k + 1 ahead of P V of tile k; a
//     warpgroup per query tile has the softmax, a thread a row.  As in fa_fwd_sm103.cu, O~ is rescaled
//     only where a row's maximum has grown by more than 2^8.
//   * Query rows are gathered by the softmax warps, straight into the swizzled tile: they lie scattered over the
//     batch, B runs of G Tq rows.  Warps whose 32 rows lie behind the last one take no part.
//   * e4m3: four more warps turn the tiles' codes into bf16, which holds every code exactly, so that q stays
//     as it is.
//   * P enters its product as bf16, as in the forward pass: 2^-8 of each probability.
// Measured: 64 sequences, 8 KV heads of 128 with 4 query heads each, 32768 entries (bf16): 34 us, of them 10 the start, the
// first tile and the states' way out and 1.9 for each 256 rows by 128 entries, the forward pass's rate; with the
// sequences' own 20 to 700 entries (26) and the join (8), one after the other, 69 us, where every sequence reading the
// prefix by itself takes 760.  16 sequences with 4 new rows, 4 KV heads of 64 with 4 query heads each, 65536 entries in
// e4m3: 33 of 48 us (each by itself: 93); there the issue slots are half busy, ex2 a quarter, and one warpgroup of four
// converts the codes.
#include <algorithm>
#include <cfloat>
#include <climits>

#include <cuda_fp16.h>

#include "fa_common.cuh"
#include "fa_internal.h"
#include "fa_pdl.cuh"

namespace fa {

// Device status words of the kernels in this file: [0] a wait that ran out, [1] an index out of range.
__device__ int g_prefix_status[2];

namespace {

constexpr int kStatusBadIndex = 5;
constexpr int BR = 128;                 // query rows of a tile
constexpr float kRescaleLog2 = 8.f;
constexpr int kSMs = 152;               // the runs are made for the GB300's; results depend on it, not on the device

enum PrefixSite : int { SITE_X_EMPTY = 1, SITE_X_REMPTY, SITE_X_RFULL, SITE_X_QFULL, SITE_X_FULL, SITE_X_SFREE, SITE_X_PFULL,
                        SITE_X_SFULL, SITE_X_ODONE };

template <int D, bool FP8>
struct XCfg {
    static constexpr int NQ = D == 256 ? 1 : 2;                 // query tiles of a CTA
    static constexpr int BC = D == 256 ? 64 : 128;              // entries a tile
    static constexpr int KCH = D / 64;                          // 128-byte chunks of a bf16 row
    static constexpr int Q_CHUNK = BR * 128, Q_TILE = KCH * Q_CHUNK;
    static constexpr int KV_CHUNK = BC * 128, KV_TILE = KCH * KV_CHUNK;
    static constexpr int PCH = BC / 64, P_CHUNK = BR * 128, P_TILE = PCH * P_CHUNK;
    static constexpr int RAW_TILE = BC * D;                     // codes
    static constexpr int OFF_Q = 0, OFF_P = NQ * Q_TILE, OFF_SLOT = OFF_P + NQ * P_TILE;
    static constexpr int AVAIL = 227 * 1024 - 1024 - 512 - OFF_SLOT;
    static constexpr int FIT = AVAIL / KV_TILE;
    static constexpr int NSLOT = FP8 ? (D == 64 ? 4 : D == 128 ? 2 : 3) : FIT < 8 ? FIT : 8;
    static constexpr int RFIT = (AVAIL - NSLOT * KV_TILE) / RAW_TILE;
    static constexpr int NRAW = FP8 ? (RFIT < 8 ? RFIT : 8) : 0;
    static_assert(NSLOT >= (FP8 ? 2 : 3) && (!FP8 || NRAW >= 2), "K/V rings");
    static constexpr int OFF_RAW = OFF_SLOT + NSLOT * KV_TILE;
    static constexpr int OFF_BAR = OFF_RAW + NRAW * RAW_TILE;
    static constexpr int B_FULL = 0, B_EMPTY = NSLOT, B_RFULL = 2 * NSLOT, B_REMPTY = B_RFULL + NRAW, B_QFULL = B_REMPTY + NRAW,
                         B_SFULL = B_QFULL + NQ, B_SFREE = B_SFULL + NQ, B_PFULL = B_SFREE + NQ, B_ODONE = B_PFULL + NQ,
                         B_DRAIN = B_ODONE + NQ, NBAR = B_DRAIN + NQ;
    static constexpr int OFF_MISC = OFF_BAR + 8 * NBAR;         // tensor memory's base, abort flag
    static constexpr int SMEM = OFF_MISC + 16 + 1024;
    static_assert(SMEM <= 227 * 1024, "shared memory");
    static constexpr int S_COL = 0, O_COL = NQ * BC, TMEM_COLS = 512;
    static_assert(O_COL + NQ * D <= TMEM_COLS, "tensor memory");
    // warps 0 to 3: loads, products; then a warpgroup per query tile; e4m3: one that converts
    static constexpr int NTHREADS = 128 + 128 * NQ + (FP8 ? 128 : 0);
    static constexpr uint32_t IDESC_S = idesc_bf16_f32(128, BC, false, false);   // Q K^T, both K-major
    static constexpr uint32_t IDESC_PV = idesc_bf16_f32(128, D, false, true);    // P K-major, V [entry][feature]
};

struct PrefixArgs {
    const __nv_bfloat16 *q;
    const float *ks, *vs;
    const int *pages, *lens;
    float *part;      // [unit][run][row] of D floats, then of (m, l)
    long long ml_at;  // floats in front of the (m, l)
    int B, Hq, Hkv, G, Tq, GT, R, RP;   // rows of a KV head, and CTAs' blocks of them
    int causal, P, num_pages, ps_shift, cap, runs;
    int run_tiles, run_more;            // tiles of a run; the first run_more have one more
    float scale_log2;
    uint64_t timeout_ns;
    int withhold;     // test builds: the arrive that is left out
};

__device__ __forceinline__ void fence_smem_to_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// The order of loads and products of n tiles: S(0), S(1), then P V(k) and S(k + 2).
template <typename FS, typename FPV>
__device__ __forceinline__ bool walk_ops(int n, FS &&fs, FPV &&fpv)
{
    if (!fs(0))
        return false;
    if (n > 1 && !fs(1))
        return false;
    for (int k = 0; k < n; ++k) {
        if (!fpv(k))
            return false;
        if (k + 2 < n && !fs(k + 2))
            return false;
    }
    return true;
}

// Sixteen e4m3 codes as bf16: through f16, which both conversions leave exact.
__device__ __forceinline__ void codes_to_bf16(uint4 c, uint4 &lo, uint4 &hi)
{
    const uint32_t in[4] = {c.x, c.y, c.z, c.w};
    uint32_t out[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t y;
            asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(y) : "r"(in[i] >> (16 * h)));
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&y));
            out[2 * i + h] = pack_bf16x2(f.x, f.y);
        }
    }
    lo = make_uint4(out[0], out[1], out[2], out[3]);
    hi = make_uint4(out[4], out[5], out[6], out[7]);
}

template <int D, bool FP8>
__global__ void __launch_bounds__(XCfg<D, FP8>::NTHREADS, 1)
    prefix_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                  const __grid_constant__ PrefixArgs a)
{
    using C = XCfg<D, FP8>;
    constexpr int BC = C::BC, NQ = C::NQ, NSLOT = C::NSLOT, NRAW = FP8 ? C::NRAW : 1;
    // Registers move from warps 0 to 3 (and those that convert) to the softmax: of three warpgroups with 168 each 104
    // and 200, or 104, 200 and 168; of four with 128 each 64, 176 twice and 96
    constexpr bool SPLIT = C::NTHREADS >= 384, FOUR = C::NTHREADS == 512;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t sbase = (raw + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (sbase - raw);
    const uint32_t bar0 = sbase + C::OFF_BAR;
    auto bar = [&](int i) -> uint32_t { return bar0 + 8u * (uint32_t)i; };
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::OFF_MISC);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::OFF_MISC + 4);
    const uint32_t warp = warp_id(), lane = lane_id();

    // row blocks of one run next to one another: they read the same entries
    const int rp = (int)blockIdx.x % a.RP, hr = (int)blockIdx.x / a.RP, run = hr % a.runs, h = hr / a.runs;
    const int row0 = rp * NQ * BR;
    const int nq = NQ == 2 && a.R - row0 > BR ? 2 : 1;   // query tiles with a row
    const int t0 = run * a.run_tiles + min(run, a.run_more), n = a.run_tiles + (run < a.run_more ? 1 : 0);
    if (threadIdx.x == 0) {
        for (int s = 0; s < NSLOT; ++s) {
            mbar_init(bar(C::B_FULL + s), FP8 ? 128 : 1);
            mbar_init(bar(C::B_EMPTY + s), nq);
        }
        for (int s = 0; s < C::NRAW; ++s) {
            mbar_init(bar(C::B_RFULL + s), 1);
            mbar_init(bar(C::B_REMPTY + s), 128);
        }
        for (int t = 0; t < NQ; ++t) {
            mbar_init(bar(C::B_QFULL + t), 128);
            mbar_init(bar(C::B_SFULL + t), 1);
            mbar_init(bar(C::B_SFREE + t), 128);
            mbar_init(bar(C::B_PFULL + t), 128);
            mbar_init(bar(C::B_ODONE + t), 1);
            mbar_init(bar(C::B_DRAIN + t), 1);
        }
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
    }
    if (warp == 0) {
        tmem_alloc(smem_u32(tmem_slot), C::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const WaitCtx ctx{abort_flag, &g_prefix_status[0], a.timeout_ns};
    // q, the lengths and the pages may come from the kernel in front of the own entries', which has ended by now;
    // but that its writes are visible here is promised behind the wait alone (68 us without it at 64 sequences and 32768
    // entries, 69 with it: CTAs that find a free SM wait for the last of the own entries)
    pdl_wait();
    pdl_launch();

    if (warp < 4) {
        if constexpr (SPLIT)
            regs_dealloc<FOUR ? 64 : 104>();
        if (warp == 0) {
            // ---------------------------------------------------- loads: lane = box (page, and 64 features in bf16)
            const int bp_shift = min(a.ps_shift, BC == 64 ? 6 : 7), boxes = BC >> bp_shift;   // rows of a box; boxes of a tile
            const int per = FP8 ? 1 : C::KCH, ops = boxes * per, box = (int)lane / per, ch = (int)lane - box * per;
            const bool mine = (int)lane < ops;
            const int nowhere = a.num_pages * a.Hkv;   // behind the pool: zeros
            const uint64_t policy = a.RP > 1 ? policy_evict_last() : policy_evict_first();
            constexpr int RING = FP8 ? NRAW : NSLOT, FIRST = FP8 ? C::B_RFULL : C::B_FULL, FREE = FP8 ? C::B_REMPTY : C::B_EMPTY;
            constexpr uint32_t BYTES = FP8 ? C::RAW_TILE : C::KV_TILE;
            uint32_t loads = 0;
            auto place_of = [&](int k) {   // of this lane's box in tile t0 + k: its page, or `nowhere`
                const int slot = (t0 + k) * BC + (box << bp_shift);
                if (!mine || k >= n || slot >= a.P)
                    return nowhere;
                const int page = __ldg(a.pages + (slot >> a.ps_shift));
                if (page >= 0 && page < a.num_pages)
                    return page * a.Hkv + h;
                atomicCAS(&g_prefix_status[1], 0, kStatusBadIndex);
                return nowhere;
            };
            auto load = [&](const CUtensorMap *map, int k, int z) -> bool {
                const uint32_t s = loads % RING;
                if (loads >= (uint32_t)RING &&
                    !mbar_wait_warp<true>(bar(FREE + s), (loads / RING - 1) & 1, ctx, FP8 ? SITE_X_REMPTY : SITE_X_EMPTY))
                    return false;
                if (lane == 0) {
#if FA_TEST_WITHHOLD
                    if (a.withhold == WITHHOLD_PREFIX_FULL && blockIdx.x == 0 && loads == 0)
                        asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar(FIRST + s)), "r"(BYTES) : "memory");
                    else
#endif
                    mbar_arrive_expect_tx(bar(FIRST + s), BYTES);
                }
                __syncwarp();
                const int y = ((t0 + k) * BC + (box << bp_shift)) & ((1 << a.ps_shift) - 1);
                if (mine) {
                    if constexpr (FP8)
                        tma_load_3d_hint(sbase + C::OFF_RAW + s * C::RAW_TILE + (uint32_t)((box << bp_shift) * D), map, bar(FIRST + s), 0, y, z,
                                         policy);
                    else
                        tma_load_4d_hint(sbase + C::OFF_SLOT + s * C::KV_TILE + (uint32_t)(ch * C::KV_CHUNK + (box << bp_shift) * 128), map,
                                         bar(FIRST + s), 0, y, ch, z, policy);
                }
                ++loads;
                return true;
            };
            // pages of the next K tile are read ahead; V's are those of K two tiles before
            int zk = place_of(0), z1 = nowhere, z2 = nowhere;   // of K(k); of K(k - 1) and K(k - 2)
            walk_ops(
                n,
                [&](int k) {
                    const int z = zk;
                    zk = place_of(k + 1);
                    z2 = z1;
                    z1 = z;
                    return load(&tm_k, k, z);
                },
                [&](int k) { return load(&tm_v, k, k + 1 < n ? z2 : z1); });
            // every copy lands before the CTA exits, whoever gave up
            for (uint32_t i = loads > (uint32_t)RING ? loads - RING : 0; i < loads; ++i)
                mbar_wait_drain(bar(FIRST + i % RING), (i / RING) & 1);
        } else if (warp <= (uint32_t)nq && lane == 0) {
            // ---------------------------------------------------- products of query tile t
            const int t = (int)warp - 1;
            const uint32_t s_col = tmem + C::S_COL + t * BC, o_col = tmem + C::O_COL + t * D;
            const uint64_t qd = sdesc_sw128(sbase + C::OFF_Q + t * C::Q_TILE, 16, 1024);
            const uint64_t pd = sdesc_sw128(sbase + C::OFF_P + t * C::P_TILE, 16, 1024);
            uint32_t ld = 0;
            auto acquire = [&](uint32_t &slot) {
                slot = ld % NSLOT;
                const bool r = mbar_wait<true>(bar(C::B_FULL + slot), (ld / NSLOT) & 1, ctx, SITE_X_FULL);
                ++ld;
                return r;
            };
            if (mbar_wait<true>(bar(C::B_QFULL + t), 0, ctx, SITE_X_QFULL))
                walk_ops(
                    n,
                    [&](int k) -> bool {
                        uint32_t s;
                        if (!acquire(s))
                            return false;
                        if (k > 0 && !mbar_wait<true>(bar(C::B_SFREE + t), (k - 1) & 1, ctx, SITE_X_SFREE))
                            return false;
                        tc_fence_after();
                        const uint64_t kd = sdesc_sw128(sbase + C::OFF_SLOT + s * C::KV_TILE, 16, 1024);
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk)
                            mma_ss(s_col, qd + (((kk >> 2) * C::Q_CHUNK + (kk & 3) * 32) >> 4),
                                   kd + (((kk >> 2) * C::KV_CHUNK + (kk & 3) * 32) >> 4), C::IDESC_S, kk > 0 ? 1u : 0u);
                        tc_commit(bar(C::B_SFULL + t));
                        tc_commit(bar(C::B_EMPTY + s));
                        return true;
                    },
                    [&](int k) -> bool {
                        uint32_t s;
                        if (!acquire(s) || !mbar_wait<true>(bar(C::B_PFULL + t), k & 1, ctx, SITE_X_PFULL))
                            return false;
                        tc_fence_after();
                        const uint64_t vd = sdesc_sw128(sbase + C::OFF_SLOT + s * C::KV_TILE, C::KV_CHUNK, 1024);
#pragma unroll
                        for (int kk = 0; kk < BC / 16; ++kk)
                            mma_ss(o_col, pd + (((kk >> 2) * C::P_CHUNK + (kk & 3) * 32) >> 4), vd + ((kk * 16 * 128) >> 4), C::IDESC_PV,
                                   k > 0 || kk > 0 ? 1u : 0u);
                        tc_commit(bar(C::B_ODONE + t));   // O~ current and P read
                        tc_commit(bar(C::B_EMPTY + s));
                        return true;
                    });
            tc_commit(bar(C::B_DRAIN + t));   // all products complete before tensor memory is released
            mbar_wait_drain(bar(C::B_DRAIN + t), 0);
        }
        __syncwarp();
    } else if (FP8 && warp >= 4 + 4 * NQ) {
        if constexpr (FOUR)
            regs_dealloc<96>();
        // -------------------------------------------------------- codes to bf16, in the loads' order
        const int tid = (int)threadIdx.x - (128 + 128 * NQ);
        constexpr int UNITS = D / 16;   // 16-code pieces of a row
        for (uint32_t i = 0; i < 2u * (uint32_t)n; ++i) {
            const uint32_t r = i % NRAW, s = i % NSLOT;
            if (!mbar_wait_warp<true>(bar(C::B_RFULL + r), (i / NRAW) & 1, ctx, SITE_X_RFULL) ||
                (i >= (uint32_t)NSLOT && !mbar_wait_warp<true>(bar(C::B_EMPTY + s), (i / NSLOT - 1) & 1, ctx, SITE_X_EMPTY)))
                break;
            const uint8_t *src = smem + C::OFF_RAW + r * C::RAW_TILE;
            uint8_t *dst = smem + C::OFF_SLOT + s * C::KV_TILE;
#pragma unroll 4
            for (int e = tid; e < BC * UNITS; e += 128) {
                const int row = e / UNITS, u = e % UNITS;   // features 16 u .. 16 u + 15: two 16-byte units of chunk u / 4
                uint4 lo, hi;
                codes_to_bf16(*reinterpret_cast<const uint4 *>(src + row * D + u * 16), lo, hi);
                uint8_t *at = dst + (u >> 2) * C::KV_CHUNK + row * 128;
                *reinterpret_cast<uint4 *>(at + (((2 * (u & 3)) ^ (row & 7)) << 4)) = lo;
                *reinterpret_cast<uint4 *>(at + (((2 * (u & 3) + 1) ^ (row & 7)) << 4)) = hi;
            }
            mbar_arrive(bar(C::B_REMPTY + r));
            fence_smem_to_async();
            mbar_arrive(bar(C::B_FULL + s));
        }
    } else if ((int)(warp - 4) / 4 < nq) {
        if constexpr (SPLIT)
            regs_alloc<FOUR ? 176 : 200>();
        // -------------------------------------------------------- softmax of query tile t: a thread a row
        const int t = (int)(warp - 4) >> 2;
        const uint32_t quarter = warp & 3u;
        const int rit = (int)(quarter * 32 + lane), r = row0 + t * BR + rit;
        const uint32_t lane_base = tmem + ((quarter * 32u) << 16);
        const bool alive = row0 + t * BR + (int)quarter * 32 < a.R;   // the warp has a row
        int lim = 0;   // entries of the prefix that the row sees
        {
            const int b = r / a.GT, i = r - b * a.GT;   // sequence, and row of its head group
            long long src = -1;
            if (r < a.R) {
                const int len = a.lens[b];
                lim = len < 0 || len > a.cap ? 0 : min(a.P, max(0, a.causal ? len - a.Tq + i % a.Tq + 1 : len));
                src = (((long long)b * a.Hq + (long long)h * a.G) * a.Tq + i) * D;
            }
            // the warp's rows, D / 8 lanes a row: whole lines (a thread's own row would be 32 lines a load)
            constexpr int LPR = D / 8, RPL = 32 / LPR;
            uint8_t *qt = smem + C::OFF_Q + t * C::Q_TILE;
#pragma unroll 8
            for (int k = 0; k < LPR; ++k) {
                const int row = k * RPL + (int)lane / LPR, u = (int)lane % LPR, at = (int)quarter * 32 + row;
                const long long from = __shfl_sync(0xffffffffu, src, row);
                const uint4 v = from >= 0 ? *reinterpret_cast<const uint4 *>(a.q + from + u * 8) : make_uint4(0, 0, 0, 0);
                *reinterpret_cast<uint4 *>(qt + (u >> 3) * C::Q_CHUNK + at * 128 + (((u & 7) ^ (at & 7)) << 4)) = v;
            }
            fence_smem_to_async();
            mbar_arrive(bar(C::B_QFULL + t));
        }
        float sl2 = a.scale_log2;
        if constexpr (FP8) {   // a normal number, so that a masked entry's -inf stays one; a NaN of the scale stays
            const float ks = a.ks[h];
            sl2 = isnan(ks) ? ks : fminf(fmaxf(sl2 * ks, FLT_MIN), FLT_MAX);
        }
        // whether the pages of a tile's groups of 16 entries are there: lane i reads group i's
        auto page_of = [&](int k) {
            const int slot = (t0 + k) * BC + 16 * (int)(lane % (BC / 16));
            return k < n && slot < a.P ? __ldg(a.pages + (slot >> a.ps_shift)) : 0;
        };
        int page = alive ? page_of(0) : 0;
        float m = -INFINITY, l = 0.f;
        bool ok = true;
        for (int k = 0; k < n; ++k) {
            if (!mbar_wait_warp<true>(bar(C::B_SFULL + t), k & 1, ctx, SITE_X_SFULL)) {
                ok = false;
                break;
            }
            if (!alive) {   // in step with the others
                mbar_arrive(bar(C::B_SFREE + t));
                if (k > 0 && !mbar_wait_warp<true>(bar(C::B_ODONE + t), (k - 1) & 1, ctx, SITE_X_ODONE)) {
                    ok = false;
                    break;
                }
                mbar_arrive(bar(C::B_PFULL + t));
                continue;
            }
            tc_fence_after();
            uint32_t sv[BC / 32][32];
#pragma unroll
            for (int c = 0; c < BC / 32; ++c)
                tmem_ld_x32_nowait(lane_base + C::S_COL + t * BC + c * 32, sv[c]);
#pragma unroll
            for (int c = 0; c < BC / 32; ++c)
                tmem_wait_ld_x32(sv[c]);
            tc_fence_before();
            mbar_arrive(bar(C::B_SFREE + t));   // S is in registers: the next may overwrite it
            float s[BC];
#pragma unroll
            for (int c = 0; c < BC / 32; ++c)
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    s[c * 32 + i] = __uint_as_float(sv[c][i]);
            const uint32_t gone = __ballot_sync(0xffffffffu, page < 0 || page >= a.num_pages) & ((1u << (BC / 16)) - 1u);
            page = page_of(k + 1);
            const int here = lim - (t0 + k) * BC;   // entries of the tile that the row sees
            if (__any_sync(0xffffffffu, here < BC) || gone) {
#pragma unroll
                for (int i = 0; i < BC; ++i)
                    if (i >= here || ((gone >> (i / 16)) & 1u))
                        s[i] = -INFINITY;
            }
            float mx0 = -INFINITY, mx1 = -INFINITY, mx2 = -INFINITY, mx3 = -INFINITY;
#pragma unroll
            for (int i = 0; i < BC; i += 8) {
                mx0 = fmax3(mx0, s[i], s[i + 1]);
                mx1 = fmax3(mx1, s[i + 2], s[i + 3]);
                mx2 = fmax3(mx2, s[i + 4], s[i + 5]);
                mx3 = fmax3(mx3, s[i + 6], s[i + 7]);
            }
            const float m_new = fmaxf(m, fmax3(mx0, mx1, fmaxf(mx2, mx3)));
            const bool resc = m != -INFINITY && (m_new - m) * sl2 > kRescaleLog2;
            float alpha = 1.f;
            if (m == -INFINITY) {
                m = m_new;   // O~ and l of the row are still 0
            } else if (resc) {
                alpha = ex2_approx((m - m_new) * sl2);
                l *= alpha;
                m = m_new;
            }
            const float mref = m == -INFINITY ? 0.f : m * sl2;
            float l0 = 0.f, l1 = 0.f, l2 = 0.f, l3 = 0.f;
            uint32_t pb[BC / 2];
#pragma unroll
            for (int i = 0; i < BC; i += 4) {
                float x0, x1, x2, x3;
                ffma2(x0, x1, s[i], s[i + 1], sl2, sl2, -mref, -mref);
                ffma2(x2, x3, s[i + 2], s[i + 3], sl2, sl2, -mref, -mref);
                x0 = ex2_approx(x0);
                x1 = ex2_approx(x1);
                x2 = ex2_approx(x2);
                x3 = ex2_approx(x3);
                fadd2(l0, l1, l0, l1, x0, x1);
                fadd2(l2, l3, l2, l3, x2, x3);
                pb[i / 2] = pack_bf16x2(x0, x1);
                pb[i / 2 + 1] = pack_bf16x2(x2, x3);
            }
            // the product before has read P, and O~ holds it
            if (k > 0 && !mbar_wait_warp<true>(bar(C::B_ODONE + t), (k - 1) & 1, ctx, SITE_X_ODONE)) {
                ok = false;
                break;
            }
            uint8_t *prow = smem + C::OFF_P + t * C::P_TILE + rit * 128;
#pragma unroll
            for (int c = 0; c < C::PCH; ++c)
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    *reinterpret_cast<uint4 *>(prow + c * C::P_CHUNK + ((u ^ (rit & 7)) << 4)) =
                        make_uint4(pb[c * 32 + 4 * u], pb[c * 32 + 4 * u + 1], pb[c * 32 + 4 * u + 2], pb[c * 32 + 4 * u + 3]);
            l += (l0 + l2) + (l1 + l3);
            if (__any_sync(0xffffffffu, resc)) {
                tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t ov[32];
                    tmem_ld_x32(lane_base + C::O_COL + t * D + c * 32, ov);
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        float y0, y1;
                        fmul2(y0, y1, __uint_as_float(ov[i]), __uint_as_float(ov[i + 1]), alpha, alpha);
                        ov[i] = __float_as_uint(y0);
                        ov[i + 1] = __float_as_uint(y1);
                    }
                    tmem_st_x32(lane_base + C::O_COL + t * D + c * 32, ov);
                }
            }
            fence_smem_to_async();
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(bar(C::B_PFULL + t));
        }
        // the row's state: O~ through the tile's P buffer, which no product reads any more, so that a warp writes
        // whole lines (4 rows of 32 features at a time)
        if (ok && mbar_wait_warp<true>(bar(C::B_ODONE + t), (n - 1) & 1, ctx, SITE_X_ODONE) && alive) {
            tc_fence_after();
            const long long at = ((long long)(h * a.RP + rp) * a.runs + run) * (NQ * BR) + t * BR + (int)quarter * 32;   // the warp's first row
            uint8_t *stage = smem + C::OFF_P + t * C::P_TILE + quarter * 4096;
            const float f = FP8 ? a.vs[h] : 1.f;
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                uint32_t v[32];
                tmem_ld_x32(lane_base + C::O_COL + t * D + c * 32, v);
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    *reinterpret_cast<float4 *>(stage + lane * 128 + ((u ^ (lane & 7)) << 4)) =
                        make_float4(__uint_as_float(v[4 * u]) * f, __uint_as_float(v[4 * u + 1]) * f, __uint_as_float(v[4 * u + 2]) * f,
                                    __uint_as_float(v[4 * u + 3]) * f);
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int row = 4 * i + (int)(lane >> 3), u = (int)(lane & 7);
                    if (row0 + t * BR + (int)quarter * 32 + row < a.R)
                        *reinterpret_cast<float4 *>(a.part + (at + row) * D + c * 32 + 4 * u) =
                            *reinterpret_cast<const float4 *>(stage + row * 128 + ((u ^ (row & 7)) << 4));
                }
                __syncwarp();
            }
            if (r < a.R)
                reinterpret_cast<float2 *>(a.part + a.ml_at)[at + lane] = make_float2(m == -INFINITY ? -INFINITY : m * sl2, l);
        }
    }
    // ------------------------------------------------------------ teardown
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, C::TMEM_COLS);
    }
}

// ------------------------------------------------------------------ join
struct PrefixJoinArgs {
    const float *part;     // states of the runs
    long long ml_at;
    OwnStates own;
    __nv_bfloat16 *o;
    float *lse;
    int Hq, G, Tq, GT, RP, runs, rows;   // rows: of a CTA of the attention
    long long n;           // rows of o
};

// x / y of nonnegative values, which seldom have more than 32 bits.
__device__ __forceinline__ long long quotient(long long x, long long y)
{
    return ((x | y) >> 32) == 0 ? (long long)((uint32_t)x / (uint32_t)y) : x / y;
}

// W warps a row: each takes every W-th state (the runs', then the own entries'), a lane D / 32 features; then the
// warps' sums.  The first states of each warp are under way before anything is known of them.
template <int D, int W>
__global__ void __launch_bounds__(128) prefix_join_kernel(const __grid_constant__ PrefixJoinArgs a)
{
    constexpr int F = D / 32, AHEAD = D == 256 ? 4 : 8;   // divides 32
    __shared__ float sum[W == 1 ? 1 : 4][D], red[4];
    pdl_launch();
    const int warp = (int)warp_id() % W, lane = (int)lane_id();
    // 32-bit divisions: those of 64 bits were 3 us of it
    const uint32_t row32 = blockIdx.x * (4 / W) + warp_id() / W;   // (b Hq + head) Tq + t
    const long long row = row32;
    if (row >= a.n) {
        pdl_wait();
        return;
    }
    const uint32_t bh = row32 / (uint32_t)a.Tq, b32 = bh / (uint32_t)a.Hq;
    const int t = (int)(row32 - bh * (uint32_t)a.Tq), head = (int)(bh - b32 * (uint32_t)a.Hq), b = (int)b32;
    const int h = head / a.G, i = (head - h * a.G) * a.Tq + t, r = b * a.GT + i;   // KV head, row of its group, of its matrix
    const long long at = (long long)(h * a.RP + r / a.rows) * a.runs * a.rows + r % a.rows;
    // The lengths may be read in front of the wait, past the L1: this kernel is launched when every CTA of the prefix's
    // is past its own wait.  Behind it, everything whose place is known goes together, the own entries' state as if it were whole
    int len = __ldcg(a.own.lens + b);
    len = len < 0 || len > a.own.cap ? 0 : len;
    pdl_wait();
    const long long where0 = a.own.whole ? 0 : __ldcg(a.own.where), where1 = a.own.whole ? 0 : __ldcg(a.own.where + 1 + b);
    const float lse0 = __ldcg(a.own.lse + row);
    float z[F];
#pragma unroll
    for (int f = 0; f < F; f += 2)
        *reinterpret_cast<float2 *>(&z[f]) = __ldcg(reinterpret_cast<const float2 *>(a.own.o + row * D + lane * F + f));
    const float2 *ml = reinterpret_cast<const float2 *>(a.part + a.ml_at) + at;
    auto run_o = [&](int s) { return a.part + (at + (long long)s * a.rows) * D + lane * F; };
    // this warp's states are the runs warp, warp + W, ...; lane j has (m, l) of the j-th of 32 at a time
    const int mine = (a.runs - warp + W - 1) / W;
    float y[AHEAD][F];
    auto fetch = [&](int u, int k) {   // the k-th of them
        if (k < mine)
#pragma unroll
            for (int f = 0; f < F; f += 2)
                *reinterpret_cast<float2 *>(&y[u][f]) = __ldcg(reinterpret_cast<const float2 *>(run_o(warp + W * k) + f));
    };
#pragma unroll
    for (int u = 0; u < AHEAD; ++u)
        fetch(u, u);
    const float2 none = make_float2(-INFINITY, 0.f);
    const float2 st0 = lane < mine ? __ldcg(&ml[(long long)(warp + W * lane) * a.rows]) : none;
    float m = -INFINITY;
    for (int s = lane; s < a.runs; s += 32)
        m = fmaxf(m, __ldcg(&ml[(long long)s * a.rows]).x);
    // the own entries' states: none, one that is whole, or those of CTAs c0 .. c0 + own - 1
    int own = 0;
    bool whole = false;
    const float *first = nullptr, *rest = nullptr;    // slots of the first CTA and, two apart, of those behind it
    const int rb = i / a.own.rows, ri = i - rb * a.own.rows;
    const long long stride = (long long)a.own.rows * (D + 2);
    const int from = min(a.own.base, len) / a.own.kt, nt = a.own.base < len ? (len + a.own.kt - 1) / a.own.kt - from : 0;
    if (nt > 0) {
        const long long share = where0;
        whole = share == 0;
        if (!whole) {
            const long long tile = where1 + (long long)(rb * a.own.Hkv + h) * nt;
            const long long c0 = quotient(tile, share), c1 = quotient(tile + nt - 1, share);
            whole = c0 == c1;
            own = (int)(c1 - c0) + 1;
            first = a.own.part + (2 * c0 + (tile == c0 * share ? 0 : 1)) * stride;
            rest = a.own.part + 2 * c0 * stride;
        }
        if (whole)
            own = 1;
    }
    auto own_slot = [&](int s) { return s == 0 ? first : rest + 2 * s * stride; };
    auto own_ml = [&](int s) {
        return whole ? make_float2(lse0 * 1.4426950408889634f, 1.f)
                     : make_float2(own_slot(s)[(long long)a.own.rows * D + ri], own_slot(s)[(long long)a.own.rows * (D + 1) + ri]);
    };
    for (int s = lane; s < own; s += 32)
        m = fmaxf(m, own_ml(s).x);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    const float ref = m == -INFINITY ? 0.f : m;
    float l = 0.f, x[F];
#pragma unroll
    for (int f = 0; f < F; ++f)
        x[f] = 0.f;
    for (int base = 0; base < mine; base += 32) {
        const float2 st = base == 0 ? st0 : base + lane < mine ? __ldcg(&ml[(long long)(warp + W * (base + lane)) * a.rows]) : none;
        const float w = st.x == -INFINITY ? 0.f : ex2_approx(st.x - ref);
        l = fmaf(w, st.y, l);   // each lane its states'; put together below
        for (int k0 = base; k0 < min(base + 32, mine); k0 += AHEAD) {
#pragma unroll
            for (int u = 0; u < AHEAD; ++u) {
                const float wu = __shfl_sync(0xffffffffu, w, (k0 + u) & 31);
                // a state that saw nothing may hold anything
                if (k0 + u < min(base + 32, mine) && wu != 0.f)
#pragma unroll
                    for (int f = 0; f < F; ++f)
                        x[f] = fmaf(wu, y[u][f], x[f]);
            }
#pragma unroll
            for (int u = 0; u < AHEAD; ++u)
                fetch(u, k0 + AHEAD + u);
        }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
        l += __shfl_xor_sync(0xffffffffu, l, off);
    for (int s = warp; s < own; s += W) {
        const float2 st = own_ml(s);
        if (st.x == -INFINITY)
            continue;
        const float w = ex2_approx(st.x - ref);
        l = fmaf(w, st.y, l);
        if (!whole) {
            const float *src = own_slot(s) + (long long)ri * D + lane * F;
#pragma unroll
            for (int f = 0; f < F; f += 2)
                *reinterpret_cast<float2 *>(&z[f]) = __ldcg(reinterpret_cast<const float2 *>(src + f));
        }
#pragma unroll
        for (int f = 0; f < F; ++f)
            x[f] = fmaf(w, z[f], x[f]);
    }
    if constexpr (W == 1) {
        const float inv = l == 0.f ? 0.f : 1.f / l;
        uint32_t *dst = reinterpret_cast<uint32_t *>(a.o + row * D) + lane * (F / 2);
#pragma unroll
        for (int f = 0; f < F; f += 2)
            dst[f / 2] = pack_bf16x2(x[f] * inv, x[f + 1] * inv);
    } else {
#pragma unroll
        for (int f = 0; f < F; ++f)
            sum[warp][lane * F + f] = x[f];
        if (lane == 0)
            red[warp] = l;
        __syncthreads();
        l = (red[0] + red[1]) + (red[2] + red[3]);
        const float inv = l == 0.f ? 0.f : 1.f / l;
        for (int f = 2 * (int)threadIdx.x; f < D; f += 256) {
            const float u = (sum[0][f] + sum[1][f]) + (sum[2][f] + sum[3][f]);
            const float v = (sum[0][f + 1] + sum[1][f + 1]) + (sum[2][f + 1] + sum[3][f + 1]);
            *reinterpret_cast<uint32_t *>(a.o + row * D + f) = pack_bf16x2(u * inv, v * inv);
        }
    }
    if (warp == 0 && lane == 0)
        a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994530942f;
}

// ------------------------------------------------------------------ host
size_t round256(size_t x) { return (x + 255) & ~(size_t)255; }

// How the rows and the prefix are cut: rows of a CTA, CTAs of a KV head's rows, runs of the prefix's tiles.
struct Cut {
    int rows, rp, tiles, runs;
};

Cut cut_of(int B, int Hq, int Hkv, int Tq, int d, long long P)
{
    Cut c;
    c.rows = d == 256 ? BR : 2 * BR;
    const long long R = (long long)B * (Hq / Hkv) * Tq;
    c.rp = (int)((R + c.rows - 1) / c.rows);
    const int bc = d == 256 ? 64 : 128;
    c.tiles = (int)((P + bc - 1) / bc);
    // As many runs as take the least time in passes of one CTA an SM, a run's start and its state costing about two
    // tiles
    const long long units = (long long)Hkv * c.rp;
    long long best = LLONG_MAX;
    c.runs = 1;
    for (int s = 1; s <= c.tiles && s <= 2 * kSMs; ++s) {
        const long long passes = (units * s + kSMs - 1) / kSMs, time = passes * ((c.tiles + s - 1) / s + 2);
        if (time < best) {
            best = time;
            c.runs = s;
        }
        if (units * s >= 4 * kSMs)
            break;
    }
    return c;
}

size_t part_floats(const Cut &c, int Hkv, int d) { return (size_t)Hkv * c.rp * c.runs * c.rows * (d + 2); }

template <int D, bool FP8>
int prefix_run(const fa_kv_cache &c, const PrefixArgs &a, cudaStream_t s)
{
    using C = XCfg<D, FP8>;
    CUtensorMap tk, tv;
    const uint64_t pages = (uint64_t)c.num_pages * c.Hkv;
    const uint32_t rows = (uint32_t)std::min(c.page_size, C::BC);
    for (int i = 0; i < 2; ++i) {
        int st;
        if (FP8) {   // codes, plain
            const uint64_t dims[3] = {(uint64_t)D, (uint64_t)c.page_size, pages};
            const uint64_t strides[2] = {(uint64_t)D, (uint64_t)c.page_size * D};
            const uint32_t box[3] = {(uint32_t)D, rows, 1};
            st = encode_tmap(i ? &tv : &tk, i ? c.v : c.k, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_NONE);
        } else {     // [page, KV head][64 features][row]
            const uint64_t dims[4] = {64, (uint64_t)c.page_size, (uint64_t)C::KCH, pages};
            const uint64_t strides[3] = {(uint64_t)D * 2, 128, (uint64_t)c.page_size * D * 2};
            const uint32_t box[4] = {64, rows, 1, 1};
            st = encode_tmap(i ? &tv : &tk, i ? c.v : c.k, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
        }
        if (st != OK)
            return st;
    }
    if (const int st = allow_smem<prefix_kernel<D, FP8>>(C::SMEM); st != OK)
        return st;
    return launch_overlapped(prefix_kernel<D, FP8>, dim3((unsigned)(a.Hkv * a.runs * a.RP)), C::NTHREADS, C::SMEM, 0, true, s, tk, tv, a);
}

// A warp a row where it has few states or where there are rows for all SMs.
template <int D>
int join_run(const PrefixJoinArgs &j, cudaStream_t s)
{
    const bool one = j.runs <= 8 || j.n >= 2048;
    return launch_overlapped(one ? prefix_join_kernel<D, 1> : prefix_join_kernel<D, 4>, dim3((unsigned)(one ? (j.n + 3) / 4 : j.n)), 128, 0, 0, true, s,
                             j);
}

}  // namespace

// Whether the prefix by itself is faster than every sequence reading it: estimates of both, less what they have in
// common, fitted to 1762 pairs of measurements (1 to 90 sequences, prefixes of 64 to 24576 entries, 1 to 256 rows a KV
// head, all widths and types) and held against 1260 more (1 to 8 sequences, 12288 to 196608 entries): the choice is 1.9%
// and 1.0% slower than the better of the two on average, 48% and 55% at worst, where both take 13 to 25 us.  Without it,
// the sequences' rows times entries count (at least eight rows, the columns of a product), the bytes, which come out of
// L2 up to some 90 MB, and the row tiles; with it, its bytes and the rows' states, and where it is long in e4m3 the
// conversion of its codes, by tiles of 128 entries an SM.  (8 KV heads of 64 over 196608 entries, two sequences: 80 us
// without, 160 with; the long ones in e4m3 were 4.9% slower on average, 99% at worst, before that term, 0.8% and 43% now.)
// us without and with, 8 KV heads of 128 and 4 query heads each, batch x entries: 2 x 8192 15.1 and 17.3, 4 x 512 10.2
// and 11.9, 4 x 8192 20.5 and 18.5, 16 x 2048 21.1 and 15.0, 64 x 128 11.5 and 19.7, 64 x 8192 177 and 31; 3 KV heads of
// 128 with 56 rows each, 1 x 2048 15.2 and 12.5, 6 x 8192 (e4m3) 35.0 and 23.5, 64 x 2048 86.0 and 37.8.
// (The test library computes it by itself whatever the sizes.)
bool prefix_pays(const fa_kv_cache &c, int Hq, int Tq, int n_pages)
{
    if (FA_TEST_WITHHOLD)
        return true;
    const bool f8 = c.dtype == FA_E4M3;
    const double P = (double)n_pages * c.page_size, once = P * c.Hkv * 2 * c.d * (f8 ? 1 : 2) * 1e-6;   // MB
    const int M = Hq / c.Hkv * Tq, blocks = (M + 63) / 64;
    const double pairs = c.B * P * c.Hkv * std::max(M, 8) * c.d * 1e-9;
    const double without = 0.9 * std::min(M, 64) / 16 + 0.022 * blocks * c.B * once + (f8 ? 16 : 40) * pairs +
                           0.1 * (c.B - 1) * std::max(0.0, once - 90);
    const double codes = f8 ? 0.8 * std::max(0.0, P * c.Hkv / 128 / kSMs - 1) : 0;
    return without >= 3.7 + 0.8 * ((double)c.B * Hq * Tq * c.d / 128e3) + 0.19 * once + codes;
}

// Behind one another: the own entries' workspace, their o (fp32) and lse, the runs' states.
size_t prefix_workspace_bytes(int B, int Hq, int Hkv, int Tq, int max_len, int d, int codes, int n_pages, int page_size)
{
    const size_t rows = (size_t)B * Hq * Tq;
    const Cut c = cut_of(B, Hq, Hkv, Tq, d, (long long)n_pages * page_size);
    return round256(paged_workspace_bytes(B, Hq, Hkv, Tq, max_len, d, 0)) + round256(rows * d * 4) + round256(rows * 4) +
           (n_pages > 0 ? round256(part_floats(c, Hkv, d) * 4) : 0);
}

int prefix_launch(const fa_kv_cache &c, const void *q, void *o, float *lse, int Hq, int Tq, int causal, const int *pages,
                  int n_pages, float scale, void *workspace, cudaStream_t s)
{
    const int P = n_pages * c.page_size, B = c.B;
    const size_t rows = (size_t)B * Hq * Tq;
    const bool f8 = c.dtype == FA_E4M3;
    const Cut cut = cut_of(B, Hq, c.Hkv, Tq, c.d, P);
    if ((long long)c.Hkv * cut.rp * cut.runs > INT_MAX || rows > INT_MAX)
        return ERR_UNSUPPORTED;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    uint8_t *own = ws + round256(paged_workspace_bytes(B, Hq, c.Hkv, Tq, c.max_pages * c.page_size, c.d, 0));
    float *own_lse = reinterpret_cast<float *>(own + round256(rows * c.d * 4));
    float *part = reinterpret_cast<float *>(reinterpret_cast<uint8_t *>(own_lse) + round256(rows * 4));
    status_in_use(STATUS_PREFIX);
    PrefixArgs a{};
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.ks = c.k_scale;
    a.vs = c.v_scale;
    a.pages = pages;
    a.lens = c.lens;
    a.part = part;
    a.ml_at = (long long)c.Hkv * cut.rp * cut.runs * cut.rows * c.d;
    a.B = B;
    a.Hq = Hq;
    a.Hkv = c.Hkv;
    a.G = Hq / c.Hkv;
    a.Tq = Tq;
    a.GT = a.G * Tq;
    a.R = B * a.GT;
    a.RP = cut.rp;
    a.causal = causal;
    a.P = P;
    a.num_pages = c.num_pages;
    while ((1 << a.ps_shift) < c.page_size)
        ++a.ps_shift;
    a.cap = c.max_pages * c.page_size;
    a.runs = cut.runs;
    a.run_tiles = cut.tiles / cut.runs;
    a.run_more = cut.tiles % cut.runs;
    a.scale_log2 = std::min(scale * 1.4426950408889634f, FLT_MAX);
    a.timeout_ns = wait_timeout_ns();
    a.withhold = WITHHOLD_NONE;
#if FA_TEST_WITHHOLD
    a.withhold = test_withhold_take(WITHHOLD_PREFIX_FULL, WITHHOLD_PREFIX_FULL);
#endif
    // the own entries first: the memory bounds them, and the prefix's CTAs take the SMs as they are done
    OwnStates states;
    int st = paged_behind_launch(c, q, reinterpret_cast<float *>(own), own_lse, Hq, Tq, causal, P, scale, workspace, &states, s);
    if (st == OK)
        st = c.d == 64    ? (f8 ? prefix_run<64, true>(c, a, s) : prefix_run<64, false>(c, a, s))
             : c.d == 128 ? (f8 ? prefix_run<128, true>(c, a, s) : prefix_run<128, false>(c, a, s))
                          : (f8 ? prefix_run<256, true>(c, a, s) : prefix_run<256, false>(c, a, s));
    if (st != OK)
        return st;
    PrefixJoinArgs j{part, a.ml_at, states, static_cast<__nv_bfloat16 *>(o), lse, Hq, a.G, Tq, a.GT, a.RP, a.runs, cut.rows,
                     (long long)rows};
    return c.d == 64 ? join_run<64>(j, s) : c.d == 128 ? join_run<128>(j, s) : join_run<256>(j, s);
}

int prefix_status_fetch_clear(cudaStream_t s, int *host_word)
{
    int word[2] = {0, 0};
    if (cudaMemcpyFromSymbolAsync(word, g_prefix_status, sizeof(word), 0, cudaMemcpyDeviceToHost, s) != cudaSuccess ||
        cudaStreamSynchronize(s) != cudaSuccess)
        return ERR_CUDA;
    *host_word = word[0] ? word[0] : word[1];
    const int zero[2] = {0, 0};
    if (*host_word != 0 &&
        (cudaMemcpyToSymbolAsync(g_prefix_status, zero, sizeof(zero), 0, cudaMemcpyHostToDevice, s) != cudaSuccess ||
         cudaStreamSynchronize(s) != cudaSuccess))
        return ERR_CUDA;
    return OK;
}

}  // namespace fa
