// fa_cache_sm103.cu -- rotary positions with several axes, the write of new tokens into the
// paged key/value cache, and eviction from it by accumulated attention weight (sm_103a).
//
// Rotation.  Pair i of a row turns by theta = p f_i (p the token's position on the pair's
// axis).  Only theta modulo one turn matters, so f_i / 2 pi is held as a 64-bit fraction of a
// turn: p times it, in wrapping 64-bit integer arithmetic, is the angle modulo one turn with no
// reduction at all and an error of p 2^-65 turns, at any position.  The two top bits (rounded)
// are the quadrant, the rest an angle in [-pi/4, pi/4], where the Taylor series of sine and
// cosine are below half an fp32 ulp after x^9 and x^10.
//
// What bounds these kernels is memory: a rotation reads and writes each element once.  A thread
// owns 8 pairs of one token (two 16-byte loads in bf16), computes their sines and cosines once
// and runs over the heads with them.
#include <climits>

#include "fa_common.cuh"
#include "fa_internal.h"
#include "fa_pdl.cuh"
#include "fa_rope.cuh"

namespace fa {

__device__ int g_cache_status;   // device status word of the kernels in this file

namespace {

constexpr int kStatusBadIndex = 5;

// ------------------------------------------------------------------ rotation
struct RopeArgs {
    Row3 x[2], y[2];
    int H0, H;            // heads of the first tensor, of both
    const int *pos;       // [axes][n]
    long long n;          // B * T
    int T, rot, heads_per_cta, groups;   // head groups
    float sign;
};

template <typename E, int D, bool INTER>
__global__ void __launch_bounds__(kRopeThreads, 2) rope_kernel(const __grid_constant__ RopeTable tab,
                                                            const __grid_constant__ RopeArgs a)
{
    constexpr int TPR = D / 16;                          // threads a row
    pdl_launch();
    pdl_wait();
    const int v = threadIdx.x % TPR;
    // head groups next to one another: CTAs that run together read whole token rows of a packed
    // projection
    const int tile = (int)(blockIdx.x / a.groups), group = (int)blockIdx.x - tile * a.groups;
    const long long tok = (long long)tile * (kRopeThreads / TPR) + threadIdx.x / TPR;
    if (tok >= a.n)
        return;
    const int b = (int)tok / a.T, t = (int)tok - b * a.T;
    const Slice sl = slice_of(v, a.rot, INTER);
    float sn[8], cs[8];
    if (sl.pair >= 0) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int p = a.pos[(long long)tab.axis[sl.pair + j] * a.n + tok];
            phase_sincos(tab.turns[sl.pair + j], p, sn[j], cs[j]);
            sn[j] *= a.sign;
        }
    }
    const int h0 = group * a.heads_per_cta, h1 = min(a.H, h0 + a.heads_per_cta);
#pragma unroll
    for (int w = 0; w < 2; ++w) {   // the group's heads of either tensor
        const int first = max(h0 - (w ? a.H0 : 0), 0), last = min(h1 - (w ? a.H0 : 0), w ? a.H - a.H0 : a.H0);
        if (first >= last)
            continue;
        const Row3 &xi = a.x[w], &yi = a.y[w];
        const E *x = static_cast<const E *>(xi.p) + b * xi.sb + first * xi.sh + t * xi.st;
        E *y = static_cast<E *>(yi.p) + b * yi.sb + first * yi.sh + t * yi.st + sl.e0;
        const int gap = sl.e1 - sl.e0;
        each_head(x, xi.sh, last - first, sl, [&](int, float(&f)[8], float(&g)[8]) {
            if (sl.pair >= 0)
                turn<INTER>(f, g, sn, cs);
            store8(y, f);
            store8(y + gap, g);
            y += yi.sh;
        });
    }
}

template <typename E, int D>
int rope_run(const RopeTable &t, const RopeArgs &a, int interleaved, cudaStream_t s)
{
    constexpr int TOK = kRopeThreads / (D / 16);
    const dim3 grid((unsigned)((a.n + TOK - 1) / TOK * a.groups));
    return launch_overlapped(interleaved ? rope_kernel<E, D, true> : rope_kernel<E, D, false>, grid, kRopeThreads, 0, 0, true, s, t, a);
}

template <typename E>
int rope_width(int d, const RopeTable &t, const RopeArgs &a, int interleaved, cudaStream_t s)
{
    return d == 64 ? rope_run<E, 64>(t, a, interleaved, s)
                   : d == 128 ? rope_run<E, 128>(t, a, interleaved, s) : rope_run<E, 256>(t, a, interleaved, s);
}

// ------------------------------------------------------------------ append
struct AppendArgs {
    Row3 q, qo, k, v;
    NormArgs norm;        // of q's and k's heads (NORM)
    int Hq, Hkv, B, T, rot, rotate, heads_per_cta, groups;
    const int *pos;
    const int *block_table, *lens, *seen, *new_lens;
    void *kp, *vp;
    const float *ks, *vs;
    float *weight;
    int *order;
    int num_pages, max_pages, ps_shift;
};

// 8 values into the cache: bf16, or e4m3 codes of x / scale, the quotient rounded to nearest.  With
// inv the rounded reciprocal of the scale, q = x inv is within one step of the quotient, and
// q + (x - q scale) inv rounds it correctly (P. Markstein, 1990): three operations for two values
// where the divide takes several each.  A quotient that could overflow
// on the way is far beyond the largest code, and stays as it is.
template <bool FP8>
__device__ __forceinline__ void put8(void *base, long long at, const float (&x)[8], float scale, float inv)
{
    if constexpr (FP8) {
        float q[8];
#pragma unroll
        for (int j = 0; j < 8; j += 2)
            fmul2(q[j], q[j + 1], x[j], x[j + 1], inv, inv);
        const float big = fmax3(fmax3(fabsf(q[0]), fabsf(q[1]), fabsf(q[2])), fmax3(fabsf(q[3]), fabsf(q[4]), fabsf(q[5])),
                                fmaxf(fabsf(q[6]), fabsf(q[7])));
        if (big < 1e30f) {
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                float r0, r1;
                ffma2(r0, r1, q[j], q[j + 1], -scale, -scale, x[j], x[j + 1]);
                ffma2(q[j], q[j + 1], r0, r1, inv, inv, q[j], q[j + 1]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float y = fmaf(fmaf(q[j], -scale, x[j]), inv, q[j]);
                q[j] = fabsf(q[j]) < 1e30f ? y : q[j];
            }
        }
        uint2 w;
        w.x = pack_e4m3x4(q[0], q[1], q[2], q[3]);
        w.y = pack_e4m3x4(q[4], q[5], q[6], q[7]);
        *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(base) + at) = w;
    } else {
        store8(static_cast<__nv_bfloat16 *>(base) + at, x);
    }
}

// Heads run q, then k, then v; a token's slot and page are looked up once per thread.  NORM: the rows of q
// and k are normed before they turn, their loads four heads ahead (4 sequences of 1000 tokens, 32 + 8 heads of 128: bf16
// 16.6 us, 17.2 with six, 14.7 without a norm; e4m3 18.9, 19.4 and 15.6; 16 + 16 heads of 64 10.0, 10.5 and 8.0).
template <int D, bool INTER, bool FP8, bool NORM>
__global__ void __launch_bounds__(kRopeThreads, 2) append_kernel(const __grid_constant__ RopeTable tab,
                                                              const __grid_constant__ AppendArgs a)
{
    constexpr int TPR = D / 16;
    pdl_launch();
    pdl_wait();
    const int vec = threadIdx.x % TPR;
    const long long n = (long long)a.B * a.T;
    // head groups next to one another: CTAs that run together read whole token rows of a packed
    // projection
    const int tile = (int)(blockIdx.x / a.groups), group = (int)blockIdx.x - tile * a.groups;
    const long long tok = (long long)tile * (kRopeThreads / TPR) + threadIdx.x / TPR;
    const Slice sl = slice_of(vec, a.rotate ? a.rot : 0, INTER);
    __shared__ __align__(16) float weight[2][NORM ? D : 1];
    if constexpr (NORM) {
        put_norm_weights<D>(a.norm, sl, weight);
        __syncthreads();
    }
    if (tok >= n)
        return;
    const int b = (int)tok / a.T, t = (int)tok - b * a.T;
    const int len = a.lens[b], cap = a.max_pages << a.ps_shift;
    const int nb = a.new_lens ? a.new_lens[b] : a.T;
    const int h0 = group * a.heads_per_cta, h1 = min(a.Hq + 2 * a.Hkv, h0 + a.heads_per_cta);
    const bool turns = sl.pair >= 0 && h0 < a.Hq + a.Hkv;
    int pos[8];
    if (turns) {   // with the lengths, not after them
#pragma unroll
        for (int j = 0; j < 8; ++j)
            pos[j] = a.pos[(long long)tab.axis[sl.pair + j] * n + tok];
    }
    if (len < 0 || len > cap || nb < 0 || nb > a.T || nb > len) {
        if (vec == 0 && t == 0 && group == 0)
            atomicCAS(&g_cache_status, 0, kStatusBadIndex);
        return;
    }
    if (t >= nb)
        return;
    const int slot = len - nb + t;
    int page = 0;
    if (h1 > a.Hq)
        page = a.block_table[(long long)b * a.max_pages + (slot >> a.ps_shift)];
    float sn[8], cs[8];
    if (turns) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            phase_sincos(tab.turns[sl.pair + j], pos[j], sn[j], cs[j]);
    }
    const bool page_ok = page >= 0 && page < a.num_pages;
    if (h1 > a.Hq && !page_ok && vec == 0)
        atomicCAS(&g_cache_status, 0, kStatusBadIndex);
    using E = __nv_bfloat16;
    const int gap = sl.e1 - sl.e0;
    auto part = [&](int from, int n, int &first, int &count) {   // the group's heads among n from `from` on
        first = max(h0 - from, 0);
        count = min(h1 - from, n) - first;
        return count > 0;
    };
    int first, count;
    if (part(0, a.Hq, first, count)) {
        const E *x = static_cast<const E *>(a.q.p) + b * a.q.sb + first * a.q.sh + t * a.q.st;
        E *o = static_cast<E *>(a.qo.p) + b * a.qo.sb + first * a.qo.sh + t * a.qo.st + sl.e0;
        auto put = [&](int, float(&f)[8], float(&g)[8]) {
            if (turns)
                turn<INTER>(f, g, sn, cs);
            store8(o, f);
            store8(o + gap, g);
            o += a.qo.sh;
        };
        if constexpr (NORM)
            each_head_normed<E, D, 4>(x, a.q.sh, count, sl, weight[0], a.norm.eps, [] {}, put);
        else
            each_head(x, a.q.sh, count, sl, put);
    }
    if (!page_ok)
        return;
    const long long row_at = (((long long)page * a.Hkv << a.ps_shift) + (slot & ((1 << a.ps_shift) - 1))) * D + sl.e0;
    const long long step = (long long)D << a.ps_shift;   // from head to head in a page
    if (part(a.Hq, a.Hkv, first, count)) {
        const E *x = static_cast<const E *>(a.k.p) + b * a.k.sb + first * a.k.sh + t * a.k.st;
        long long at = row_at + first * step;
        auto put = [&](int i, float(&f)[8], float(&g)[8]) {
            if (turns)
                turn<INTER>(f, g, sn, cs);
            const float scale = FP8 ? a.ks[first + i] : 1.f, inv = FP8 ? __frcp_rn(scale) : 1.f;
            put8<FP8>(a.kp, at, f, scale, inv);
            put8<FP8>(a.kp, at + gap, g, scale, inv);
            at += step;
            if (vec == 0) {
                const long long w = ((long long)b * a.Hkv + first + i) * cap + slot;
                if (a.weight)
                    a.weight[w] = 0.f;
                if (a.order)
                    a.order[w] = (a.seen ? a.seen[b] - nb : len - nb) + t;
            }
        };
        if constexpr (NORM)
            each_head_normed<E, D, 4>(x, a.k.sh, count, sl, weight[1], a.norm.eps, [] {}, put);
        else
            each_head(x, a.k.sh, count, sl, put);
    }
    if (part(a.Hq + a.Hkv, a.Hkv, first, count)) {
        const E *x = static_cast<const E *>(a.v.p) + b * a.v.sb + first * a.v.sh + t * a.v.st;
        long long at = row_at + first * step;
        each_head(x, a.v.sh, count, sl, [&](int i, float(&f)[8], float(&g)[8]) {
            const float scale = FP8 ? a.vs[first + i] : 1.f, inv = FP8 ? __frcp_rn(scale) : 1.f;
            put8<FP8>(a.vp, at, f, scale, inv);
            put8<FP8>(a.vp, at + gap, g, scale, inv);
            at += step;
        });
    }
}

template <int D, bool FP8, bool NORM>
int append_with(const RopeTable &t, const AppendArgs &a, int interleaved, cudaStream_t s)
{
    constexpr int TOK = kRopeThreads / (D / 16);
    const long long n = (long long)a.B * a.T;
    const dim3 grid((unsigned)((n + TOK - 1) / TOK * a.groups));
    return launch_overlapped(interleaved ? append_kernel<D, true, FP8, NORM> : append_kernel<D, false, FP8, NORM>, grid, kRopeThreads, 0, 0,
                             true, s, t, a);
}

template <int D, bool FP8>
int append_run(const RopeTable &t, const AppendArgs &a, int interleaved, bool norm, cudaStream_t s)
{
    return norm ? append_with<D, FP8, true>(t, a, interleaved, s) : append_with<D, FP8, false>(t, a, interleaved, s);
}

// ------------------------------------------------------------------ evict
struct EvictArgs {
    const float *weight;
    const int *order, *lens, *seen, *block_table;
    float *weight_out;
    int *order_out, *lens_out, *kept;
    uint8_t *k, *v;
    int B, Hkv, budget, n_first, n_recent, cap, num_pages, max_pages, ps_shift, row_bytes;
};

constexpr int kSelThreads = 1024;

// Rank of an entry: larger stays.  Floats in their order (-0 as 0, a NaN as the least); the
// largest value is kept for protected entries.
__device__ __forceinline__ uint32_t rank_key(float w, bool is_protected)
{
    if (is_protected)
        return 0xFFFFFFFFu;
    if (w != w)
        return 0u;
    const uint32_t u = __float_as_uint(w + 0.f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Sum of x over the block, in every thread.
__device__ __forceinline__ int block_sum(int x, int *scratch)
{
    x = __reduce_add_sync(0xffffffffu, x);
    __syncthreads();
    if (lane_id() == 0)
        scratch[warp_id()] = x;
    __syncthreads();
    return __reduce_add_sync(0xffffffffu, lane_id() < blockDim.x / 32 ? scratch[lane_id()] : 0);
}

// Number of true predicates in the lower threads of the block, and in all of it.
__device__ __forceinline__ int block_rank(bool p, int &total, int *scratch)
{
    const uint32_t m = __ballot_sync(0xffffffffu, p);
    __syncthreads();
    if (lane_id() == 0)
        scratch[warp_id()] = __popc(m);
    __syncthreads();
    const int c = lane_id() < blockDim.x / 32 ? scratch[lane_id()] : 0;
    total = __reduce_add_sync(0xffffffffu, c);
    const int before = __reduce_add_sync(0xffffffffu, lane_id() < warp_id() ? c : 0);
    return before + __popc(m & ((1u << lane_id()) - 1u));
}

// ---- selection by a cluster per (sequence, KV head)
// The entries' ranks are read once and stay in shared memory, a contiguous run of slots per CTA.
// Up to four passes of a radix select of 8 bits (counts of the whole cluster read over distributed
// shared memory, every CTA finds the digit for itself; fewer when all that match a prefix stay)
// give the rank of the last entry that stays.  Then one scan over runs of consecutive slots per
// thread numbers the holes in front of the new length and the kept entries behind it, which each
// CTA lists; then the cluster's threads take hole and entry number g from whichever CTAs list them.
// It is bound by latency, a chain of a dozen block- and cluster-wide steps, and not by its 20 bytes
// an entry; what an entry that stays in its slot needs (kept, weight, order) is written when it is
// read.  With 512 threads a CTA the selection of 64 units of 4112 entries and of 32 of up to 32768 took 14.7
// and 18 us, with 256 15.7 and 19.5, with 1024 15.8 and 18.  The cluster then moves the rows itself:
// a second kernel for them cost 3 us more.
constexpr int kPickThreads = 512;
constexpr int kSelBins = 256, kSelPasses = 4;
constexpr int kSelCap = 32767;                               // entries a CTA, at most (two counts share an int)
constexpr int kSelCopies = 8;                                // of the first pass's counts: most ranks share a few digits
constexpr int kSelFixed = (kSelPasses + kSelCopies) * kSelBins * 4 + 32 * 4 + 32;   // shared memory besides the entries

// All threads of the cluster meet; not the .aligned form, which wants whole warps: the loops before it
// go by the data.
__device__ __forceinline__ void cluster_sync()
{
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_addr(const void *p, int rank)   // the same place in another CTA
{
    uint32_t addr;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_u32(p)), "r"(rank));
    return addr;
}
__device__ __forceinline__ int cluster_load(const int *p, int rank)
{
    int x;
    asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(x) : "r"(cluster_addr(p, rank)) : "memory");
    return x;
}
__device__ __forceinline__ int cluster_load16(const uint16_t *p, int rank)
{
    uint16_t x;
    asm volatile("ld.shared::cluster.u16 %0, [%1];" : "=h"(x) : "r"(cluster_addr(p, rank)) : "memory");
    return x;
}

// Sum of x over the lower threads of the block, and over all of it.
__device__ __forceinline__ int block_scan(int x, int &total, int *scratch)
{
    int inc = x;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, off);
        if ((int)lane_id() >= off)
            inc += y;
    }
    __syncthreads();
    if (lane_id() == 31)
        scratch[warp_id()] = inc;
    __syncthreads();
    const int c = lane_id() < blockDim.x / 32 ? scratch[lane_id()] : 0;
    total = __reduce_add_sync(0xffffffffu, c);
    return __reduce_add_sync(0xffffffffu, lane_id() < warp_id() ? c : 0) + inc - x;
}

// The length after eviction; one out of range stays as it is.
__device__ __forceinline__ int new_length(const EvictArgs &a, int len)
{
    return len < 0 || len > a.cap ? len : min(len, a.budget);
}

// Byte offset of a slot's row in the pools, -1 if its page is out of range.
__device__ __forceinline__ long long row_of(const EvictArgs &a, int b, int h, int slot)
{
    const int page = a.block_table[(long long)b * a.max_pages + (slot >> a.ps_shift)];
    if (page < 0 || page >= a.num_pages)
        return -1;
    return ((((long long)page * a.Hkv + h) << a.ps_shift) + (slot & ((1 << a.ps_shift) - 1))) * a.row_bytes;
}

// Copies the K and V rows of `n` moves (byte offsets from, to), one warp, eight 16-byte loads in
// flight a lane.  Sources lie behind the new length and targets in front of it.
__device__ __forceinline__ void copy_rows(const EvictArgs &a, const long long (*moves)[2], int n)
{
    const int vshift = 31 - __clz(a.row_bytes / 16), vecs = 1 << vshift;   // 16-byte vectors of a row
    const int count = n << (vshift + 1);                                   // of K and V
    for (int e0 = (int)lane_id(); e0 < count; e0 += 32 * 8) {
        uint4 x[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int e = e0 + 32 * u;
            if (e < count)
                x[u] = *reinterpret_cast<const uint4 *>((e & vecs ? a.v : a.k) + moves[e >> (vshift + 1)][0] + (e & (vecs - 1)) * 16);
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int e = e0 + 32 * u;
            if (e < count)
                *reinterpret_cast<uint4 *>((e & vecs ? a.v : a.k) + moves[e >> (vshift + 1)][1] + (e & (vecs - 1)) * 16) = x[u];
        }
    }
}

// Lists the moves of a warp's lanes (from < 0: none) and copies them.
__device__ __forceinline__ void move_rows(const EvictArgs &a, long long (*moves)[2], long long from, long long to)
{
    const uint32_t todo = __ballot_sync(0xffffffffu, from >= 0);
    if (from >= 0) {
        const int r = __popc(todo & ((1u << lane_id()) - 1u));
        moves[r][0] = from;
        moves[r][1] = to;
    }
    __syncwarp();
    copy_rows(a, moves, __popc(todo));
    __syncwarp();
}

// Byte offsets of a move's rows; from < 0 if a page is out of range.
__device__ __forceinline__ void move_of(const EvictArgs &a, int b, int h, int i, int j, long long &from, long long &to)
{
    from = row_of(a, b, h, i);
    to = row_of(a, b, h, j);
    if (from < 0 || to < 0) {
        atomicCAS(&g_cache_status, 0, kStatusBadIndex);
        from = -1;
    }
}

__global__ void __launch_bounds__(kPickThreads) evict_select_kernel(const __grid_constant__ EvictArgs a, int cs, int per)
{
    constexpr int T = kPickThreads;
    __shared__ long long moves[T / 32][32][2];
    __shared__ int lists[8];   // of each CTA: holes in the low half, entries behind the new length in the high half
    extern __shared__ __align__(16) int sel_smem[];
    int *copies = sel_smem, *hist = copies + kSelCopies * kSelBins, *scratch = hist + kSelPasses * kSelBins;
    int *share = scratch + 32, *pick = share + 4;
    uint32_t *keys = reinterpret_cast<uint32_t *>(pick + 4);
    uint16_t *list = reinterpret_cast<uint16_t *>(keys + per);   // holes, then movers
    const int rank = (int)blockIdx.x % cs, unit = (int)blockIdx.x / cs, b = unit / a.Hkv, h = unit - b * a.Hkv;
    const int tid = threadIdx.x;
    pdl_launch();
    for (int i = tid; i < (kSelCopies + kSelPasses) * kSelBins; i += T)
        copies[i] = 0;
    pdl_wait();
    const int len = a.lens[b];
    int *kept = a.kept + (long long)unit * a.budget;
    const long long base = (long long)unit * a.cap;
    const bool bad = len < 0 || len > a.cap;
    const int end = bad ? 0 : min(len, a.budget);
    if (bad && tid == 0)
        atomicCAS(&g_cache_status, 0, kStatusBadIndex);
    for (int j = end + rank * T + tid; j < a.budget; j += cs * T)
        kept[j] = -1;
    if (h == 0 && rank == 0 && tid == 0 && a.lens_out != a.lens)
        a.lens_out[b] = new_length(a, len);
    if (bad)
        return;   // the whole cluster
    const float *weight = a.weight + base;
    const int *order = a.order ? a.order + base : nullptr;
    const int lo = min(len, rank * per), n = min(len, lo + per) - lo;
    const int recent = (a.seen ? a.seen[b] : len) - a.n_recent;
    const bool ages = order && (a.n_first > 0 || a.n_recent > 0);
    __syncthreads();
    for (int i0 = tid; i0 < n; i0 += 8 * T) {   // eight loads in flight
        float w[8];
        int at[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int i = i0 + u * T;
            w[u] = i < n ? weight[lo + i] : 0.f;
            at[u] = order && i < n ? order[lo + i] : 0;
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int i = i0 + u * T, j = lo + i;
            if (i >= n)
                break;
            if (j < end) {   // right for an entry that stays in its slot
                kept[j] = j;
                a.weight_out[base + j] = w[u];
                if (order)
                    a.order_out[base + j] = at[u];
            }
            const uint32_t k = rank_key(w[u], ages && (at[u] < a.n_first || (a.n_recent > 0 && at[u] >= recent)));
            keys[i] = k;
            atomicAdd(&copies[(k >> 24) * kSelCopies + (tid & (kSelCopies - 1))], 1);
        }
    }
    if (len <= a.budget)
        return;   // all stay; the whole cluster
    uint32_t prefix = 0;
    int need = end, edge = INT_MAX;   // still to be taken among those that match the prefix; see below
#pragma unroll 1
    for (int pass = 0; pass < kSelPasses; ++pass) {
        const int shift = 24 - 8 * pass;
        int *hp = hist + pass * kSelBins;
        if (pass > 0) {
            for (int i = tid; i < n; i += T) {
                const uint32_t u = keys[i];
                if ((u ^ prefix) >> (shift + 8) == 0)
                    atomicAdd(&hp[(u >> shift) & 255], 1);
            }
        } else {
            __syncthreads();
            if (tid < kSelBins) {
                const int4 x = reinterpret_cast<const int4 *>(copies)[2 * tid], y = reinterpret_cast<const int4 *>(copies)[2 * tid + 1];
                hp[tid] = x.x + x.y + x.z + x.w + y.x + y.y + y.z + y.w;
            }
        }
        cluster_sync();
        // T / 256 threads a bin, bins from the top
        constexpr int TPB = T / kSelBins;
        const int d = kSelBins - 1 - tid / TPB;
        int c = 0;
        for (int r = tid % TPB; r < cs; r += TPB)
            c += cluster_load(hp + d, r);
#pragma unroll
        for (int off = 1; off < TPB; off <<= 1)
            c += __shfl_xor_sync(0xffffffffu, c, off);
        int total;
        const int before = block_scan(tid % TPB ? 0 : c, total, scratch);
        if (tid % TPB == 0 && before < need && need <= before + c) {
            pick[0] = d;
            pick[1] = need - before;
            pick[2] = c;
        }
        __syncthreads();
        prefix |= (uint32_t)pick[0] << shift;
        need = pick[1];
        const int equal = pick[2];
        if (equal == need)   // all that match stay: the lower digits do not matter
            break;
        if (pass == kSelPasses - 1) {   // of equal ranks the first `need` stay: those below slot `edge`
            int done = 0;
            for (int r = 0; r < rank; ++r)
                done += cluster_load(hp + (prefix & 255), r);
            edge = done >= need ? 0 : done + hp[prefix & 255] <= need ? INT_MAX : -1;
            if (edge < 0) {   // this CTA has the last one
                const int q = ((n + T - 1) / T) | 1, i0 = min(n, tid * q), i1 = min(n, i0 + q);
                int mine = 0;
                for (int i = i0; i < i1; ++i)
                    mine += keys[i] == prefix;
                int r = done + block_scan(mine, total, scratch);
                for (int i = i0; i < i1; ++i)
                    if (keys[i] == prefix && r++ == need - 1)
                        pick[3] = i + 1;
                __syncthreads();
                edge = pick[3];
            }
        }
    }
    auto stays = [&](int i) {
        const uint32_t u = keys[i];
        return u > prefix || (u == prefix && i < edge) || (edge == INT_MAX && u >= prefix);
    };
    // holes in front of the new length in the low half, kept entries behind it in the high half; an
    // odd run of consecutive slots per thread: the runs of a warp lie in different banks
    const int q = ((n + T - 1) / T) | 1, i0 = min(n, tid * q), i1 = min(n, i0 + q);
    int mine = 0, total;
    for (int i = i0; i < i1; ++i)
        mine += lo + i < end ? (stays(i) ? 0 : 1) : (stays(i) ? 1 << 16 : 0);
    const int before = block_scan(mine, total, scratch);
    if (mine) {
        int x = before & 0xFFFF, m = (total & 0xFFFF) + (before >> 16);
        for (int i = i0; i < i1; ++i) {
            const bool stay = stays(i);
            if (lo + i < end && !stay)
                list[x++] = (uint16_t)i;
            if (lo + i >= end && stay)
                list[m++] = (uint16_t)i;
        }
    }
    if (tid == 0)
        share[0] = total;
    cluster_sync();
    if (tid < 8)
        lists[tid] = tid < cs ? cluster_load(share, tid) : 0;
    __syncthreads();
    int all = 0, behind = 0;
    for (int r = 0; r < cs; ++r) {
        all += lists[r] & 0xFFFF;
        behind += lists[r] >> 16;
    }
    // as many holes as entries for them: anything else means that the lengths changed under the call,
    // and nothing is moved
    if (all != behind) {
        if (tid == 0)
            atomicCAS(&g_cache_status, 0, kStatusBadIndex);
        all = 0;
    }
    // hole and entry number g of the cluster; each of its warps takes up to 32 of them
    const int warps = cs * T / 32, chunk = min(32, (all + warps - 1) / warps);
    for (int g0 = (rank * (T / 32) + (int)warp_id()) * chunk; g0 < all; g0 += warps * chunk) {
        const int g = g0 + (int)lane_id();
        long long from = -1, to = -1;
        if ((int)lane_id() < chunk && g < all) {
            int r = 0, m = g, c = 0, x = g;   // the CTAs that list them, and their places there
            while (m >= (lists[r] & 0xFFFF))
                m -= lists[r++] & 0xFFFF;
            while (x >= lists[c] >> 16)
                x -= lists[c++] >> 16;
            const int j = r * per + cluster_load16(list + m, r);
            const int i = c * per + cluster_load16(list + (lists[c] & 0xFFFF) + x, c);
            if (j < end && i < len) {   // the same
                kept[j] = i;
                a.weight_out[base + j] = weight[i];
                if (order)
                    a.order_out[base + j] = order[i];
                move_of(a, b, h, i, j, from, to);
            }
        }
        move_rows(a, moves[warp_id()], from, to);
    }
    cluster_sync();   // no CTA ends while another may read its list
}

// The lengths, where lens_out is lens, which every CTA of the selection reads.
__global__ void __launch_bounds__(256) evict_lens_kernel(const __grid_constant__ EvictArgs a)
{
    pdl_launch();
    pdl_wait();
    for (int b = blockIdx.x * 256 + threadIdx.x; b < a.B; b += gridDim.x * 256)
        a.lens_out[b] = new_length(a, a.lens[b]);
}

// The same for lengths whose ranks do not fit the shared memory of a cluster: one CTA per
// (sequence, KV head) reads them at every pass.  Finds the rank of the last entry that stays
// (radix select, 8 bits a pass) and the slot up to which entries of that very rank stay, then pairs the kept
// entries behind the new length with the holes in front of it.
__global__ void __launch_bounds__(kSelThreads) evict_select_long_kernel(const __grid_constant__ EvictArgs a)
{
    __shared__ int hist[256], scratch[32], pick[2];
    const int unit = blockIdx.x, b = unit / a.Hkv, tid = threadIdx.x;
    pdl_launch();
    pdl_wait();
    const int len = a.lens[b];
    int *kept = a.kept + (long long)unit * a.budget;
    const long long base = (long long)unit * a.cap;
    if (len < 0 || len > a.cap) {
        if (tid == 0)
            atomicCAS(&g_cache_status, 0, kStatusBadIndex);
        for (int j = tid; j < a.budget; j += kSelThreads)
            kept[j] = -1;
        return;
    }
    const float *weight = a.weight + base;
    const int *order = a.order ? a.order + base : nullptr;
    const int end = min(len, a.budget);
    const int recent = (a.seen ? a.seen[b] : len) - a.n_recent;
    auto key = [&](int i) {
        const bool prot = order && (order[i] < a.n_first || (a.n_recent > 0 && order[i] >= recent));
        return rank_key(weight[i], prot);
    };
    if (len <= a.budget) {
        for (int j = tid; j < a.budget; j += kSelThreads)
            kept[j] = j < end ? j : -1;
    } else {
        uint32_t prefix = 0, mask = 0;
        int need = end;   // entries still to be taken among those that match the prefix
        for (int shift = 24; shift >= 0; shift -= 8) {
            for (int i = tid; i < 256; i += kSelThreads)
                hist[i] = 0;
            __syncthreads();
            for (int i = tid; i < len; i += kSelThreads) {
                const uint32_t u = key(i);
                if ((u & mask) == prefix)
                    atomicAdd(&hist[(u >> shift) & 255], 1);
            }
            __syncthreads();
            if (tid == 0) {
                int left = need, d = 255;
                while (d > 0 && hist[d] < left)
                    left -= hist[d--];
                pick[0] = d;
                pick[1] = left;
            }
            __syncthreads();
            prefix |= (uint32_t)pick[0] << shift;
            mask |= 255u << shift;
            need = pick[1];
            __syncthreads();
        }
        // slots up to `edge` of the entries whose rank is `prefix` itself stay
        int equal = 0;
        for (int i = tid; i < len; i += kSelThreads)
            equal += key(i) == prefix;
        equal = block_sum(equal, scratch);
        int edge = INT_MAX;
        if (equal > need) {
            int done = 0;
            for (int i0 = 0; i0 < len && edge == INT_MAX; i0 += kSelThreads) {
                const int i = i0 + tid;
                const bool eq = i < len && key(i) == prefix;
                int total;
                const int r = done + block_rank(eq, total, scratch);
                if (tid == 0)
                    pick[0] = INT_MAX;
                __syncthreads();
                if (eq && r == need - 1)
                    pick[0] = i;
                __syncthreads();
                edge = pick[0];
                done += total;
            }
        }
        auto stays = [&](int i) {
            const uint32_t u = key(i);
            return u > prefix || (u == prefix && i <= edge);
        };
        // kept entries behind the new length, in order, for the moment at the front of `kept`
        int movers = 0;
        for (int i0 = end; i0 < len; i0 += kSelThreads) {
            const int i = i0 + tid;
            const bool m = i < len && stays(i);
            int total;
            const int r = movers + block_rank(m, total, scratch);
            if (m)
                kept[r] = i;
            movers += total;
        }
        __syncthreads();
        // the holes take them, from the last tile to the first: a hole's rank is at most its
        // slot, so a tile overwrites no entry that a lower tile still has to read
        int left = movers;
        for (int i0 = (end - 1) / kSelThreads * kSelThreads; i0 >= 0; i0 -= kSelThreads) {
            const int i = i0 + tid;
            const bool hole = i < end && !stays(i);
            int total;
            const int r = block_rank(hole, total, scratch);
            left -= total;
            const int from = hole ? kept[left + r] : i;
            __syncthreads();
            if (i < end)
                kept[i] = from;
        }
    }
    __syncthreads();
    for (int j = tid; j < end; j += kSelThreads) {
        const int i = kept[j];
        a.weight_out[base + j] = weight[i];
        if (order)
            a.order_out[base + j] = order[i];
    }
}

// Rows of the moved entries after the selection of long lengths: each warp takes 32 entries of one
// (sequence, KV head).
__global__ void __launch_bounds__(256) evict_move_kernel(const __grid_constant__ EvictArgs a)
{
    __shared__ long long moves[8][32][2];
    const int unit = blockIdx.x, b = unit / a.Hkv, h = unit - b * a.Hkv;
    pdl_launch();
    pdl_wait();
    if (blockIdx.y == 0 && h == 0 && threadIdx.x == 0)
        a.lens_out[b] = new_length(a, a.lens[b]);
    for (int j0 = (blockIdx.y * 8 + (int)warp_id()) * 32; j0 < a.budget; j0 += gridDim.y * 256) {
        const int j = j0 + (int)lane_id();
        const int i = j < a.budget ? a.kept[(long long)unit * a.budget + j] : -1;
        long long from = -1, to = -1;
        if (i >= 0 && i != j)
            move_of(a, b, h, i, j, from, to);
        move_rows(a, moves[warp_id()], from, to);
    }
}

int shift_of(int page_size)
{
    int s = 0;
    while ((1 << s) < page_size)
        ++s;
    return s;
}

}  // namespace

int rope_launch(const fa_heads *x, const fa_heads *y, int n, const int *positions, const fa_rope_spec &spec, int B,
                int T, int dtype, int inverse, cudaStream_t s)
{
    RopeArgs a;
    for (int i = 0; i < 2; ++i) {
        a.x[i] = row3(x[i < n ? i : 0]);
        a.y[i] = row3(y[i < n ? i : 0]);
    }
    a.H0 = x[0].H;
    a.H = x[0].H + (n > 1 ? x[1].H : 0);
    a.pos = positions;
    a.n = (long long)B * T;
    a.T = T;
    a.rot = spec.rot;
    a.heads_per_cta = heads_per_cta(a.n, a.H, spec.d);
    a.groups = (a.H + a.heads_per_cta - 1) / a.heads_per_cta;
    if ((a.n / 16 + 1) * a.groups > INT_MAX)
        return ERR_UNSUPPORTED;
    a.sign = inverse ? -1.f : 1.f;
    const RopeTable t = table_of(spec);
    return dtype == FA_F32 ? rope_width<float>(spec.d, t, a, spec.interleaved, s)
                           : rope_width<__nv_bfloat16>(spec.d, t, a, spec.interleaved, s);
}

int append_launch(const fa_kv_cache &c, const fa_heads &k, const fa_heads &v, const fa_heads *q,
                  const fa_heads *q_out, const int *positions, const fa_rope_spec *spec, const fa_head_norm *norm,
                  const int *new_lens, int T, cudaStream_t s)
{
    status_in_use(STATUS_CACHE);
    AppendArgs a;
    a.norm = norm ? norm_args(*norm) : NormArgs{};
    a.k = row3(k);
    a.v = row3(v);
    a.q = q ? row3(*q) : Row3{nullptr, 0, 0, 0};
    a.qo = q ? row3(*q_out) : Row3{nullptr, 0, 0, 0};
    a.Hq = q ? q->H : 0;
    a.Hkv = c.Hkv;
    a.B = c.B;
    a.T = T;
    a.rotate = spec != nullptr;
    a.rot = spec ? spec->rot : 0;
    a.pos = positions;
    a.block_table = c.block_table;
    a.lens = c.lens;
    a.seen = c.seen;
    a.new_lens = new_lens;
    a.kp = c.k;
    a.vp = c.v;
    a.ks = c.k_scale;
    a.vs = c.v_scale;
    a.weight = c.weight;
    a.order = c.order;
    a.num_pages = c.num_pages;
    a.max_pages = c.max_pages;
    a.ps_shift = shift_of(c.page_size);
    const int H = a.Hq + 2 * a.Hkv;
    a.heads_per_cta = heads_per_cta((long long)c.B * T, H, c.d);
    a.groups = (H + a.heads_per_cta - 1) / a.heads_per_cta;
    if (((long long)c.B * T / 16 + 1) * a.groups > INT_MAX)
        return ERR_UNSUPPORTED;
    RopeTable t{};
    if (spec)
        t = table_of(*spec);
    const int inter = spec ? spec->interleaved : 0;
    const bool f8 = c.dtype == FA_E4M3;
    switch (c.d) {
    case 64:
        return f8 ? append_run<64, true>(t, a, inter, norm, s) : append_run<64, false>(t, a, inter, norm, s);
    case 128:
        return f8 ? append_run<128, true>(t, a, inter, norm, s) : append_run<128, false>(t, a, inter, norm, s);
    default:
        return f8 ? append_run<256, true>(t, a, inter, norm, s) : append_run<256, false>(t, a, inter, norm, s);
    }
}

int evict_launch(const fa_kv_cache &c, int budget, int n_first, int n_recent, float *weight_out, int *order_out,
                 int *lens_out, int *kept, cudaStream_t s)
{
    status_in_use(STATUS_CACHE);
    EvictArgs a;
    a.weight = c.weight;
    a.order = c.order;
    a.lens = c.lens;
    a.seen = c.seen;
    a.block_table = c.block_table;
    a.weight_out = weight_out;
    a.order_out = order_out;
    a.lens_out = lens_out;
    a.kept = kept;
    a.k = static_cast<uint8_t *>(c.k);
    a.v = static_cast<uint8_t *>(c.v);
    a.B = c.B;
    a.Hkv = c.Hkv;
    a.budget = budget;
    a.n_first = n_first;
    a.n_recent = n_recent;
    a.cap = c.max_pages * c.page_size;
    a.num_pages = c.num_pages;
    a.max_pages = c.max_pages;
    a.ps_shift = shift_of(c.page_size);
    a.row_bytes = c.d * (c.dtype == FA_E4M3 ? 1 : 2);
    const int units = c.B * c.Hkv;
    // CTAs per (sequence, KV head): as many as there are SMs for, with 512 entries or more each (the
    // rows are moved by as many), or two an SM with 2048 or more.  us with 1, 2, 4 and 8 of them:
    //   64 units of 4112 entries, 16 evicted                   13.2  12.1  14.4  29.5   (2)
    //   32 units of up to 32768, 4096 stay                    110    55.0  37.3  32.1   (8)
    //   1 unit of 5935, d 256, 3851 stay                       42.2  29.1  16.8  13.3   (8)
    //   256 units of 2100, 2000 stay                           14.7  23.2  42.8  80.1   (1)
    int cs = 1;
    auto worth = [&](int n) {
        return (long long)units * n <= device_sm_count() ? a.cap / n >= 512
                                                         : (long long)units * n <= 2 * device_sm_count() && a.cap / n >= 2048;
    };
    while (cs < 8 && worth(2 * cs))
        cs *= 2;
    while (cs < 8 && (a.cap + cs - 1) / cs > kSelCap)
        cs *= 2;
    const int per = (a.cap + cs - 1) / cs;
    const bool wide = per <= kSelCap && (long long)units * cs <= INT_MAX;
    if (wide) {
        int st = allow_smem<evict_select_kernel>(kSelFixed + kSelCap * 6);
        if (st != OK)
            return st;
        st = launch_overlapped(evict_select_kernel, dim3((unsigned)(units * cs)), kPickThreads, kSelFixed + per * 6,
                                         cs, true, s, a, cs, per);
        if (st != OK || lens_out != c.lens)
            return st;
        return launch_overlapped(evict_lens_kernel, dim3((unsigned)((c.B + 255) / 256)), 256, 0, 0, true, s, a);
    }
    const int st = launch_overlapped(evict_select_long_kernel, dim3((unsigned)units), kSelThreads, 0, 0, false, s, a);
    if (st != OK)
        return st;
    const int blocks = (budget + 255) / 256;
    return launch_overlapped(evict_move_kernel, dim3((unsigned)units, blocks < 64 ? blocks : 64), 256, 0, 0, true, s, a);
}

int cache_status_fetch_clear(cudaStream_t s, int *host_word)
{
    int zero = 0;
    if (cudaMemcpyFromSymbolAsync(host_word, g_cache_status, sizeof(int), 0, cudaMemcpyDeviceToHost, s) != cudaSuccess ||
        cudaStreamSynchronize(s) != cudaSuccess)
        return ERR_CUDA;
    if (*host_word != 0 &&
        (cudaMemcpyToSymbolAsync(g_cache_status, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, s) != cudaSuccess ||
         cudaStreamSynchronize(s) != cudaSuccess))
        return ERR_CUDA;
    return OK;
}

}  // namespace fa
