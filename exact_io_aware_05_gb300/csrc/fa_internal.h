// fa_internal.h -- host-side glue between the C-ABI layer (fa_api.cu) and the
// kernel translation units.  Not part of the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/fa.h"

namespace fa {

// Status codes, identical to fa_status in include/fa.h.
enum : int { OK = 0, ERR_INVALID_ARG = 1, ERR_UNSUPPORTED = 2, ERR_CUDA = 3, ERR_TIMEOUT = 4, ERR_BAD_INDEX = 5 };

// Encodes a 3-D tiled TMA map over a contiguous [planes][rows][inner] tensor
// with 128-byte swizzle; the box is [1][box_rows][box_inner].  Returns OK or
// ERR_CUDA (driver entry point missing, or the driver rejected the map).
int encode_tmap_3d(CUtensorMap *map, const void *base, CUtensorMapDataType dtype, int elem_bytes,
                   uint64_t inner, uint64_t rows, uint64_t planes, uint32_t box_inner,
                   uint32_t box_rows);

// Argument checks shared by the entry points: 16-byte alignment, a buffer of n elements that
// is non-null and aligned (or anything when n == 0), overlap of two byte ranges, and the
// sm_103 check of the current device (cached).
bool aligned16(const void *p);
bool present16(const void *p, size_t n);
bool overlaps(const void *a, size_t na, const void *b, size_t nb);
int check_device();

int device_sm_count();          // SMs of the current device (cached per device)
uint64_t wait_timeout_ns();     // bounded-wait limit for device spin waits

// Test-only build of the library (compiled with FA_TEST_WITHHOLD=1 into a separate
// shared object; the product library is built without it and has none of this): one
// launch may leave out one mbarrier arrive, so that a bounded wait of one CTA runs out
// and the timeout path (abort flag, drains, status word) runs.  The case is armed from
// the host, once, and taken by the next launch of the matching kernel:
//   WITHHOLD_FWD_KV   forward, CTA 0: query tile 0's release of its first K/V slot;
//                     the producer waits for that slot again (the MMA issuers and the
//                     softmax then wait for copies that never come)
//   WITHHOLD_FWD_EPI  forward, CTA 0: the "O~ final" signal of query tile 0 in the first
//                     unit; only that tile's softmax waits for it (epilogue)
//   WITHHOLD_BWD_DKV  backward tile loop, CTA 0: the "dK, dV complete" signal of its
//                     first unit; only the drain warpgroup waits for it
//   WITHHOLD_PAGED_FULL  paged decode, CTA 0: the loader's arrive for its first tile; the math
//                     warps wait for it, and in a unit longer than the ring the loader for them
//   WITHHOLD_RANGE_FULL  the same of the paged decode over a part of the entries
//   WITHHOLD_PREFIX_FULL  the same of the shared prefix's attention
#ifndef FA_TEST_WITHHOLD
#define FA_TEST_WITHHOLD 0
#endif
enum : int { WITHHOLD_NONE = 0, WITHHOLD_FWD_KV = 1, WITHHOLD_FWD_EPI = 2, WITHHOLD_BWD_DKV = 3, WITHHOLD_PAGED_FULL = 4, WITHHOLD_RANGE_FULL = 5,
                 WITHHOLD_PREFIX_FULL = 6 };
#if FA_TEST_WITHHOLD
int test_withhold_take(int lo, int hi);   // the armed case if in [lo, hi] (then disarmed), else 0
#endif
// Heads per group of a persistent kernel's unit order.  gmax keeps the group's
// tensors within the L2 budget; where a group size in [gmax/2, gmax] makes a group
// a whole number of passes over the grid (levels units per head), the snake order
// of the passes balances the CTAs, so that size is taken.
inline int grid_aligned_group(int gmax, int levels, int grid)
{
    if (gmax < 1)
        gmax = 1;
    for (int g = gmax; g >= 1 && 2 * g >= gmax; --g)
        if (grid > 0 && ((long long)g * levels) % grid == 0)
            return g;
    return gmax;
}

// Heads per group where all passes run the same way: units go round the heads of a group, and the CTAs, neighbours
// presumably on different dies, round the units, so that with an even number a head's units keep to one die.  Backward
// under a window of 1024 with 4 sinks, B8 H32 T4096 d128: 1571 to 1640 us with 4, 6, 8, 10 and 12 heads, 1850 to 1930
// with 3, 5, 7 and 9; forward 495 to 513 and 504 to 529.  A single head stays one: backward under a block mask of which 5% is
// left, 65536 rows of d 128, one, two and four heads 6.73, 7.66 and 8.54 ms.
inline int even_group(int g, int BH)
{
    return g >= BH ? BH : g < 2 ? 1 : g & ~1;
}

// Heads per group under a left bound: `most`, unless what one head keeps in use alone is more than `budget`, and several
// would drive each other out of the L2.  Under a window of left keys it is that of `left` rows and of those that 152
// units of `unit_rows` rows span, at most all T; bytes_row: of K and V forward, of Q, dO and dQ's fp32 sums backward.
// Measured with 1 and 8 heads forward, 1 and 4 backward, in ms (d 128 but where said):
//   T 131072, 130000 keys 25.8 and 27.1, 67.1 and 70.7; 100000 24.5 and 25.8, 62.7 and 64.9; 60000 18.2 and 18.9, 46.5
//   and 47.6; 30000 (35 and 51 MB) 10.5 and 10.6, 26.9 and 26.9; T 65536, 60000 keys (34 and 67 MB) 6.91 and 6.58, 16.6
//   and 16.4; 30000 4.86 and 4.76, 11.7 and 11.5; T 32768, 31000 keys 3.53 and 3.39, 8.66 and 8.45; d 256, T 131072, 120000
//   keys 26.9 and 27.5 (4 heads); d 64, T 262144, 200000 keys 40.4 and 40.5 (4), 90.0 and 89.8.
inline int window_group(int T, int left, int unit_rows, int bytes_row, long long budget, int most)
{
    const long long rows = (long long)left + 152ll * unit_rows;
    return (rows < T ? rows : T) * bytes_row > budget ? 1 : most;
}
constexpr long long kFwdWindowBytes = 48ll << 20, kBwdWindowBytes = 72ll << 20;

// Allowed (row, key) pairs: key l is allowed for row r iff
//   r + Tk - Tq - left <= l <= r + Tk - Tq + right   (left, right = -1: that side unbounded)
// and, with a block mask, block[(r / 128) * nkbm + l / 128] != 0 for the head's mask
// ([heads][ceil(Tq / 128)][ceil(Tk / 128)] bytes in device memory, one mask per head when
// per_head, else one for all heads).  Causal is left = -1, right = 0.  The left bound does not hold for keys
// below sinks (right = 0 and no block mask with them).
struct MaskSpec {
    int left, right;
    const uint8_t *block;
    int per_head;
    int sinks = 0;
};
// A left bound that hides no key of Tk (every row's position is below Tk) is none.  Causal with one and without, us, B8 H32
// T4096 d128: forward 1002 and 803, backward 2512 and 2346; T 1024 109 and 94, 296 and 276; B1 H16 T32768 3440 and 3130, 8440
// and 8480; B1 H6 T65536 d64 4310 and 3910, 9240 and 8810.
inline MaskSpec effective_mask(MaskSpec m, int Tk)
{
    if (m.left >= 0 && (long long)m.left + m.sinks >= Tk - 1)   // keys from sinks to Tk - 2 - left would be hidden
        m.left = -1;
    if (m.left < 0)
        m.sinks = 0;
    return m;
}
inline MaskSpec causal_spec(int causal) { return MaskSpec{-1, causal ? 0 : -1, nullptr, 0}; }

// Kernel launchers (arguments already validated by the ABI layer).
int fwd_bf16_launch(const void *q, const void *k, const void *v, void *o, float *lse, int BH,
                    int Tq, int Tk, int d, const MaskSpec &mask, float scale, cudaStream_t s);
int fwd_f32_launch(const float *q, const float *k, const float *v, float *o, float *lse, int BH,
                   int Tq, int Tk, int d, int causal, float scale, cudaStream_t s);
int fill_empty_launch(void *o, float *lse, size_t rows, int d, int elem_bytes, cudaStream_t s);

// FP8 forward (fa_fp8_sm103.cu, fa_fwd_sm103.cu): row stride in bytes of the
// transposed V codes, the quantization pass, and the forward over its output.
size_t fp8_vt_stride(int Tk);
int fp8_quantize_launch(const void *q, const void *k, const void *v, const float *signs, int BH, int Tq, int Tk,
                        int d, void *q8, void *k8, void *vt8, float *qd, float *kd, float *vd, cudaStream_t s);
int fwd_fp8_launch(const void *q8, const void *k8, const void *vt8, const float *qd, const float *kd,
                   const float *vd, void *o, float *lse, int BH, int Tq, int Tk, int d, int causal, float scale,
                   cudaStream_t s);
// encode_tmap_3d without swizzle (the box is plain row-major in shared memory)
int encode_tmap_3d_plain(CUtensorMap *map, const void *base, CUtensorMapDataType dtype, int elem_bytes,
                         uint64_t inner, uint64_t rows, uint64_t planes, uint32_t box_inner, uint32_t box_rows);
// encode_tmap_3d with an explicit row stride in bytes (a multiple of 16)
int encode_tmap_3d_strided(CUtensorMap *map, const void *base, CUtensorMapDataType dtype, int elem_bytes,
                           uint64_t inner, uint64_t rows, uint64_t planes, uint64_t row_stride,
                           uint32_t box_inner, uint32_t box_rows);

// Backward workspace; rows of every head are padded to Tq_pad = roundup(Tq, 128).
struct BwdWorkspace {
    float *lse2;     // [BH][Tq_pad]    -lse * log2(e); -inf for padding rows and rows without keys
    float *delta;    // [BH][Tq_pad]    -D_r = -(dO_r . O_r) (0 for padding rows)
    float *dq_acc;   // [BH][Tq_pad][d] fp32 dQ accumulator (unscaled)
    // deterministic mode: dq_acc holds int32 fixed point; per head the largest |V_l|_2
    // and |K_lc| (float bits), and per 128-row query block a bound on |dq_acc| (float bits)
    float *kvmax;    // [BH][2]
    int *bound;      // [BH][Tq_pad / 128]
    float *sink_part = nullptr;   // behind them: partial dV, dK of split key blocks (bwd_sink_bytes; 0: none)
};
int bwd_sink_parts(size_t BH, int Tq, int Tk, const MaskSpec &mask);
size_t bwd_sink_bytes(size_t BH, int Tq, int Tk, int d, const MaskSpec &mask);
size_t bwd_row_stride(int Tq);
size_t bwd_workspace_bytes(size_t BH, int Tq, int d);
BwdWorkspace bwd_workspace_carve(void *ws, int BH, int Tq, int d);
// stages: bit 0 = preprocess (D, lse2, zero dQ accumulator; fixed-point bounds),
// bit 1 = tile loop (dK, dV, dQ accumulation), bit 2 = dQ scale-and-round;
// kBwdDeterministic: dQ is accumulated as int32 fixed point (order-independent sums).
constexpr int kBwdDeterministic = 8;
// Every check of fa_bwd's arguments except the workspace's and the device's (no CUDA call).
int bwd_check_args(const void *q, const void *k, const void *v, const void *o, const float *lse, const void *dO,
                   const void *dq, const void *dk, const void *dv, int B, int H, int Tq, int Tk, int d,
                   const MaskSpec &mask, float scale);
int bwd_launch(const void *q, const void *k, const void *v, const void *o, const float *lse,
               const void *dO, void *dq, void *dk, void *dv, int BH, int Tq, int Tk, int d,
               const MaskSpec &mask, float scale, const BwdWorkspace &ws, int stages, cudaStream_t s);

// Split-KV decode (fa_decode_sm103.cu): chunks per head and key tiles per
// chunk for these sizes, partial-state workspace bytes, query rows allowed per
// head at head width d, and the launch (split kernel + merge kernel).
void decode_split(int BH, int Tk, int *nsplit, int *tps);
size_t decode_workspace_bytes(int BH, int Tq, int Tk, int d);
int decode_max_rows(int d);
int decode_launch(const void *q, const void *k, const void *v, void *o, float *lse, int BH, int Tq, int Tk, int d,
                  int causal, float scale, void *workspace, cudaStream_t s);

// Device status words of the kernel translation units: read, add into *acc
// the first nonzero value, and clear.  Stream-ordered; the caller syncs.
int fwd_status_fetch_clear(cudaStream_t s, int *host_word);
int bwd_status_fetch_clear(cudaStream_t s, int *host_word);
int dec_status_fetch_clear(cudaStream_t s, int *host_word);

// Encodes a tiled TMA map of `rank` dimensions (innermost first; strides in bytes of all but the
// innermost) with the given swizzle.  Returns OK or ERR_CUDA.
int encode_tmap(CUtensorMap *map, const void *base, CUtensorMapDataType dtype, int rank, const uint64_t *dims,
                const uint64_t *strides, const uint32_t *box, CUtensorMapSwizzle swizzle);

// Rotary positions and the paged cache (fa_cache_sm103.cu, fa_paged_sm103.cu); arguments
// already validated by fa_cache_api.cu.  Structures as in include/fa.h.
int rope_launch(const fa_heads *x, const fa_heads *y, int n, const int *positions, const fa_rope_spec &spec, int B,
                int T, int dtype, int inverse, cudaStream_t s);
int append_launch(const fa_kv_cache &c, const fa_heads &k, const fa_heads &v, const fa_heads *q,
                  const fa_heads *q_out, const int *positions, const fa_rope_spec *spec, const fa_head_norm *norm,
                  const int *new_lens, int T, cudaStream_t s);
// Head norms with the rotation (fa_norm_sm103.cu).  rows of n tensors; the gradients of the weights may be null.
int norm_rope_launch(const fa_heads *x, const fa_heads *y, int n, const fa_head_norm &norm, const int *positions,
                     const fa_rope_spec &spec, int B, int T, int dtype, cudaStream_t s);
size_t norm_bwd_workspace_bytes(int d);
int norm_rope_bwd_launch(const fa_heads *x, const fa_heads *dy, const fa_heads *dx, int n, const fa_head_norm &norm,
                         const int *positions, const fa_rope_spec &spec, int B, int T, int dtype, float *dq_weight,
                         float *dk_weight, void *workspace, cudaStream_t s);
int evict_launch(const fa_kv_cache &c, int budget, int n_first, int n_recent, float *weight_out, int *order_out,
                 int *lens_out, int *kept, cudaStream_t s);
size_t paged_workspace_bytes(int B, int Hq, int Hkv, int Tq, int max_len, int d, int accumulate);
// first_pages: the first n_first pages of every sequence, read in place of their entries in the block table.
int paged_launch(const fa_kv_cache &c, const void *q, void *o, float *lse, int Hq, int Tq, int causal, float scale,
                 int accumulate, void *workspace, cudaStream_t s, const int *first_pages = nullptr, int n_first = 0);
int paged_window_launch(const fa_kv_cache &c, const void *q, void *o, float *lse, int Hq, int Tq, int left, int sinks,
                        float scale, void *workspace, cudaStream_t s);
// Where the states of the entries behind a prefix are, for the kernel that joins them with the prefix's.
struct OwnStates {
    const float *o, *lse;      // of units that one CTA had
    const float *part;         // of the others: two slots a CTA, [rows][d] then m, l [rows]
    const long long *where;    // the share of a CTA (0: whole units), and the first tile of each sequence
    const int *lens;
    int whole;                 // whole units, whatever `where` says
    int rows, RB, Hkv, kt, base, cap;
};
int paged_behind_launch(const fa_kv_cache &c, const void *q, float *o, float *lse, int Hq, int Tq, int causal, int base, float scale,
                        void *workspace, OwnStates *states, cudaStream_t s);
// Attention over a shared prefix and the entries behind it (fa_prefix_sm103.cu); n_pages > 0, pages of the prefix.
size_t prefix_workspace_bytes(int B, int Hq, int Hkv, int Tq, int max_len, int d, int codes, int n_pages, int page_size);
bool prefix_pays(const fa_kv_cache &c, int Hq, int Tq, int n_pages);
int prefix_launch(const fa_kv_cache &c, const void *q, void *o, float *lse, int Hq, int Tq, int causal, const int *pages,
                  int n_pages, float scale, void *workspace, cudaStream_t s);
int cache_status_fetch_clear(cudaStream_t s, int *host_word);
int paged_status_fetch_clear(cudaStream_t s, int *host_word);
int paged_range_status_fetch_clear(cudaStream_t s, int *host_word);
int prefix_status_fetch_clear(cudaStream_t s, int *host_word);

// The status words of the cache kernels are read from the first launch of one of them in this process
// on (a captured one may run again at any time): fa_sync_status of a program that has no cache costs no more for them.
enum StatusWords : int { STATUS_CACHE = 0, STATUS_PAGED = 1, STATUS_RANGE = 2, STATUS_PREFIX = 3 };
void status_in_use(StatusWords w);

}  // namespace fa
