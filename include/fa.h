/*
 * fa.h -- C ABI of libfa.so: IO-aware exact attention for GB300 (sm_103a).
 *
 * Every tensor is a plain device pointer to a contiguous row-major array:
 *   q, o, dO, dq : [B][H][Tq][d]      k, v, dk, dv : [B][H][Tk][d]
 *   lse          : [B][H][Tq] float32 (natural-log log-sum-exp of the scaled scores)
 * "bf16" tensors hold IEEE bfloat16 values; "f32" tensors hold float32.
 * Every base pointer must be 16-byte aligned.
 *
 * Semantics.  S = scale * Q K^T per (b, h); P = softmax(S) row-wise over the
 * allowed keys; O = P V; lse_r = log sum_l exp(S_rl).  With causal != 0 key l
 * is allowed for query r iff l <= r + (Tk - Tq) (bottom-right alignment; for
 * Tq == Tk this is "query r sees keys l <= r").  A query row with no allowed
 * key gets O = 0, lse = -inf and zero gradients.  scale must be finite and
 * > 0 (the usual value is 1/sqrt(d)); there is no implicit default.
 *
 * Sources (page titles and sections):
 *   zerotofrontier.app "FlashAttention" (Efficient attention 12.3):
 *     "The forward pass" -- O_i = diag(l)^-1 O~ and lse_i = m + log l written once;
 *     "The causal mask, and the tiles you never visit" -- the three tile kinds;
 *     "What the forward pass leaves behind" -- O plus one lse per row is all
 *       the backward pass needs;
 *     "The backward pass, derived" -- D_r = dO_r . O_r, dS = P o (dP - D),
 *       key blocks outside, dQ accumulated by atomic additions.
 *   atlas.blal.pro "FlashAttention -- IO-Aware Exact Attention":
 *     "Online softmax" and "Recomputation in the backward pass".
 *
 * Ownership.  The caller allocates and owns every buffer, including the
 * backward workspace.  The library keeps no per-call state; tensor maps are
 * built on the host per call and passed by value.  Calls are thread-safe.
 *
 * Errors.  Calls are asynchronous on `stream` (a cudaStream_t; NULL is the
 * legacy default stream).  The return value reports argument validation and
 * launch errors only.  A device-side failure (a bounded wait that timed out)
 * is recorded in a per-device status word and returned by fa_sync_status();
 * so is a length, count or page number in device memory that is out of range
 * (the cache calls below, which then leave that sequence or page alone).
 * On any nonzero return, no kernel was launched and outputs are untouched,
 * except FA_ERR_CUDA from a failed launch.
 */
#ifndef FA_H_
#define FA_H_

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    FA_OK = 0,
    FA_ERR_INVALID_ARG = 1,   /* null/misaligned pointer, bad size, aliasing outputs, bad scale */
    FA_ERR_UNSUPPORTED = 2,   /* head width not supported, or the device is not sm_103 */
    FA_ERR_CUDA = 3,          /* a CUDA runtime/driver call failed */
    FA_ERR_TIMEOUT = 4,       /* a device-side bounded wait ran out (from fa_sync_status) */
    FA_ERR_BAD_INDEX = 5      /* a length, count or page number on the device is out of range
                                 (from fa_sync_status) */
} fa_status;

typedef struct CUstream_st *fa_stream_t;   /* identical to cudaStream_t */

/*
 * Forward pass, bf16 in / bf16 O / f32 lse, fp32 accumulation on tcgen05
 * tensor cores.  d in {64, 128, 256}.  B, H, Tq, Tk >= 0; a call with
 * B*H*Tq == 0 is a no-op; Tk == 0 writes O = 0 and lse = -inf.
 * o and lse must not overlap q, k, v or each other.
 */
int fa_fwd(const void *q, const void *k, const void *v, void *o, float *lse,
           int B, int H, int Tq, int Tk, int d, int causal, float scale,
           fa_stream_t stream);

/*
 * Forward pass with f32 tensors and plain fp32 FFMA arithmetic (no tensor
 * cores): the debug/reference-precision build of the same tiled online
 * softmax.  Same shapes, rules and errors as fa_fwd.
 */
int fa_fwd_f32(const float *q, const float *k, const float *v, float *o, float *lse,
               int B, int H, int Tq, int Tk, int d, int causal, float scale,
               fa_stream_t stream);

/*
 * fa_fwd under a sliding window and/or a block mask (zerotofrontier.app
 * "FlashAttention", "Dropout, block-sparsity, and other real-kernel
 * details": windows are functions of (r, l) computed inside the tile, and
 * tiles a block mask marks empty are skipped exactly as causal tiles are).
 * Key l is allowed for query row r iff
 *     r + Tk - Tq - window_left <= l <= r + Tk - Tq + window_right
 * (-1 leaves that side unbounded: (-1, 0) is fa_fwd's causal mask, (-1, -1)
 * no mask) and, when block_mask is not NULL, its byte for the 128 x 128 block
 * (r / 128, l / 128) is nonzero.  block_mask is device memory, row-major
 * [mask_per_head ? B*H : 1][ceil(Tq / 128)][ceil(Tk / 128)], read-only,
 * owned by the caller, not overlapping o or lse.  Rows with no allowed key
 * get O = 0 and lse = -inf.  Other arguments and errors as fa_fwd; a window
 * side below -1 or mask_per_head outside {0, 1} is FA_ERR_INVALID_ARG.
 */
int fa_fwd_masked(const void *q, const void *k, const void *v, void *o, float *lse,
                  int B, int H, int Tq, int Tk, int d, int window_left, int window_right,
                  const unsigned char *block_mask, int mask_per_head, float scale,
                  fa_stream_t stream);

/*
 * fa_fwd under a causal sliding window with sinks: key l is allowed for query row r, at position
 * p = r + Tk - Tq, iff
 *     l <= p  and  (l >= p - window_left  or  l < n_sinks)
 * so that the first n_sinks keys stay visible to every row behind them, however far (window_left -1:
 * no left bound, plain causal).  Tiles between the sinks and the window are never loaded.  Other arguments and
 * errors as fa_fwd_masked; n_sinks >= 0, any number.
 */
int fa_fwd_sinks(const void *q, const void *k, const void *v, void *o, float *lse, int B, int H, int Tq, int Tk,
                 int d, int window_left, int n_sinks, float scale, fa_stream_t stream);

/*
 * FP8 forward (atlas.blal.pro "FlashAttention -- IO-Aware Exact Attention",
 * "The version ladder: FA1 -> FA2 -> FA3", the FA3 entry: e4m3 tensor-core
 * products with block quantization and incoherent processing; "Honest caveats &
 * open questions": a precision trade-off).  Two calls: fa_fp8_quantize turns the
 * bf16 q, k, v of fa_fwd into e4m3 codes and fp32 dequantization factors, and
 * fa_fwd_fp8 runs the forward over them.
 *
 * fa_fp8_quantize: q [B][H][Tq][d], k, v [B][H][Tk][d] bf16 as in fa_fwd.
 * signs: d fp32 values of +-1.0 in device memory (the random rotation), or NULL
 * for none.  With signs, each row x of q and k becomes x diag(signs) H (H the
 * Sylvester Hadamard matrix, unnormalised, in fp32), which leaves q k^T unchanged
 * up to the factor d folded into the descales.  Then, per 128-row block of q and of
 * k, the block's largest |value| a maps to 448: code = e4m3(x * (448 / a)), both
 * steps rounded to fp32, the last to nearest even with saturation; descale =
 * a / 448 (/ sqrt(d) with signs).  v gets one scale per channel over all Tk keys
 * and is stored transposed.  Outputs (device memory, caller-owned, 16-byte
 * aligned, overlapping nothing else):
 *   q8 [B][H][Tq][d], k8 [B][H][Tk][d]   e4m3 codes (one byte each);
 *   vt8 [B][H][d][fa_fp8_vt_stride(Tk)]  e4m3 codes of v transposed; the bytes of a
 *                                        row past Tk are zero;
 *   q_descale [B][H][ceil(Tq/128)], k_descale [B][H][ceil(Tk/128)],
 *   v_descale [B][H][d]                  fp32.
 * d in {64, 128, 256}; other errors as fa_fwd.
 *
 * fa_fwd_fp8: O and lse of attention over q^ = q8 * q_descale (per row block),
 * k^ = k8 * k_descale, v^ = vt8^T * v_descale (per channel):
 *     O = softmax(scale q^ k^T) v^,  lse = log sum exp(scale q^ k^T)
 * with fa_fwd's causal convention, output layouts and empty-row rules.  The
 * probabilities enter the P V product as e4m3 (relative rounding error at most
 * 2^-4 each); scores and the row sums stay fp32.  d = 128 only, else
 * FA_ERR_UNSUPPORTED.  Arguments as produced by fa_fp8_quantize with the same
 * sizes (every buffer 16-byte aligned); o and lse must not overlap them.  With
 * no elements (Tq = 0, or Tk = 0 for the key side) a buffer may be NULL.
 */
size_t fa_fp8_vt_stride(int Tk);          /* bytes per row of vt8: Tk rounded up to 16 */
int fa_fp8_quantize(const void *q, const void *k, const void *v, const float *signs,
                    int B, int H, int Tq, int Tk, int d, void *q8, void *k8, void *vt8,
                    float *q_descale, float *k_descale, float *v_descale, fa_stream_t stream);
int fa_fwd_fp8(const void *q8, const void *k8, const void *vt8, const float *q_descale,
               const float *k_descale, const float *v_descale, void *o, float *lse,
               int B, int H, int Tq, int Tk, int d, int causal, float scale, fa_stream_t stream);

/*
 * Split-KV attention for decoding: the O and lse of fa_fwd for a few query
 * rows per head against a long key/value sequence (atlas.blal.pro
 * "FlashAttention -- IO-Aware Exact Attention", "Honest caveats & open
 * questions": one query row leaves the tiled kernel idle; FlashDecoding
 * splits the keys instead).  Each chunk of 32-key tiles of a head is reduced
 * to a partial (m, l, O~) per row by the online softmax, and the chunks are
 * merged by its rescale (zerotofrontier.app "FlashAttention", "The forward
 * pass", step 2.5).  Same layouts, causal convention (bottom-right), scale
 * and edge cases as fa_fwd; scores and P stay fp32.  Tq must be at most 16
 * (d = 64, 128) or 8 (d = 256), else FA_ERR_UNSUPPORTED: use fa_fwd for more
 * rows.  workspace: at least fa_decode_workspace_bytes(...) bytes, 256-byte
 * aligned, not overlapping any argument; contents on entry ignored.  The
 * chunking depends on the sizes only, so results do not depend on the device.
 */
size_t fa_decode_workspace_bytes(int B, int H, int Tq, int Tk, int d);   /* 0: invalid or unsupported sizes */
int fa_decode(const void *q, const void *k, const void *v, void *o, float *lse,
              int B, int H, int Tq, int Tk, int d, int causal, float scale,
              void *workspace, size_t workspace_bytes, fa_stream_t stream);

/* ------------------------------------------------------------------------
 * Rotary positions and the paged key/value cache.  One serving step is
 *     fa_cache_append (rotate q and k, write k and v into the pages)
 *     fa_decode_paged (attend over the pages, add up the attention weights)
 *     fa_cache_evict  (now and then: give the least used entries back)
 * and fa_rope is the rotation by itself, before fa_fwd and, transposed, after
 * fa_bwd.
 * ------------------------------------------------------------------------ */

/* Element types of fa_rope and of a cache. */
typedef enum {
    FA_BF16 = 0,
    FA_F32 = 1,
    FA_E4M3 = 2
} fa_dtype;

/*
 * A [B][H][T][d] tensor by strides, in elements; the d values of a row are
 * contiguous.  Strides are nonnegative and, in bytes, multiples of 16 (a view
 * of a packed [B][T][heads][d] projection is one).
 */
typedef struct {
    void *data;
    long long stride_b, stride_h, stride_t;
    int H;
} fa_heads;

/*
 * Rotary positions with up to FA_ROPE_MAX_AXES axes (time, height, width, ...).
 * The first `rot` of the d features form rot / 2 pairs (x_i, y_i): features i
 * and i + rot / 2, or, interleaved, 2i and 2i + 1.  Pair i turns by
 * theta_i = p f_i with f_i its frequency (radians per position) and p the
 * token's position on the pair's axis:
 *     x_i' = x_i cos theta_i - y_i sin theta_i
 *     y_i' = y_i cos theta_i + x_i sin theta_i
 * Features from rot on pass through.  Angles are exact to 2^-32 turns plus the
 * rounding of f_i to 2^-64 turns times the position, however far the position.
 * Fill it with fa_rope_spec_init (host memory; nothing on the device).
 */
#define FA_ROPE_MAX_AXES 8
typedef struct {
    int d, rot, n_axes, interleaved;
    unsigned long long turns[128];   /* f_i / 2 pi in units of 2^-64 turns */
    unsigned char axis[128];
} fa_rope_spec;

/*
 * d in {64, 128, 256}; rot a multiple of 16, 16 <= rot <= d; freqs: rot / 2
 * finite values, |f| < 2^31; axis: rot / 2 values below n_axes (1 to
 * FA_ROPE_MAX_AXES), or NULL for axis 0 throughout; interleaved 0 or 1.
 */
int fa_rope_spec_init(fa_rope_spec *spec, int d, int rot, int n_axes, const double *freqs,
                      const unsigned char *axis, int interleaved);

/*
 * y = x rotated, for n (1 or 2, such as q and k) tensors that share B, T and
 * the positions: x[i], y[i] with x[i].H == y[i].H.  inverse = 1 turns the other
 * way, which is the rotation's transpose: applied to the gradient of y it gives
 * the gradient of x.  positions: int32 [n_axes][B][T] in device memory, any
 * value.  dtype FA_BF16 or FA_F32, for x and y alike; the arithmetic is fp32,
 * rounded once.  y[i] may be x[i] itself (same data and strides); otherwise no
 * element of y is shared with x, with the positions or within y (checked where
 * the tensors are contiguous; strided views of one buffer are the caller's
 * care).  B, T and H may be 0.
 */
int fa_rope(const fa_heads *x, const fa_heads *y, int n, const int *positions, const fa_rope_spec *spec,
            int B, int T, int dtype, int inverse, fa_stream_t stream);

/*
 * Norms of query and key heads with the rotation in the same pass.  A row x of d features becomes the
 * rotation of w x / sqrt(mean(x^2) + eps): x[0] (such as q) with weights q_weight, x[1] (such as k)
 * with k_weight, [d] each for all heads, bf16 or f32 (dtype), 16-byte aligned; NULL: ones.  eps finite
 * and > 0.  The arithmetic is fp32, rounded once; the squares' sum must not leave fp32.
 */
typedef struct {
    const void *q_weight, *k_weight;
    int d, dtype;
    float eps;
} fa_head_norm;

/*
 * y = x normed and rotated: tensors, positions, spec and errors as in fa_rope (norm->d == spec->d; no
 * output shares memory with the weights).
 */
int fa_norm_rope(const fa_heads *x, const fa_heads *y, int n, const fa_head_norm *norm, const int *positions,
                 const fa_rope_spec *spec, int B, int T, int dtype, fa_stream_t stream);

/*
 * Backward of fa_norm_rope: dx[i], the gradient of x[i], from dy[i], the gradient of y[i], and x[i]
 * itself (not y[i]: where fa_norm_rope's output took its input's place there is no backward).  dx[i]
 * may be dy[i]; otherwise no output shares memory with an input.  dq_weight and dk_weight: f32 [d],
 * 16-byte aligned, the gradients of the weights (of either type), summed in fp32 over all rows in a fixed order;
 * each may be NULL, and is where its weight is.  They are written, not added to: zeros where there are
 * no rows.  workspace: fa_norm_rope_bwd_workspace_bytes(d) bytes, 256-byte aligned, contents on entry
 * ignored, not shared by calls that may overlap in time; not needed without gradients of weights.
 */
size_t fa_norm_rope_bwd_workspace_bytes(int d);   /* 0: unsupported width */
int fa_norm_rope_bwd(const fa_heads *dy, const fa_heads *x, const fa_heads *dx, int n, const fa_head_norm *norm,
                     const int *positions, const fa_rope_spec *spec, int B, int T, int dtype, float *dq_weight,
                     float *dk_weight, void *workspace, size_t workspace_bytes, fa_stream_t stream);

/*
 * A paged cache of B sequences, all pointers to device memory:
 *   k, v         [num_pages][Hkv][page_size][d], bf16 (FA_BF16) or e4m3 codes
 *                (FA_E4M3)
 *   k_scale, v_scale  [Hkv] f32, FA_E4M3 only: a code c of head h stands for
 *                c * scale[h] (2^-64 to 2^64); NULL for FA_BF16
 *   block_table  [B][max_pages] int32: entry i of sequence b (its slot i) is
 *                row i % page_size of page block_table[b][i / page_size]
 *   lens         [B] int32: entries of each sequence, 0 to max_pages * page_size
 *   seen         [B] int32: tokens ever appended to each sequence; NULL: lens
 *                (right until something is evicted)
 *   weight       [B][Hkv][max_pages * page_size] f32: accumulated attention
 *                weight of each entry, or NULL
 *   order        [B][Hkv][max_pages * page_size] int32: arrival number of each
 *                entry (the first token of a sequence has 0), or NULL
 * k and v are 128-byte, weight and order 16-byte, the other arrays 4-byte aligned;
 * an array without an element may be NULL.
 * page_size is 16, 32, 64, 128 or 256; d 64, 128 or 256.  Only the pages and
 * rows in front of lens are read: what lies behind them may hold anything.
 * Sequences may share pages that none of them writes to (fa_cache_append and
 * fa_cache_evict write).  num_pages * Hkv and B * Hkv must fit in 31 bits;
 * max_pages * page_size is at most 2^30.  The struct is read during the call only; a page
 * number outside 0 .. num_pages - 1 in front of lens, or a length outside its
 * range, is FA_ERR_BAD_INDEX from fa_sync_status and is never dereferenced.
 */
typedef struct {
    void *k, *v;
    const float *k_scale, *v_scale;
    const int *block_table;
    const int *lens;
    const int *seen;
    float *weight;
    int *order;
    int B, Hkv, d, page_size, num_pages, max_pages;
    int dtype;
} fa_kv_cache;

/*
 * Writes new tokens into the cache.  k and v: bf16 [B][Hkv][T][d] by strides.
 * Of sequence b the first new_lens[b] (NULL: T) of its T rows are new tokens;
 * `lens` counts them already: they take slots lens[b] - new_lens[b] up to
 * lens[b] - 1, in order, with weight 0 and arrival number seen[b] - new_lens[b]
 * onwards.  Rows past new_lens[b] are not read, and nothing else is written.
 * With a spec, k is rotated first (fp32, positions as in fa_rope: [n_axes][B][T]),
 * and q, if given, is rotated into q_out (bf16 [B][Hq][T][d] by strides; q_out
 * may be q; rows past new_lens[b] are left alone).  Without a spec, positions, q
 * and q_out are NULL.  What is written is the fp32 value rounded once to bf16,
 * or to e4m3 after division by the head's scale (to nearest even, saturating at
 * +-448; NaN stays NaN).  The new rows of different sequences must fall on
 * different pages.  A sequence with new_lens outside 0 .. min(T, lens) is left
 * alone (FA_ERR_BAD_INDEX).
 */
int fa_cache_append(const fa_kv_cache *cache, const fa_heads *k, const fa_heads *v, const fa_heads *q,
                    const fa_heads *q_out, const int *positions, const fa_rope_spec *spec,
                    const int *new_lens, int T, fa_stream_t stream);

/*
 * fa_cache_append with the rows of q and k normed before they are rotated (fa_head_norm above; v is
 * written as it is).  norm needs a spec with norm->d == spec->d; NULL: fa_cache_append.  The weights lie
 * outside of the cache and of q_out.
 */
int fa_cache_append_norm(const fa_kv_cache *cache, const fa_heads *k, const fa_heads *v, const fa_heads *q,
                         const fa_heads *q_out, const int *positions, const fa_rope_spec *spec, const fa_head_norm *norm,
                         const int *new_lens, int T, fa_stream_t stream);

/*
 * Attention of the last Tq (1 to 16) tokens of every sequence over the cache:
 * q, o bf16 [B][Hq][Tq][d], lse f32 [B][Hq][Tq], contiguous.  Hq is a multiple
 * of Hkv; query head h reads KV head h / (Hq / Hkv).  With causal != 0 row t sees
 * slots up to lens[b] - Tq + t (bottom-right, as fa_decode; the Tq rows' own
 * tokens are the last entries), else every slot.  A row that sees nothing gets
 * O = 0 and lse = -inf.  An infinity or NaN in the v of an entry that any row of
 * the call sees may reach every row of its head group.  Scores, statistics and
 * the row sums are fp32; a probability meets v with 16 bits, in an FA_E4M3 cache
 * with 11, or, below 2^-29 of the row's largest, to a multiple of 2^-39 of it.
 * There q meets the codes exactly, but a feature below 2^-31 of its row's largest
 * to a multiple of 2^-38 of that.
 * The keys are split over the thread blocks in equal shares of the whole batch,
 * and partial results are joined in a fixed order: the same call gives the same
 * bits, but a sequence's last bits may depend on the other lengths.
 * accumulate = 1 adds, for every entry, the sum of its probabilities over the
 * head group's rows (Hq / Hkv heads x Tq) to cache->weight.
 * Its time and workspace, and the time of fa_cache_evict, grow with the table's
 * max_pages * page_size and not with lens alone.
 * workspace: fa_decode_paged_workspace_bytes bytes, 256-byte aligned, contents
 * on entry ignored, not shared by calls that may overlap in time.  A sequence
 * with a length out of range counts as empty, a page out of range as masked.
 */
size_t fa_decode_paged_workspace_bytes(int B, int Hq, int Hkv, int Tq, int max_pages, int page_size, int d,
                                       int accumulate);   /* 0: invalid or unsupported sizes */
int fa_decode_paged(const fa_kv_cache *cache, const void *q, void *o, float *lse, int Hq, int Tq, int causal,
                    float scale, int accumulate, void *workspace, size_t workspace_bytes, fa_stream_t stream);

/*
 * fa_decode_paged, causal, under a sliding window with sinks: the row at position p = lens[b] - Tq + t sees
 * slot j iff
 *     j <= p  and  (j >= p - window_left  or  j < n_sinks)
 * (window_left -1: no left bound).  Slots, not arrival numbers: in a cache that fa_cache_evict has reordered
 * the two differ.  Time goes with the visible slots, not with lens.  Pages without a slot that some row sees are not
 * read and their table entries not looked at: they may have been given back.  No accumulated weights.
 * workspace: fa_decode_paged_workspace_bytes(..., accumulate = 0); other arguments, results and errors as there.
 */
int fa_decode_paged_window(const fa_kv_cache *cache, const void *q, void *o, float *lse, int Hq, int Tq,
                           int window_left, int n_sinks, float scale, void *workspace, size_t workspace_bytes,
                           fa_stream_t stream);

/*
 * fa_decode_paged for a batch whose sequences all begin with the same n_prefix_pages full pages,
 * prefix_pages (int32, device memory), which stands for the first entries of every sequence's row of the block table:
 * those are not looked at.  The prefix is read once for the rows of all sequences, in matrix products of
 * 128 rows; each sequence's own entries, behind it, as by fa_decode_paged; and the two are joined.  (Where the sizes
 * say that reading so little for every sequence is faster, it is, by fa_decode_paged's kernel.)  Results as
 * fa_decode_paged's, except that a probability meets a v of the prefix as bf16, 2^-8 of it off at most, and that
 * an infinity or NaN in the v of a prefix's entry may reach every row of its KV head in the batch.  A sequence
 * may be shorter than the prefix (one of length 0, a place of the batch without a request, sees
 * nothing).  A page of prefix_pages out of range counts as masked for all (FA_ERR_BAD_INDEX; where no sequence
 * reaches it, it may go unreported).  n_prefix_pages 0 to max_pages; 0 is fa_decode_paged.  workspace: fa_decode_paged_shared_workspace_bytes bytes (dtype: the cache's),
 * 256-byte aligned, contents on entry ignored, not shared by calls that may overlap in time.
 */
size_t fa_decode_paged_shared_workspace_bytes(int B, int Hq, int Hkv, int Tq, int max_pages, int page_size, int d,
                                              int dtype, int n_prefix_pages);   /* 0: invalid or unsupported sizes */
int fa_decode_paged_shared(const fa_kv_cache *cache, const void *q, void *o, float *lse, int Hq, int Tq, int causal,
                           const int *prefix_pages, int n_prefix_pages, float scale, void *workspace,
                           size_t workspace_bytes, fa_stream_t stream);

/*
 * Evicts, for every sequence and KV head on its own, down to `budget` (1 to 2^30)
 * entries.  Kept are the min(lens, budget) first ones in this order: protected
 * entries (arrival number below n_first, or at least seen - n_recent), then by
 * larger weight, a NaN counting as the least; of equals the lower slot.  The
 * kept entries that lie behind the new length move, in order, into the slots of
 * the evicted ones in front of it: nothing else moves, so the order of slots is
 * not the order of arrival afterwards (`order` has that).  Written:
 *   K and V rows of the moved entries, in place;
 *   kept       [B][Hkv][budget] int32: the old slot of each entry, -1 behind the
 *              new length;
 *   weight_out, order_out  like cache->weight and cache->order (which they may
 *              be), the entries in front of the new length only; order_out NULL
 *              exactly when cache->order is;
 *   lens_out   [B] int32 (may be cache->lens): min(lens, budget), or lens where it
 *              is out of range.
 * n_first, n_recent >= 0 with n_first + n_recent <= budget; either one > 0 needs
 * cache->order.  cache->weight is needed.  A sequence with a length out of range
 * is left alone; so is a row whose page is out of range.
 */
int fa_cache_evict(const fa_kv_cache *cache, int budget, int n_first, int n_recent, float *weight_out,
                   int *order_out, int *lens_out, int *kept, fa_stream_t stream);

/*
 * Bytes of device workspace fa_bwd and fa_bwd_deterministic need for these
 * sizes: a log2-domain copy of lse and the row terms D (each [B][H][Tq_pad]
 * f32), the dQ accumulator [B][H][Tq_pad][d] (f32, or int32 fixed point in
 * fa_bwd_deterministic), two f32 per head and one int32 per 128-row query
 * block (the fixed-point bounds), where Tq_pad rounds Tq up to a multiple of
 * 128; each region is 256-byte aligned.  Returns 0 for invalid sizes.
 */
size_t fa_bwd_workspace_bytes(int B, int H, int Tq, int Tk, int d);

/*
 * Backward pass, bf16 q, k, v, o, dO, dq, dk, dv; f32 lse.  o and lse must be
 * what fa_fwd returned for the same q, k, v, causal and scale.  d in {64, 128}
 * (d = 256 returns FA_ERR_UNSUPPORTED).  workspace must hold at least
 * fa_bwd_workspace_bytes(...) bytes, 256-byte aligned; its contents on entry
 * are ignored.  dq, dk, dv must not overlap any input, the workspace or each
 * other.  dQ is accumulated with fp32 atomic additions, so its last bits may
 * differ from run to run.
 */
int fa_bwd(const void *q, const void *k, const void *v, const void *o, const float *lse,
           const void *dO, void *dq, void *dk, void *dv,
           int B, int H, int Tq, int Tk, int d, int causal, float scale,
           void *workspace, size_t workspace_bytes, fa_stream_t stream);

/*
 * fa_bwd with dq bitwise the same on every run with the same inputs
 * (zerotofrontier.app "FlashAttention", "The backward pass, derived", "Which
 * loop goes outside?": dQ_i is a sum over key blocks added by different
 * thread blocks, and floating-point additions in arrival order make its last
 * bits vary between runs).  Here the contributions are added as int32 fixed
 * point, whose sums do not depend on the order: query block i (128 rows) uses
 * the grid 2^(e-30) where 2^e exceeds the bound 2 |dO_r|_2 max_l |V_l|_2
 * max |K| of every partial sum of its rows (the rows of P sum to one), so
 * nothing overflows and each term is rounded to about 1e-9 of that bound.
 * dk and dv are computed as by fa_bwd.  It costs one more pass over K and V
 * (the per-head maxima) and the conversions.  Non-finite inputs give no
 * meaningful dq.  Arguments, workspace, validation and errors are those of
 * fa_bwd.
 */
int fa_bwd_deterministic(const void *q, const void *k, const void *v, const void *o,
                         const float *lse, const void *dO, void *dq, void *dk, void *dv,
                         int B, int H, int Tq, int Tk, int d, int causal, float scale,
                         void *workspace, size_t workspace_bytes, fa_stream_t stream);

/*
 * Backward of fa_fwd_masked: the gradients under the same window and block
 * mask (see fa_fwd_masked for their meaning, layout and ownership; o and lse
 * must come from fa_fwd_masked with the same mask).  Each 128-key block
 * visits only the query blocks that its window and mask admit.
 * deterministic = 1 selects fa_bwd_deterministic's order-independent dQ.
 * Other arguments, workspace and errors as fa_bwd; window sides below -1,
 * mask_per_head or deterministic outside {0, 1} are FA_ERR_INVALID_ARG.
 */
int fa_bwd_masked(const void *q, const void *k, const void *v, const void *o,
                  const float *lse, const void *dO, void *dq, void *dk, void *dv,
                  int B, int H, int Tq, int Tk, int d, int window_left, int window_right,
                  const unsigned char *block_mask, int mask_per_head, int deterministic,
                  float scale, void *workspace, size_t workspace_bytes, fa_stream_t stream);

/*
 * Backward of fa_fwd_sinks (o and lse from it, with the same window and sinks).  Each 128-key block visits
 * the query blocks of its window; blocks with sinks, which every query block behind them sees, are
 * cut into parts where one of them would outlast the rest, with fp32 sums joined in a fixed order: the workspace is
 * fa_bwd_sinks_workspace_bytes(...) (at least fa_bwd_workspace_bytes; 0 for invalid sizes).
 * deterministic = 1 selects fa_bwd_deterministic's order-independent dQ.  Other arguments and errors as
 * fa_bwd.
 */
size_t fa_bwd_sinks_workspace_bytes(int B, int H, int Tq, int Tk, int d, int window_left, int n_sinks);
int fa_bwd_sinks(const void *q, const void *k, const void *v, const void *o, const float *lse, const void *dO,
                 void *dq, void *dk, void *dv, int B, int H, int Tq, int Tk, int d, int window_left, int n_sinks,
                 int deterministic, float scale, void *workspace, size_t workspace_bytes, fa_stream_t stream);

/*
 * One stage of fa_bwd, for callers that schedule or time the three kernels
 * separately: stage 1 computes D_r = dO_r . O_r and the log2-domain lse into
 * the workspace and zeroes the dQ accumulator; stage 2 runs the tile loop
 * (recomputes P from lse, writes dK and dV, adds dQ into the accumulator);
 * stage 3 scales the accumulator by `scale` and writes dq.  Running stages
 * 1, 2, 3 in that order on one stream with the same arguments and workspace
 * is exactly fa_bwd.  Arguments, validation and errors are those of fa_bwd;
 * stage outside 1..3 returns FA_ERR_INVALID_ARG.
 */
int fa_bwd_stage(int stage, const void *q, const void *k, const void *v, const void *o,
                 const float *lse, const void *dO, void *dq, void *dk, void *dv,
                 int B, int H, int Tq, int Tk, int d, int causal, float scale,
                 void *workspace, size_t workspace_bytes, fa_stream_t stream);

/*
 * Size of the fixed device scratch array behind fa_bwd_noalloc (64 MiB).  It
 * holds fa_bwd_workspace_bytes(B, H, Tq, Tk, d) bytes, about 520 bytes per
 * padded query row at d = 128 and 264 at d = 64, when B*H*Tq_pad is at most
 * about 129,000 rows at d = 128 (B8 H8 T1920, B1 H32 T3840; not B8 H8 T2048)
 * or 254,000 rows at d = 64 (B8 H16 T1920), where Tq_pad rounds Tq up to 128.
 */
#define FA_BWD_NOALLOC_SCRATCH_BYTES (64u << 20)

/*
 * fa_bwd for callers that cannot allocate device memory.  The pages have no
 * counterpart: this serves callers that are handed only their input and
 * output buffers and may not call cudaMalloc -- plug-ins whose host framework
 * owns all device memory and offers them no allocator, or latency-critical
 * code that cannot take cudaMalloc's implicit device synchronisation.
 * Arguments, results and errors are those of fa_bwd without the workspace:
 * the scratch comes from a fixed array of FA_BWD_NOALLOC_SCRATCH_BYTES that
 * the library keeps in device memory (each device holds it until the process
 * exits).  The call allocates nothing.
 *   - Arguments are checked as fa_bwd checks them (FA_ERR_INVALID_ARG,
 *     FA_ERR_UNSUPPORTED for d = 256) before anything else.  Then sizes whose
 *     fa_bwd_workspace_bytes(...) exceeds FA_BWD_NOALLOC_SCRATCH_BYTES return
 *     FA_ERR_UNSUPPORTED, still before any CUDA call; use fa_bwd with a
 *     caller-owned workspace for those.
 *   - The first call on a device looks the array's device address up
 *     (cudaGetSymbolAddress, with that device current) and caches it with the
 *     current CUDA context; make that first call before any stream capture.
 *     A call under a different context (after cudaDeviceReset, for one) looks
 *     the address up again, so make the first call after a reset before any
 *     capture too.
 *   - Every call on a device shares the one array.  Each call rewrites all of
 *     the scratch it uses before reading it (the dQ accumulator is zeroed),
 *     so nothing carries over between calls, but calls that overlap on the
 *     GPU (different streams or threads on one device) race and corrupt each
 *     other's results: order them, e.g. on one stream.
 */
int fa_bwd_noalloc(const void *q, const void *k, const void *v, const void *o, const float *lse,
                   const void *dO, void *dq, void *dk, void *dv,
                   int B, int H, int Tq, int Tk, int d, int causal, float scale,
                   fa_stream_t stream);

/*
 * Synchronises `stream`, then returns and clears the device status word of
 * the current device: FA_OK, FA_ERR_TIMEOUT (a kernel's bounded wait ran out;
 * its outputs are invalid), FA_ERR_BAD_INDEX (see fa_kv_cache; where both
 * happened, FA_ERR_TIMEOUT) or FA_ERR_CUDA (the synchronise failed).
 */
int fa_sync_status(fa_stream_t stream);

/* Static, never-NULL description of a status code. */
const char *fa_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* FA_H_ */
