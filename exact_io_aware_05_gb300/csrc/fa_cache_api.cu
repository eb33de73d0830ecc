// fa_cache_api.cu -- the C ABI of the rotary positions and the paged key/value cache
// (declared in include/fa.h): argument validation and the rotation's table of phases.  No
// compute happens here; the kernels are in fa_cache_sm103.cu and fa_paged_sm103.cu.
#include <climits>
#include <cmath>
#include <cstring>

#include "../../include/fa.h"
#include "fa_internal.h"

namespace {

// Slots of a sequence, and the budget of an eviction: slot numbers past the end of a tile, and a loop's step
// past the budget, fit an int.
constexpr long long kMaxSlots = 1ll << 30;

bool width_ok(int d) { return d == 64 || d == 128 || d == 256; }
bool page_size_ok(int ps) { return ps == 16 || ps == 32 || ps == 64 || ps == 128 || ps == 256; }

// A strided [B][H][T][d] tensor: present, 16-byte aligned rows, strides in range.
bool heads_ok(const fa_heads *x, int elem)
{
    if (!x || x->H < 0)
        return false;
    if (x->stride_b < 0 || x->stride_h < 0 || x->stride_t < 0)
        return false;
    const long long m = 16 / elem;
    return x->stride_b % m == 0 && x->stride_h % m == 0 && x->stride_t % m == 0;
}

bool heads_present(const fa_heads *x, size_t n) { return n == 0 || (x->data && fa::aligned16(x->data)); }

bool contiguous(const fa_heads *x, int B, int T, int d)
{
    return (x->stride_t == d || T <= 1) && (x->stride_h == (long long)T * d || x->H <= 1) &&
           (x->stride_b == (long long)x->H * T * d || B <= 1);
}

bool same_place(const fa_heads *a, const fa_heads *b, int B, int T)
{
    return a->data == b->data && (a->stride_b == b->stride_b || B <= 1) && (a->stride_h == b->stride_h || a->H <= 1) &&
           (a->stride_t == b->stride_t || T <= 1);
}

// Rows of an output must not be each other: each stride at least spans what lies inside it,
// in some order of the three.  (Sorted by stride, each must be >= the extent below it.)
bool self_disjoint(const fa_heads *x, int B, int T, int d)
{
    long long st[3] = {x->stride_b, x->stride_h, x->stride_t};
    long long n[3] = {B, x->H, T};
    for (int i = 0; i < 3; ++i)
        for (int j = i + 1; j < 3; ++j)
            if (st[j] < st[i]) {
                const long long a = st[i], b = n[i];
                st[i] = st[j], n[i] = n[j];
                st[j] = a, n[j] = b;
            }
    long long ext = d;
    for (int i = 0; i < 3; ++i) {
        if (n[i] <= 1)
            continue;
        if (st[i] < ext)
            return false;
        ext += st[i] * (n[i] - 1);
    }
    return true;
}

bool spec_ok(const fa_rope_spec *s)
{
    if (!s || !width_ok(s->d) || s->rot < 16 || s->rot > s->d || s->rot % 16 != 0)
        return false;
    if (s->n_axes < 1 || s->n_axes > FA_ROPE_MAX_AXES || s->interleaved < 0 || s->interleaved > 1)
        return false;
    for (int i = 0; i < s->rot / 2; ++i)
        if (s->axis[i] >= s->n_axes)
            return false;
    return true;
}

// Everything about a cache that the host can see.  OK also when B == 0.
int cache_check(const fa_kv_cache *c)
{
    if (!c || c->B < 0 || c->Hkv < 1 || c->num_pages < 0 || c->max_pages < 0)
        return FA_ERR_INVALID_ARG;
    if (c->dtype != FA_BF16 && c->dtype != FA_E4M3)
        return FA_ERR_INVALID_ARG;
    if (!width_ok(c->d))
        return FA_ERR_UNSUPPORTED;
    const int ps = c->page_size;
    if (!page_size_ok(ps))
        return FA_ERR_UNSUPPORTED;
    if ((long long)c->num_pages * c->Hkv > INT_MAX || (long long)c->B * c->Hkv > INT_MAX ||
        (long long)c->max_pages * ps > kMaxSlots)
        return FA_ERR_INVALID_ARG;
    if (c->B == 0)
        return FA_OK;
    if (!c->lens || (c->max_pages > 0 && !c->block_table))
        return FA_ERR_INVALID_ARG;
    if (c->num_pages > 0 && (!c->k || !c->v))
        return FA_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(c->k) & 127u) || (reinterpret_cast<uintptr_t>(c->v) & 127u))
        return FA_ERR_INVALID_ARG;
    const uintptr_t words = reinterpret_cast<uintptr_t>(c->lens) | reinterpret_cast<uintptr_t>(c->block_table) |
                            reinterpret_cast<uintptr_t>(c->seen) | reinterpret_cast<uintptr_t>(c->k_scale) |
                            reinterpret_cast<uintptr_t>(c->v_scale);
    if ((words & 3u) || !fa::aligned16(c->weight) || !fa::aligned16(c->order))
        return FA_ERR_INVALID_ARG;
    if ((c->dtype == FA_E4M3) != (c->k_scale != nullptr) || (c->dtype == FA_E4M3) != (c->v_scale != nullptr))
        return FA_ERR_INVALID_ARG;
    return FA_OK;
}

size_t pool_bytes(const fa_kv_cache *c)
{
    return (size_t)c->num_pages * c->Hkv * c->page_size * c->d * (c->dtype == FA_E4M3 ? 1 : 2);
}

size_t slots_bytes(const fa_kv_cache *c) { return (size_t)c->B * c->Hkv * c->max_pages * c->page_size * 4; }

// Whether [p, p + n) touches any part of the cache; `state`: weight, order and lens too.
bool touches_cache(const fa_kv_cache *c, const void *p, size_t n, bool state)
{
    const size_t np = pool_bytes(c);
    if (fa::overlaps(p, n, c->k, np) || fa::overlaps(p, n, c->v, np) ||
        fa::overlaps(p, n, c->block_table, (size_t)c->B * c->max_pages * 4) ||
        fa::overlaps(p, n, c->seen, (size_t)c->B * 4) || fa::overlaps(p, n, c->k_scale, (size_t)c->Hkv * 4) ||
        fa::overlaps(p, n, c->v_scale, (size_t)c->Hkv * 4))
        return true;
    return state && (fa::overlaps(p, n, c->lens, (size_t)c->B * 4) || fa::overlaps(p, n, c->weight, slots_bytes(c)) ||
                     fa::overlaps(p, n, c->order, slots_bytes(c)));
}

// K and V of one cache must be different memory, and its state not inside them.
bool cache_disjoint(const fa_kv_cache *c)
{
    const size_t np = pool_bytes(c), ns = slots_bytes(c);
    return !fa::overlaps(c->k, np, c->v, np) && !touches_cache(c, c->weight, ns, false) &&
           !touches_cache(c, c->order, ns, false) && !touches_cache(c, c->lens, (size_t)c->B * 4, false) &&
           !fa::overlaps(c->weight, ns, c->order, ns) && !fa::overlaps(c->weight, ns, c->lens, (size_t)c->B * 4) &&
           !fa::overlaps(c->order, ns, c->lens, (size_t)c->B * 4);
}

}  // namespace

extern "C" {

int fa_rope_spec_init(fa_rope_spec *spec, int d, int rot, int n_axes, const double *freqs, const unsigned char *axis,
                      int interleaved)
{
    if (!spec || !freqs)
        return FA_ERR_INVALID_ARG;
    if (!width_ok(d))
        return FA_ERR_UNSUPPORTED;
    if (rot < 16 || rot > d || rot % 16 != 0 || n_axes < 1 || n_axes > FA_ROPE_MAX_AXES || interleaved < 0 ||
        interleaved > 1)
        return FA_ERR_INVALID_ARG;
    fa_rope_spec s;
    std::memset(&s, 0, sizeof(s));
    s.d = d;
    s.rot = rot;
    s.n_axes = n_axes;
    s.interleaved = interleaved;
    // 1 / (2 pi) as the sum of two doubles: the product below is good to about 2^-105
    constexpr double kInv2PiHi = 0.15915494309189535, kInv2PiLo = -9.839338337591243e-18;
    for (int i = 0; i < rot / 2; ++i) {
        const double f = freqs[i];
        if (!std::isfinite(f) || std::fabs(f) >= 2147483648.0)
            return FA_ERR_INVALID_ARG;
        const double hi = f * kInv2PiHi;
        const double lo = std::fma(f, kInv2PiHi, -hi) + f * kInv2PiLo;
        // the turns behind the point, exactly; in units of 2^-64 turns (sums wrap modulo one turn)
        const double units = std::ldexp(std::fabs(hi - std::trunc(hi)), 64);   // below 2^64
        const unsigned long long whole = static_cast<unsigned long long>(units);
        const double rest = units - static_cast<double>(whole);
        const double fine = (hi < 0 ? -rest : rest) + std::ldexp(lo, 64);
        s.turns[i] = (hi < 0 ? 0ull - whole : whole) +
                     static_cast<unsigned long long>(static_cast<long long>(std::nearbyint(fine)));
        s.axis[i] = axis ? axis[i] : 0;
        if (s.axis[i] >= n_axes)
            return FA_ERR_INVALID_ARG;
    }
    *spec = s;
    return FA_OK;
}

int fa_rope(const fa_heads *x, const fa_heads *y, int n, const int *positions, const fa_rope_spec *spec, int B, int T,
            int dtype, int inverse, fa_stream_t stream)
{
    if (!x || !y || n < 1 || n > 2 || B < 0 || T < 0 || inverse < 0 || inverse > 1)
        return FA_ERR_INVALID_ARG;
    if (dtype != FA_BF16 && dtype != FA_F32)
        return FA_ERR_INVALID_ARG;
    if (!spec_ok(spec))
        return FA_ERR_INVALID_ARG;
    const int elem = dtype == FA_F32 ? 4 : 2, d = spec->d;
    const size_t np = (size_t)spec->n_axes * B * T * 4;
    if ((long long)B * T > INT_MAX)
        return FA_ERR_INVALID_ARG;
    long long rows = 0, heads = 0;
    for (int i = 0; i < n; ++i) {
        if (!heads_ok(&x[i], elem) || !heads_ok(&y[i], elem) || x[i].H != y[i].H)
            return FA_ERR_INVALID_ARG;
        const size_t rows_i = (size_t)B * x[i].H * T;
        if (!heads_present(&x[i], rows_i) || !heads_present(&y[i], rows_i))
            return FA_ERR_INVALID_ARG;
        if (rows_i > 0 && !self_disjoint(&y[i], B, T, d))
            return FA_ERR_INVALID_ARG;
        rows += (long long)rows_i;
        heads += x[i].H;
    }
    if (heads > INT_MAX)
        return FA_ERR_INVALID_ARG;
    if (rows == 0)
        return FA_OK;
    if (!positions || (reinterpret_cast<uintptr_t>(positions) & 3u))
        return FA_ERR_INVALID_ARG;
    for (int i = 0; i < n; ++i) {
        if (!contiguous(&y[i], B, T, d))
            continue;
        const size_t ny = (size_t)B * y[i].H * T * d * elem;
        if (fa::overlaps(y[i].data, ny, positions, np))
            return FA_ERR_INVALID_ARG;
        for (int j = 0; j < n; ++j) {
            const size_t nx = (size_t)B * x[j].H * T * d * elem;
            if (contiguous(&x[j], B, T, d) && !(i == j && same_place(&x[j], &y[i], B, T)) &&
                fa::overlaps(y[i].data, ny, x[j].data, nx))
                return FA_ERR_INVALID_ARG;
            if (j != i && contiguous(&y[j], B, T, d) && fa::overlaps(y[i].data, ny, y[j].data, nx))
                return FA_ERR_INVALID_ARG;
        }
    }
    const int st = fa::check_device();
    if (st != fa::OK)
        return st;
    return fa::rope_launch(x, y, n, positions, *spec, B, T, dtype, inverse, reinterpret_cast<cudaStream_t>(stream));
}

int fa_cache_append(const fa_kv_cache *cache, const fa_heads *k, const fa_heads *v, const fa_heads *q,
                    const fa_heads *q_out, const int *positions, const fa_rope_spec *spec, const int *new_lens, int T,
                    fa_stream_t stream)
{
    int st = cache_check(cache);
    if (st != FA_OK)
        return st;
    const int B = cache->B, d = cache->d;
    if (T < 0 || (long long)B * T > INT_MAX || !heads_ok(k, 2) || !heads_ok(v, 2) || k->H != cache->Hkv ||
        v->H != cache->Hkv)
        return FA_ERR_INVALID_ARG;
    if (spec ? (!spec_ok(spec) || spec->d != d) : (positions || q || q_out))
        return FA_ERR_INVALID_ARG;
    if ((q != nullptr) != (q_out != nullptr))
        return FA_ERR_INVALID_ARG;
    if (q && (!heads_ok(q, 2) || !heads_ok(q_out, 2) || q->H != q_out->H || (long long)q->H + 2ll * cache->Hkv > INT_MAX))
        return FA_ERR_INVALID_ARG;
    if ((size_t)B * T == 0)
        return FA_OK;
    const size_t rows = (size_t)B * T;
    if (!heads_present(k, rows) || !heads_present(v, rows) || (spec && !positions) ||
        ((reinterpret_cast<uintptr_t>(positions) | reinterpret_cast<uintptr_t>(new_lens)) & 3u))
        return FA_ERR_INVALID_ARG;
    if (!cache_disjoint(cache))
        return FA_ERR_INVALID_ARG;
    const size_t nk = rows * cache->Hkv * d * 2, npos = spec ? (size_t)spec->n_axes * rows * 4 : 0;
    if ((contiguous(k, B, T, d) && touches_cache(cache, k->data, nk, true)) ||
        (contiguous(v, B, T, d) && touches_cache(cache, v->data, nk, true)) ||
        touches_cache(cache, positions, npos, true) || fa::overlaps(new_lens, (size_t)B * 4, cache->k, pool_bytes(cache)) ||
        fa::overlaps(new_lens, (size_t)B * 4, cache->v, pool_bytes(cache)) ||
        fa::overlaps(new_lens, (size_t)B * 4, cache->weight, slots_bytes(cache)) ||
        fa::overlaps(new_lens, (size_t)B * 4, cache->order, slots_bytes(cache)))
        return FA_ERR_INVALID_ARG;
    if (q && q->H > 0) {
        const size_t nq = rows * q->H * d * 2;
        if (!heads_present(q, rows) || !heads_present(q_out, rows) || !self_disjoint(q_out, B, T, d))
            return FA_ERR_INVALID_ARG;
        if (contiguous(q, B, T, d) && touches_cache(cache, q->data, nq, true))
            return FA_ERR_INVALID_ARG;
        if (contiguous(q_out, B, T, d)) {
            if (touches_cache(cache, q_out->data, nq, true) || fa::overlaps(q_out->data, nq, positions, npos) ||
                fa::overlaps(q_out->data, nq, new_lens, new_lens ? (size_t)B * 4 : 0) ||
                (contiguous(q, B, T, d) && !same_place(q, q_out, B, T) && fa::overlaps(q_out->data, nq, q->data, nq)) ||
                (contiguous(k, B, T, d) && fa::overlaps(q_out->data, nq, k->data, nk)) ||
                (contiguous(v, B, T, d) && fa::overlaps(q_out->data, nq, v->data, nk)))
                return FA_ERR_INVALID_ARG;
        }
    }
    if ((st = fa::check_device()) != fa::OK)
        return st;
    return fa::append_launch(*cache, *k, *v, q && q->H > 0 ? q : nullptr, q_out, positions, spec, new_lens, T,
                             reinterpret_cast<cudaStream_t>(stream));
}

// Sizes of a paged decode: 0 for what fa_decode_paged refuses.
static bool paged_sizes_ok(int B, int Hq, int Hkv, int Tq, int max_pages, int page_size, int d)
{
    if (B < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || Tq < 1 || Tq > 16 || max_pages < 0 || !page_size_ok(page_size))
        return false;
    if (!width_ok(d) || (long long)max_pages * page_size > kMaxSlots)
        return false;
    // row indexes of q, and units of (sequence, KV head, 64 rows of a head group), in 31 bits
    return (long long)B * Hq <= INT_MAX / Tq;
}

size_t fa_decode_paged_workspace_bytes(int B, int Hq, int Hkv, int Tq, int max_pages, int page_size, int d,
                                       int accumulate)
{
    if (!paged_sizes_ok(B, Hq, Hkv, Tq, max_pages, page_size, d) || accumulate < 0 || accumulate > 1)
        return 0;
    const size_t n = fa::paged_workspace_bytes(B, Hq, Hkv, Tq, max_pages * page_size, d, accumulate);
    return n > 256 ? n : 256;
}

int fa_decode_paged(const fa_kv_cache *cache, const void *q, void *o, float *lse, int Hq, int Tq, int causal,
                    float scale, int accumulate, void *workspace, size_t workspace_bytes, fa_stream_t stream)
{
    int st = cache_check(cache);
    if (st != FA_OK)
        return st;
    if (causal < 0 || causal > 1 || accumulate < 0 || accumulate > 1 || !std::isfinite(scale) || !(scale > 0.0f))
        return FA_ERR_INVALID_ARG;
    if (Tq > 16)
        return FA_ERR_UNSUPPORTED;
    const int B = cache->B, d = cache->d;
    if (!paged_sizes_ok(B, Hq, cache->Hkv, Tq, cache->max_pages, cache->page_size, d))
        return FA_ERR_INVALID_ARG;
    if (accumulate && !cache->weight && slots_bytes(cache) > 0)
        return FA_ERR_INVALID_ARG;
    if (B == 0)
        return FA_OK;
    const size_t rows = (size_t)B * Hq * Tq, nq = rows * d * 2, nl = rows * 4;
    if (!q || !o || !lse || !fa::aligned16(q) || !fa::aligned16(o) || !fa::aligned16(lse))
        return FA_ERR_INVALID_ARG;
    const size_t need = fa::paged_workspace_bytes(B, Hq, cache->Hkv, Tq, cache->max_pages * cache->page_size, d, accumulate);
    if (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
        return FA_ERR_INVALID_ARG;
    if (!cache_disjoint(cache) && accumulate)
        return FA_ERR_INVALID_ARG;
    void *outs[3] = {o, lse, workspace};
    const size_t out_n[3] = {nq, nl, need};
    for (int i = 0; i < 3; ++i) {
        if (fa::overlaps(outs[i], out_n[i], q, nq) || touches_cache(cache, outs[i], out_n[i], true))
            return FA_ERR_INVALID_ARG;
        for (int j = i + 1; j < 3; ++j)
            if (fa::overlaps(outs[i], out_n[i], outs[j], out_n[j]))
                return FA_ERR_INVALID_ARG;
    }
    if (accumulate && fa::overlaps(cache->weight, slots_bytes(cache), q, nq))
        return FA_ERR_INVALID_ARG;
    if ((st = fa::check_device()) != fa::OK)
        return st;
    return fa::paged_launch(*cache, q, o, lse, Hq, Tq, causal, scale, accumulate, workspace,
                            reinterpret_cast<cudaStream_t>(stream));
}

int fa_cache_evict(const fa_kv_cache *cache, int budget, int n_first, int n_recent, float *weight_out, int *order_out,
                   int *lens_out, int *kept, fa_stream_t stream)
{
    int st = cache_check(cache);
    if (st != FA_OK)
        return st;
    if (budget < 1 || budget > kMaxSlots || n_first < 0 || n_recent < 0 || (long long)n_first + n_recent > budget)
        return FA_ERR_INVALID_ARG;
    const int B = cache->B;
    if (B == 0)
        return FA_OK;
    const size_t ns = slots_bytes(cache);
    // without a slot the arrays have no element, and no address need be given
    if (ns > 0 && (!cache->weight || !weight_out || ((n_first > 0 || n_recent > 0) && !cache->order) ||
                   (order_out != nullptr) != (cache->order != nullptr)))
        return FA_ERR_INVALID_ARG;
    if (!lens_out || !kept)
        return FA_ERR_INVALID_ARG;
    if (!fa::aligned16(weight_out) || !fa::aligned16(order_out) || !fa::aligned16(kept) ||
        (reinterpret_cast<uintptr_t>(lens_out) & 3u))
        return FA_ERR_INVALID_ARG;
    if (!cache_disjoint(cache))
        return FA_ERR_INVALID_ARG;
    const size_t nb = (size_t)B * 4, nk = (size_t)B * cache->Hkv * budget * 4;
    const void *outs[4] = {weight_out, order_out, lens_out, kept};
    const size_t out_n[4] = {ns, ns, nb, nk};
    const void *same[4] = {cache->weight, cache->order, cache->lens, nullptr};
    const void *state[3] = {cache->weight, cache->order, cache->lens};
    const size_t state_n[3] = {ns, ns, nb};
    for (int i = 0; i < 4; ++i) {
        if (!outs[i])
            continue;
        if (touches_cache(cache, outs[i], out_n[i], false))
            return FA_ERR_INVALID_ARG;
        for (int j = 0; j < 3; ++j)
            if (!(outs[i] == same[i] && i == j) && fa::overlaps(outs[i], out_n[i], state[j], state_n[j]))
                return FA_ERR_INVALID_ARG;
        for (int j = i + 1; j < 4; ++j)
            if (fa::overlaps(outs[i], out_n[i], outs[j], out_n[j]))
                return FA_ERR_INVALID_ARG;
    }
    if ((st = fa::check_device()) != fa::OK)
        return st;
    return fa::evict_launch(*cache, budget, n_first, n_recent, weight_out, order_out, lens_out, kept,
                            reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
