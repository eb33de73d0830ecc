// fa_rope.cuh -- what the kernels that rotate share (fa_cache_sm103.cu, fa_norm_sm103.cu): the angles,
// a thread's slice of a row, the loop over a token's heads, and the norm of a head's row.
#pragma once

#include "fa_common.cuh"
#include "fa_internal.h"

namespace fa {
namespace {

struct RopeTable {
    unsigned long long turns[128];
    unsigned char axis[128];
};

struct Row3 {   // one strided [B][H][T][d] tensor
    void *p;
    long long sb, sh, st;
};

__device__ __forceinline__ void phase_sincos(unsigned long long turns, int pos, float &sn, float &cs)
{
    const unsigned long long ph = turns * (unsigned long long)(long long)pos;
    const unsigned long long up = ph + (1ull << 61);      // to the nearest quarter turn
    const uint32_t quad = (uint32_t)(up >> 62);
    const int rest = (int)((long long)(ph - ((up >> 62) << 62)) >> 30);   // units of 2^-34 turns
    const float x = (float)rest * 3.6572952e-10f;         // 2 pi 2^-34: |x| <= pi / 4
    const float z = x * x;
    float s = fmaf(z, 2.7557319e-6f, -1.9841270e-4f);
    s = fmaf(z, s, 8.3333333e-3f);
    s = fmaf(z, s, -1.6666667e-1f);
    s = fmaf(x * z, s, x);
    float c = fmaf(z, -2.7557319e-7f, 2.4801587e-5f);
    c = fmaf(z, c, -1.3888889e-3f);
    c = fmaf(z, c, 4.1666667e-2f);
    c = fmaf(z, c, -0.5f);
    c = fmaf(z, c, 1.0f);
    const float a = (quad & 1) ? c : s, b = (quad & 1) ? s : c;
    sn = (quad & 2) ? -a : a;
    cs = ((quad + 1) & 2) ? -b : b;
}

// 8 consecutive elements as they lie in memory, and as fp32.
template <typename E>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
    uint4 w;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { w = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void get(float (&x)[8]) const
    {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(u[i] << 16);
            x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
        }
    }
};
template <>
struct Raw8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p)
    {
        a = reinterpret_cast<const float4 *>(p)[0];
        b = reinterpret_cast<const float4 *>(p)[1];
    }
    __device__ __forceinline__ void get(float (&x)[8]) const
    {
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
};
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&x)[8])
{
    *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                               pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}
__device__ __forceinline__ void store8(float *p, const float (&x)[8])
{
    reinterpret_cast<float4 *>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

// The 16 features of one thread: two runs of 8 at e0 and e1.  Thread v < rot / 16 has pairs
// 8 v .. 8 v + 7; the others 16 features that pass through.
struct Slice {
    int e0, e1, pair;   // pair < 0: pass through
};
__device__ __forceinline__ Slice slice_of(int v, int rot, int interleaved)
{
    Slice s;
    if (v < rot / 16) {
        s.pair = 8 * v;
        s.e0 = interleaved ? 16 * v : 8 * v;
        s.e1 = interleaved ? 16 * v + 8 : rot / 2 + 8 * v;
    } else {
        s.pair = -1;
        s.e0 = 16 * v;
        s.e1 = 16 * v + 8;
    }
    return s;
}

// Turns the pairs held in (a, b): pair j is (a[j], b[j]), or, interleaved, two neighbours.  Two
// pairs an instruction.
template <bool INTER>
__device__ __forceinline__ void turn(float (&a)[8], float (&b)[8], const float (&sn)[8], const float (&cs)[8])
{
    auto two = [&](float &x0, float &x1, float &y0, float &y1, int j) {
        float u0, u1, w0, w1;
        fmul2(u0, u1, x0, x1, cs[j], cs[j + 1]);
        fmul2(w0, w1, y0, y1, cs[j], cs[j + 1]);
        ffma2(w0, w1, x0, x1, sn[j], sn[j + 1], w0, w1);
        ffma2(x0, x1, y0, y1, -sn[j], -sn[j + 1], u0, u1);
        y0 = w0;
        y1 = w1;
    };
    if constexpr (!INTER) {
#pragma unroll
        for (int j = 0; j < 8; j += 2)
            two(a[j], a[j + 1], b[j], b[j + 1], j);
    } else {
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
            two(a[2 * j], a[2 * j + 2], a[2 * j + 1], a[2 * j + 3], j);
            two(b[2 * j], b[2 * j + 2], b[2 * j + 1], b[2 * j + 3], 4 + j);
        }
    }
}

// Runs over `n` heads of one token: x points at the first one's row, sx elements apart.  The loads
// of AHEAD heads are under way at once; put(head, values at e0, values at e1) takes them.  q and k of B8 H32 T4096
// d128 with 4, 6 and 8 heads ahead: 162.4, 160.9 and 160.1 us; prompts of 4193 tokens in e4m3 21.1, 20.5 and 20.2;
// 512 tokens 5.5, 5.8 and 6.3.  fp32 rows are twice as long.
template <typename E, typename Put>
__device__ __forceinline__ void each_head(const E *x, long long sx, int n, const Slice &sl, Put put)
{
    constexpr int AHEAD = sizeof(E) == 2 ? 6 : 3;
    x += sl.e0;
    const int gap = sl.e1 - sl.e0;
    for (int i = 0; i < n; i += AHEAD, x += AHEAD * sx) {
        Raw8<E> p[AHEAD], q[AHEAD];
#pragma unroll
        for (int u = 0; u < AHEAD; ++u)
            if (i + u < n) {
                p[u].load(x + u * sx);
                q[u].load(x + u * sx + gap);
            }
#pragma unroll
        for (int u = 0; u < AHEAD; ++u)
            if (i + u < n) {
                float f[8], g[8];
                p[u].get(f);
                q[u].get(g);
                put(i + u, f, g);
            }
    }
}

// ------------------------------------------------------------------ norms by head
// y = w x r with r = (mean x^2 + eps)^(-1/2) over the d features of a row, in fp32.
struct NormArgs {
    const void *w[2];   // weights of the first and second tensor, [d]; null: ones
    int wf32;
    float eps;
};

// Weights of features e .. e + 7.
__device__ __forceinline__ void norm_weights(const NormArgs &a, int which, int e, float (&w)[8])
{
    if (!a.w[which]) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            w[j] = 1.f;
    } else if (a.wf32) {
        Raw8<float> r;
        r.load(static_cast<const float *>(a.w[which]) + e);
        r.get(w);
    } else {
        Raw8<__nv_bfloat16> r;
        r.load(static_cast<const __nv_bfloat16 *>(a.w[which]) + e);
        r.get(w);
    }
}

// Sum of x over the TPR neighbouring lanes that have a row; the lanes of one row are in step, those of
// other rows of the warp may have left.
template <int TPR>
__device__ __forceinline__ float row_sum(float x)
{
    const uint32_t mask = (TPR == 32 ? 0xffffffffu : (1u << (TPR & 31)) - 1u) << (lane_id() & ~(TPR - 1u));
#pragma unroll
    for (int off = 1; off < TPR; off <<= 1)
        x += __shfl_xor_sync(mask, x, off);
    return x;
}

__device__ __forceinline__ float sum_squares(const float (&f)[8], const float (&g)[8])
{
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        ffma2(s0, s1, f[j], f[j + 1], f[j], f[j + 1], s0, s1);
        ffma2(s0, s1, g[j], g[j + 1], g[j], g[j + 1], s0, s1);
    }
    return s0 + s1;
}

// The weights of both tensors in shared memory, [2][D]; the threads of the block's first row or two put them there.
template <int D>
__device__ __forceinline__ void put_norm_weights(const NormArgs &a, const Slice &sl, float (*weight)[D])
{
    constexpr int TPR = D / 16;
    if (threadIdx.x < 2 * TPR) {
        const int w = threadIdx.x / TPR;
        float t[8];
        norm_weights(a, w, sl.e0, t);
        store8(weight[w] + sl.e0, t);
        norm_weights(a, w, sl.e1, t);
        store8(weight[w] + sl.e1, t);
    }
}

// each_head with rows normed by `weight` (shared memory) on the way.  Loads run AHEAD heads ahead: a head's values go
// to fp32 registers, its buffer is filled again, and only then they are used.  between() runs behind the first
// loads.
template <typename E, int D, int AHEAD, typename Between, typename Put>
__device__ __forceinline__ void each_head_normed(const E *x, long long sx, int n, const Slice &sl, const float *weight, float eps,
                                                 Between between, Put put)
{
    x += sl.e0;
    const int gap = sl.e1 - sl.e0;
    Raw8<E> p[AHEAD], q[AHEAD];
    auto fill = [&](int u) {
        p[u].load(x);
        q[u].load(x + gap);
        x += sx;
    };
#pragma unroll
    for (int u = 0; u < AHEAD; ++u)
        if (u < n)
            fill(u);
    between();
    for (int i = 0; i < n; i += AHEAD) {
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            if (i + u >= n)
                break;
            float f[8], g[8];
            p[u].get(f);
            q[u].get(g);
            if (i + u + AHEAD < n)
                fill(u);
            const float r = __frsqrt_rn(fmaf(row_sum<D / 16>(sum_squares(f, g)), 1.f / D, eps));
            auto scale = [&](float(&z)[8], int e) {
                Raw8<float> rw;
                float ww[8];
                rw.load(weight + e);
                rw.get(ww);
#pragma unroll
                for (int j = 0; j < 8; j += 2) {
                    fmul2(z[j], z[j + 1], z[j], z[j + 1], r, r);
                    fmul2(z[j], z[j + 1], z[j], z[j + 1], ww[j], ww[j + 1]);
                }
            };
            scale(f, sl.e0);
            scale(g, sl.e1);
            put(i + u, f, g);
        }
    }
}

// ------------------------------------------------------------------ host
constexpr int kRopeThreads = 256;

inline RopeTable table_of(const fa_rope_spec &s)
{
    RopeTable t;
    for (int i = 0; i < 128; ++i) {
        t.turns[i] = s.turns[i];
        t.axis[i] = s.axis[i];
    }
    return t;
}

inline Row3 row3(const fa_heads &x) { return Row3{x.data, x.stride_b, x.stride_h, x.stride_t}; }

// Heads one thread runs over: as few as let all CTAs be resident (two an SM), 32 at most.  With 8, 16,
// 32 and 48 heads the q and k of B8 H32 T4096 d128 take 175, 163, 162 and 163 us, and 4193 new tokens of
// 32 + 16 heads in e4m3 24.6, 24.1, 21.1 and 26.7, with 24 18.1: what counts is the groups, not the average (5 heads of
// B2 T3817 d128, normed: groups of 4 and 1 10.3 us, of 5 7.5).
inline int heads_per_cta(long long tokens, int H, int d)
{
    const long long tiles = (tokens * (d / 16) + kRopeThreads - 1) / kRopeThreads, slots = 2 * device_sm_count();
    long long n = (tiles * H + slots - 1) / slots;
    n = n < 1 ? 1 : n;
    while (n < 32 && n < H && tiles * ((H + n - 1) / n) > slots)   // groups of n heads, the last with fewer
        ++n;
    return (int)(n > 32 ? 32 : n);
}

inline NormArgs norm_args(const fa_head_norm &n)
{
    return NormArgs{{n.q_weight, n.k_weight}, n.dtype == FA_F32, n.eps};
}

}  // namespace
}  // namespace fa
