// fa_norm_sm103.cu -- norms of query and key heads with the rotation in the same pass, and their
// gradients (sm_103a).
//
// Formulas, per row of d features: r = (mean x^2 + eps)^(-1/2), u = x r, y = R(w u), where R turns the
// pairs by the token's positions (fa_cache_sm103.cu).  Backward, with g = R^T dy:
//     dw = sum over all rows of g u,    dx = r (w g - u mean(w g u)).
// r is found again from x: it is one sum more, and nothing has to be kept between the passes.
//
// What bounds them is memory: forward reads and writes each element once, backward reads x and dy and
// writes dx.  A thread has 16 features of one token (8 pairs) and runs over heads with the token's
// sines and cosines in registers and the weights in shared memory; the D / 16 threads of a row put their sums
// together by shuffles, while the loads of the next heads are under way.  Measured, q and k of B8 H32 T4096 d128 in
// bf16: 162 us forward (6.6 TB/s), 255 backward (6.3).  Backward, a head group has as many CTAs as any other, and where
// their heads differ the largest groups end last: 32 + 8 heads 209 us (4.8 TB/s; B4 in fp32 195, 5.2), 40 + 8 305 (4.0),
// 64 + 8 334 (5.4).  dw: each thread adds up its features over all its rows, each CTA its threads, and a second kernel
// the CTAs, in a fixed order: the same bits on every run.
#include <climits>

#include "fa_common.cuh"
#include "fa_internal.h"
#include "fa_pdl.cuh"
#include "fa_rope.cuh"

namespace fa {
namespace {

struct NormRopeArgs {
    Row3 x[2], y[2];
    NormArgs norm;
    int H0, H;            // heads of the first tensor, of both
    const int *pos;       // [axes][n]
    long long n;          // B * T
    int T, rot, heads_per_cta, groups;
};

template <typename E, int D, bool INTER>
__global__ void __launch_bounds__(kRopeThreads, 2) norm_rope_kernel(const __grid_constant__ RopeTable tab,
                                                                 const __grid_constant__ NormRopeArgs a)
{
    constexpr int TPR = D / 16;                          // threads a row
    // Heads ahead: q and k of B8 H32 T4096 d128 with 2, 3, 4 and 6 182, 169, 165 and 162 us (B4 in fp32 with 1 and 2 188
    // and 167); rounds of four that did not overlap, with the weights in registers, 174
    constexpr int AHEAD = sizeof(E) == 2 ? 6 : 2;
    __shared__ __align__(16) float weight[2][D];
    pdl_launch();
    pdl_wait();
    const int v = threadIdx.x % TPR;
    // head groups next to one another: CTAs that run together read whole token rows of a packed
    // projection
    const int tile = (int)(blockIdx.x / a.groups), group = (int)blockIdx.x - tile * a.groups;
    const long long tok = (long long)tile * (kRopeThreads / TPR) + threadIdx.x / TPR;
    const Slice sl = slice_of(v, a.rot, INTER);
    put_norm_weights<D>(a.norm, sl, weight);
    __syncthreads();
    if (tok >= a.n)
        return;
    const int b = (int)tok / a.T, t = (int)tok - b * a.T;
    float sn[8], cs[8];
    bool known = false;   // the sines and cosines
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
        each_head_normed<E, D, AHEAD>(
            x, xi.sh, last - first, sl, weight[w], a.norm.eps,
            [&]() {
                if (known || sl.pair < 0)
                    return;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int p = a.pos[(long long)tab.axis[sl.pair + j] * a.n + tok];
                    phase_sincos(tab.turns[sl.pair + j], p, sn[j], cs[j]);
                }
            },
            [&](int, float(&f)[8], float(&g)[8]) {
                if (sl.pair >= 0)
                    turn<INTER>(f, g, sn, cs);
                store8(y, f);
                store8(y + gap, g);
                y += yi.sh;
            });
        known = true;
    }
}

// ------------------------------------------------------------------ backward
struct NormBwdArgs {
    Row3 x[2], dy[2], dx[2];
    NormArgs norm;
    int H[2], G0;         // heads of either tensor; head groups of the first
    const int *pos;       // [axes][n]
    long long n;          // B * T
    int T, rot, heads_per_cta, groups, tiles;
    float *part;          // [CTA][d], or null: no gradients of the weights
    float *dw[2];         // or null
    int ctas;
};

constexpr int kNormCtas = 304;   // two an SM; the sums' order depends on it, not on the device
// Threads of a CTA: 168 registers each are enough for two heads ahead without a spill.  q and k of B8 H32
// T4096 d128, us by threads, CTAs an SM and heads ahead: 192 2 2 256, 128 3 2 257, 256 1 4 267, 256 2 1 272, 192 2 3
// (60 bytes of spills) 301, 256 2 2 (200) 381.
constexpr int kNormThreads = 192;

// A CTA has one head group, of one tensor, and every ctas / groups-th tile of tokens.  A thread's loads run one
// or two heads ahead: a head's values go to fp32 registers, its buffer is filled again, and only then they are
// used.  The weights stay in shared memory.
template <typename E, int D, bool INTER>
__global__ void __launch_bounds__(kNormThreads, 2) norm_bwd_kernel(const __grid_constant__ RopeTable tab,
                                                                const __grid_constant__ NormBwdArgs a)
{
    constexpr int TPR = D / 16, TOK = kNormThreads / TPR;
    constexpr int AHEAD = sizeof(E) == 2 ? 2 : 1;
    __shared__ float sums[TOK * D];
    __shared__ __align__(16) float weights[2][D];
    pdl_wait();
    const int v = threadIdx.x % TPR, row = threadIdx.x / TPR;
    const int group = (int)blockIdx.x % a.groups, w = group >= a.G0;
    const int h0 = (group - (w ? a.G0 : 0)) * a.heads_per_cta, nh = min(a.heads_per_cta, a.H[w] - h0);
    const Slice sl = slice_of(v, a.rot, INTER);
    const int gap = sl.e1 - sl.e0;
    put_norm_weights<D>(a.norm, sl, weights);
    const float *weight = weights[w];
    __syncthreads();
    float af[8], ag[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
        af[j] = ag[j] = 0.f;
    const Row3 &xi = a.x[w], &gi = a.dy[w], &oi = a.dx[w];
    for (int tile = (int)blockIdx.x / a.groups; tile < a.tiles; tile += a.ctas / a.groups) {
        const long long tok = (long long)tile * TOK + row;
        if (tok >= a.n)
            break;
        const int b = (int)tok / a.T, t = (int)tok - b * a.T;
        const E *x = static_cast<const E *>(xi.p) + b * xi.sb + h0 * xi.sh + t * xi.st + sl.e0;
        const E *dy = static_cast<const E *>(gi.p) + b * gi.sb + h0 * gi.sh + t * gi.st + sl.e0;
        E *dx = static_cast<E *>(oi.p) + b * oi.sb + h0 * oi.sh + t * oi.st + sl.e0;
        Raw8<E> px[AHEAD][2], pg[AHEAD][2];
        auto fill = [&](int u) {
            px[u][0].load(x);
            px[u][1].load(x + gap);
            pg[u][0].load(dy);
            pg[u][1].load(dy + gap);
            x += xi.sh;
            dy += gi.sh;
        };
#pragma unroll
        for (int u = 0; u < AHEAD; ++u)
            if (u < nh)
                fill(u);
        float sn[8], cs[8];
        if (sl.pair >= 0) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int p = a.pos[(long long)tab.axis[sl.pair + j] * a.n + tok];
                phase_sincos(tab.turns[sl.pair + j], p, sn[j], cs[j]);
                sn[j] = -sn[j];   // the transpose turns the other way
            }
        }
        for (int i = 0; i < nh; i += AHEAD) {
#pragma unroll
            for (int u = 0; u < AHEAD; ++u) {
                if (i + u >= nh)
                    break;
                float x0[8], x1[8], f[8], g[8];   // x, and R^T dy
                px[u][0].get(x0);
                px[u][1].get(x1);
                pg[u][0].get(f);
                pg[u][1].get(g);
                if (i + u + AHEAD < nh)
                    fill(u);
                if (sl.pair >= 0)
                    turn<INTER>(f, g, sn, cs);
                // sums of x^2 and of w g x
                const float s = row_sum<TPR>(sum_squares(x0, x1));
                float z0 = 0.f, z1 = 0.f;
                auto dots = [&](const float(&gy)[8], const float(&xx)[8], int e) {
                    Raw8<float> r;
                    float ww[8];
                    r.load(weight + e);
                    r.get(ww);
#pragma unroll
                    for (int j = 0; j < 8; j += 2) {
                        float t0, t1;
                        fmul2(t0, t1, gy[j], gy[j + 1], ww[j], ww[j + 1]);
                        ffma2(z0, z1, t0, t1, xx[j], xx[j + 1], z0, z1);
                    }
                };
                dots(f, x0, sl.e0);
                dots(g, x1, sl.e1);
                const float z = row_sum<TPR>(z0 + z1);
                const float r = __frsqrt_rn(fmaf(s, 1.f / D, a.norm.eps));
                const float m = -z * (1.f / D) * r * r;   // dx = r (w g - x (r^2 mean(w g x)))
                auto half = [&](float(&gy)[8], const float(&xx)[8], int e, float(&acc)[8]) {
                    Raw8<float> rw;
                    float ww[8];
                    rw.load(weight + e);
                    rw.get(ww);
#pragma unroll
                    for (int j = 0; j < 8; j += 2) {
                        float t0, t1;
                        fmul2(t0, t1, xx[j], xx[j + 1], r, r);
                        ffma2(acc[j], acc[j + 1], gy[j], gy[j + 1], t0, t1, acc[j], acc[j + 1]);
                        fmul2(t0, t1, gy[j], gy[j + 1], ww[j], ww[j + 1]);
                        ffma2(t0, t1, xx[j], xx[j + 1], m, m, t0, t1);
                        fmul2(gy[j], gy[j + 1], t0, t1, r, r);
                    }
                };
                half(f, x0, sl.e0, af);
                half(g, x1, sl.e1, ag);
                store8(dx, f);
                store8(dx + gap, g);
                dx += oi.sh;
            }
        }
    }
    pdl_launch();
    if (!a.part)
        return;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        sums[row * D + sl.e0 + j] = af[j];
        sums[row * D + sl.e1 + j] = ag[j];
    }
    __syncthreads();
    for (int f = threadIdx.x; f < D; f += kNormThreads) {
        float x = 0.f;
#pragma unroll 8
        for (int i = 0; i < TOK; ++i)
            x += sums[i * D + f];
        a.part[(long long)blockIdx.x * D + f] = x;
    }
}

// dw[tensor][32 features of a block]: the CTAs' sums, kRuns runs of CTAs side by side, so that a warp's loads are two
// or three rounds (5.1 us with eight runs and four loads at once, at 228 CTAs).
constexpr int kRuns = 16;
__global__ void __launch_bounds__(32 * kRuns) norm_dweight_kernel(const __grid_constant__ NormBwdArgs a, int d)
{
    __shared__ float red[kRuns][32];
    pdl_launch();
    pdl_wait();
    const int w = (int)blockIdx.y, f = (int)blockIdx.x * 32 + (threadIdx.x & 31), run = threadIdx.x >> 5;
    if (!a.dw[w])
        return;
    const int from = w ? a.G0 : 0, count = w ? a.groups - a.G0 : a.G0;   // its head groups
    const int total = count * (a.ctas / a.groups);
    float x = 0.f;
#pragma unroll 8
    for (int i = run; i < total; i += kRuns)
        x += __ldcg(a.part + (long long)(i / count * a.groups + from + i % count) * d + f);
    red[run][threadIdx.x & 31] = x;
    __syncthreads();
    if (run == 0) {
#pragma unroll
        for (int i = 1; i < kRuns; ++i)
            x += red[i][threadIdx.x];
        a.dw[w][f] = x;
    }
}

template <typename E, int D>
int norm_run(const RopeTable &t, const NormRopeArgs &a, int interleaved, cudaStream_t s)
{
    constexpr int TOK = kRopeThreads / (D / 16);
    const dim3 grid((unsigned)((a.n + TOK - 1) / TOK * a.groups));
    return launch_overlapped(interleaved ? norm_rope_kernel<E, D, true> : norm_rope_kernel<E, D, false>, grid, kRopeThreads, 0, 0,
                             true, s, t, a);
}

template <typename E, int D>
int norm_bwd_run(const RopeTable &t, NormBwdArgs &a, int interleaved, cudaStream_t s)
{
    constexpr int TOK = kNormThreads / (D / 16);
    a.tiles = (int)((a.n + TOK - 1) / TOK);
    const int runs = kNormCtas / a.groups;   // CTAs of a head group
    a.ctas = a.groups * (a.tiles < runs ? a.tiles : runs);
    if (a.ctas == 0)   // no row: the sums are 0
        return launch_overlapped(norm_dweight_kernel, dim3(D / 32, 2), 32 * kRuns, 0, 0, true, s, a, D);
    const int st = launch_overlapped(interleaved ? norm_bwd_kernel<E, D, true> : norm_bwd_kernel<E, D, false>, dim3((unsigned)a.ctas),
                                     kNormThreads, 0, 0, true, s, t, a);
    if (st != OK || !a.part)
        return st;
    return launch_overlapped(norm_dweight_kernel, dim3(D / 32, 2), 32 * kRuns, 0, 0, true, s, a, D);
}

template <typename E>
int norm_width(int d, const RopeTable &t, const NormRopeArgs &a, int interleaved, cudaStream_t s)
{
    return d == 64 ? norm_run<E, 64>(t, a, interleaved, s)
                   : d == 128 ? norm_run<E, 128>(t, a, interleaved, s) : norm_run<E, 256>(t, a, interleaved, s);
}

template <typename E>
int norm_bwd_width(int d, const RopeTable &t, NormBwdArgs &a, int interleaved, cudaStream_t s)
{
    return d == 64 ? norm_bwd_run<E, 64>(t, a, interleaved, s)
                   : d == 128 ? norm_bwd_run<E, 128>(t, a, interleaved, s) : norm_bwd_run<E, 256>(t, a, interleaved, s);
}

}  // namespace

int norm_rope_launch(const fa_heads *x, const fa_heads *y, int n, const fa_head_norm &norm, const int *positions,
                     const fa_rope_spec &spec, int B, int T, int dtype, cudaStream_t s)
{
    NormRopeArgs a{};
    a.H = 0;
    for (int i = 0; i < n; ++i) {
        a.x[i] = row3(x[i]);
        a.y[i] = row3(y[i]);
        a.H += x[i].H;
    }
    a.H0 = x[0].H;
    a.norm = norm_args(norm);
    a.pos = positions;
    a.n = (long long)B * T;
    a.T = T;
    a.rot = spec.rot;
    a.heads_per_cta = heads_per_cta(a.n, a.H, spec.d);
    a.groups = (a.H + a.heads_per_cta - 1) / a.heads_per_cta;
    if ((a.n / 16 + 1) * a.groups > INT_MAX)
        return ERR_UNSUPPORTED;
    const RopeTable t = table_of(spec);
    return dtype == FA_F32 ? norm_width<float>(spec.d, t, a, spec.interleaved, s)
                           : norm_width<__nv_bfloat16>(spec.d, t, a, spec.interleaved, s);
}

size_t norm_bwd_workspace_bytes(int d) { return (size_t)kNormCtas * d * sizeof(float); }

int norm_rope_bwd_launch(const fa_heads *x, const fa_heads *dy, const fa_heads *dx, int n, const fa_head_norm &norm,
                         const int *positions, const fa_rope_spec &spec, int B, int T, int dtype, float *dq_weight,
                         float *dk_weight, void *workspace, cudaStream_t s)
{
    NormBwdArgs a{};
    long long H = 0;
    for (int i = 0; i < n; ++i) {
        a.x[i] = row3(x[i]);
        a.dy[i] = row3(dy[i]);
        a.dx[i] = row3(dx[i]);
        a.H[i] = x[i].H;
        H += x[i].H;
    }
    a.norm = norm_args(norm);
    a.pos = positions;
    a.n = (long long)B * T;
    a.T = T;
    a.rot = spec.rot;
    // Heads of a group: as few as let every tile of every group have a CTA of its own, up to 32, and so many that every
    // group has a CTA.  B2 T1021 of 6 + 2 heads of 64, fp32: a head a group is 344 tiles, two of them for some CTAs
    const int tok = kNormThreads / (spec.d / 16), least = (int)((H + kNormCtas - 3) / (kNormCtas - 2));
    const long long tiles = (a.n + tok - 1) / tok;
    auto groups_of = [&](int w, int hpc) { return a.H[w] / hpc + (a.H[w] % hpc > 0); };
    a.heads_per_cta = least > 1 ? least : 1;
    while (a.heads_per_cta < 32 && (groups_of(0, a.heads_per_cta) + groups_of(1, a.heads_per_cta)) * tiles > kNormCtas)
        ++a.heads_per_cta;
    a.G0 = groups_of(0, a.heads_per_cta);
    a.groups = a.G0 + groups_of(1, a.heads_per_cta);
    a.groups = a.groups > 0 ? a.groups : 1;
    a.dw[0] = dq_weight;
    a.dw[1] = dk_weight;
    a.part = dq_weight || dk_weight ? static_cast<float *>(workspace) : nullptr;
    const RopeTable t = table_of(spec);
    return dtype == FA_F32 ? norm_bwd_width<float>(spec.d, t, a, spec.interleaved, s)
                           : norm_bwd_width<__nv_bfloat16>(spec.d, t, a, spec.interleaved, s);
}

}  // namespace fa
