// fa_paged_sm103.cu -- attention of a few new rows over the paged key/value cache, split over
// the cache's length and joined (sm_103a).
//
// Formulas, per sequence, KV head and query row r of its head group: s_j = c q_r . k_j over the
// row's slots j, m = max s, p_j = e^{s_j - m} / l with l = sum e^{s_j - m}, o = sum p_j v_j,
// lse = m + ln l; with accumulate, weight_j += sum_r p_j.  The slots are split into chunks, each
// chunk leaves (m, l, sum e^{s - m} v) per row, and a second kernel joins them.
#include <climits>

#include "fa_common.cuh"
#include "fa_internal.h"

namespace fa {

__device__ int g_paged_status;   // device status word of the kernels in this file

namespace {

constexpr int kStatusBadIndex = 5;
constexpr int kChunk = 256;      // slots a CTA

struct PagedArgs {
    const __nv_bfloat16 *q;
    __nv_bfloat16 *o;
    float *lse, *weight;
    const void *k, *v;
    const float *ks, *vs;
    const int *block_table, *lens;
    float *part;     // [unit][chunk][row][D + 2]
    float *scores;   // [unit][row][cap], log2 units
    int Hq, Hkv, G, Tq, causal, num_pages, max_pages, ps_shift, cap, chunks;
    float scale_log2;
};

template <bool FP8>
__device__ __forceinline__ float element(const void *p, long long i)
{
    if constexpr (FP8)
        return __half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<const uint8_t *>(p)[i], __NV_E4M3)));
    else
        return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
}

__device__ __forceinline__ int length_of(const PagedArgs &a, int b)
{
    const int len = a.lens[b];
    if (len < 0 || len > a.cap) {
        atomicCAS(&g_paged_status, 0, kStatusBadIndex);
        return 0;
    }
    return len;
}

// Slots row r = g Tq + t of a head group sees.
__device__ __forceinline__ int seen_by(const PagedArgs &a, int len, int r)
{
    return a.causal ? len - a.Tq + r % a.Tq + 1 : len;
}

// Block-wide maximum and sum over kChunk threads.
template <bool MAX>
__device__ __forceinline__ float block_reduce(float x, float *scratch)
{
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        const float y = __shfl_xor_sync(0xffffffffu, x, off);
        x = MAX ? fmaxf(x, y) : x + y;
    }
    __syncthreads();
    if (lane_id() == 0)
        scratch[warp_id()] = x;
    __syncthreads();
    x = scratch[0];
    for (int i = 1; i < kChunk / 32; ++i)
        x = MAX ? fmaxf(x, scratch[i]) : x + scratch[i];
    return x;
}

template <int D, bool FP8>
__global__ void __launch_bounds__(kChunk) paged_kernel(const __grid_constant__ PagedArgs a)
{
    __shared__ float q[D], p[kChunk], scratch[8];
    __shared__ long long rows[kChunk];
    const long long unit = blockIdx.x / a.chunks;
    const int chunk = (int)(blockIdx.x - unit * a.chunks), tid = threadIdx.x;
    const int b = (int)(unit / a.Hkv), h = (int)(unit - (long long)b * a.Hkv), M = a.G * a.Tq;
    const int len = length_of(a, b), slot = chunk * kChunk + tid;
    if (chunk * kChunk >= len)
        return;
    long long at = -1;
    if (slot < len) {
        const int page = a.block_table[(long long)b * a.max_pages + (slot >> a.ps_shift)];
        if (page >= 0 && page < a.num_pages)
            at = ((((long long)page * a.Hkv + h) << a.ps_shift) + (slot & ((1 << a.ps_shift) - 1))) * D;
        else
            atomicCAS(&g_paged_status, 0, kStatusBadIndex);
    }
    rows[tid] = at;
    const float ks = FP8 ? a.ks[h] : 1.f, vs = FP8 ? a.vs[h] : 1.f;
    for (int r = 0; r < M; ++r) {
        const __nv_bfloat16 *qg = a.q + (((long long)b * a.Hq + h * a.G) * a.Tq + r) * D;
        __syncthreads();
        for (int e = tid; e < D; e += kChunk)
            q[e] = __bfloat162float(qg[e]);
        __syncthreads();
        float s = -INFINITY;
        if (at >= 0 && slot < seen_by(a, len, r)) {
            float dot = 0.f;
            for (int e = 0; e < D; ++e)
                dot = fmaf(q[e], element<FP8>(a.k, at + e), dot);
            s = dot * (ks * a.scale_log2);
        }
        if (a.scores && slot < len)
            a.scores[((long long)unit * M + r) * a.cap + slot] = s;
        const float m = block_reduce<true>(s, scratch);
        const float w = s == -INFINITY ? 0.f : exp2f(s - m);
        p[tid] = w;
        const float l = block_reduce<false>(w, scratch);
        float *dst = a.part + ((unit * a.chunks + chunk) * M + r) * (D + 2);
        if (tid < D) {
            float acc = 0.f;
            for (int j = 0; j < kChunk; ++j)
                if (rows[j] >= 0)
                    acc = fmaf(p[j], element<FP8>(a.v, rows[j] + tid), acc);
            dst[tid] = acc * vs;
        }
        if (tid == 0) {
            dst[D] = m;
            dst[D + 1] = l;
        }
    }
}

// One CTA per (unit, row): o and lse from the chunks' states.
template <int D>
__global__ void __launch_bounds__(D) paged_join_kernel(const __grid_constant__ PagedArgs a)
{
    const int M = a.G * a.Tq;
    const long long unit = blockIdx.x / M;
    const int r = (int)(blockIdx.x - unit * M), b = (int)(unit / a.Hkv), h = (int)(unit - (long long)b * a.Hkv);
    const int n = (length_of(a, b) + kChunk - 1) / kChunk;
    const float *src = a.part + (unit * a.chunks * M + r) * (D + 2);
    const long long stride = (long long)M * (D + 2);
    float m = -INFINITY, l = 0.f, acc = 0.f;
    for (int i = 0; i < n; ++i)
        m = fmaxf(m, src[i * stride + D]);
    if (m != -INFINITY)
        for (int i = 0; i < n; ++i) {
            const float mi = src[i * stride + D];
            const float w = mi == -INFINITY ? 0.f : exp2f(mi - m);
            l = fmaf(w, src[i * stride + D + 1], l);
            acc = fmaf(w, src[i * stride + threadIdx.x], acc);
        }
    const long long row = ((long long)b * a.Hq + h * a.G) * a.Tq + r;
    a.o[row * D + threadIdx.x] = __float2bfloat16(l == 0.f ? 0.f : acc / l);
    if (threadIdx.x == 0)
        a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994530942f;
}

// weight_j += sum over the head group's rows of p_j, from the stored scores and lse.
__global__ void __launch_bounds__(256) paged_weight_kernel(const __grid_constant__ PagedArgs a)
{
    const int M = a.G * a.Tq;
    const long long unit = blockIdx.x;
    const int b = (int)(unit / a.Hkv), h = (int)(unit - (long long)b * a.Hkv), len = length_of(a, b);
    for (int j = blockIdx.y * 256 + threadIdx.x; j < len; j += gridDim.y * 256) {
        float sum = 0.f;
        for (int r = 0; r < M; ++r) {
            const float lse = a.lse[((long long)b * a.Hq + h * a.G) * a.Tq + r];
            const float s = a.scores[(unit * M + r) * a.cap + j];
            if (s != -INFINITY)
                sum += exp2f(s - lse * 1.4426950408889634f);
        }
        a.weight[unit * a.cap + j] += sum;
    }
}

template <int D, bool FP8>
int paged_run(const PagedArgs &a, int units, cudaStream_t s)
{
    if (a.chunks > 0)
        paged_kernel<D, FP8><<<(unsigned)((long long)units * a.chunks), kChunk, 0, s>>>(a);
    paged_join_kernel<D><<<units * a.G * a.Tq, D, 0, s>>>(a);
    if (a.scores && a.chunks > 0)
        paged_weight_kernel<<<dim3(units, a.chunks < 64 ? a.chunks : 64), 256, 0, s>>>(a);
    return cudaGetLastError() == cudaSuccess ? OK : ERR_CUDA;
}

size_t round256(size_t x) { return (x + 255) & ~(size_t)255; }

size_t part_bytes(int B, int Hq, int Tq, int max_len, int d)
{
    return round256((size_t)B * Hq * Tq * ((max_len + kChunk - 1) / kChunk) * (d + 2) * sizeof(float));
}

}  // namespace

size_t paged_workspace_bytes(int B, int Hq, int Hkv, int Tq, int max_len, int d, int accumulate)
{
    (void)Hkv;
    return part_bytes(B, Hq, Tq, max_len, d) + (accumulate ? round256((size_t)B * Hq * Tq * max_len * sizeof(float)) : 0);
}

int paged_launch(const fa_kv_cache &c, const void *q, void *o, float *lse, int Hq, int Tq, int causal, float scale,
                 int accumulate, void *workspace, cudaStream_t s)
{
    PagedArgs a;
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.o = static_cast<__nv_bfloat16 *>(o);
    a.lse = lse;
    a.weight = c.weight;
    a.k = c.k;
    a.v = c.v;
    a.ks = c.k_scale;
    a.vs = c.v_scale;
    a.block_table = c.block_table;
    a.lens = c.lens;
    a.Hq = Hq;
    a.Hkv = c.Hkv;
    a.G = Hq / c.Hkv;
    a.Tq = Tq;
    a.causal = causal;
    a.num_pages = c.num_pages;
    a.max_pages = c.max_pages;
    a.ps_shift = 0;
    while ((1 << a.ps_shift) < c.page_size)
        ++a.ps_shift;
    a.cap = c.max_pages * c.page_size;
    a.chunks = (a.cap + kChunk - 1) / kChunk;
    a.part = static_cast<float *>(workspace);
    a.scores = accumulate ? reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) +
                                                      part_bytes(c.B, Hq, Tq, a.cap, c.d))
                          : nullptr;
    a.scale_log2 = scale * 1.4426950408889634f;
    const int units = c.B * c.Hkv;
    if ((long long)units * (a.chunks > 0 ? a.chunks : 1) > INT_MAX)
        return ERR_UNSUPPORTED;
    const bool f8 = c.dtype == FA_E4M3;
    switch (c.d) {
    case 64:
        return f8 ? paged_run<64, true>(a, units, s) : paged_run<64, false>(a, units, s);
    case 128:
        return f8 ? paged_run<128, true>(a, units, s) : paged_run<128, false>(a, units, s);
    default:
        return f8 ? paged_run<256, true>(a, units, s) : paged_run<256, false>(a, units, s);
    }
}

int paged_status_fetch_clear(cudaStream_t s, int *host_word)
{
    int zero = 0;
    if (cudaMemcpyFromSymbolAsync(host_word, g_paged_status, sizeof(int), 0, cudaMemcpyDeviceToHost, s) != cudaSuccess ||
        cudaMemcpyToSymbolAsync(g_paged_status, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, s) != cudaSuccess ||
        cudaStreamSynchronize(s) != cudaSuccess)
        return ERR_CUDA;
    return OK;
}

}  // namespace fa
