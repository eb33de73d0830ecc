// fa_api.cu -- the C ABI of libfa.so (declared in include/fa.h): argument
// validation, TMA descriptor encoding, kernel dispatch and the device status
// word.  No compute happens here; every step of the path runs in the kernels
// of fa_fwd_sm103.cu, fa_fwd_f32.cu and fa_bwd_sm103.cu.
#include <atomic>
#include <climits>
#include <cmath>
#include <cstdlib>
#include <mutex>

#include "../../include/fa.h"
#include "fa_internal.h"

namespace fa {

// ------------------------------------------------------------ driver glue
namespace {

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                   const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn()
{
    static std::once_flag once;
    static EncodeTiledFn fn = nullptr;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

constexpr int kMaxDevices = 64;

}  // namespace

int encode_tmap_3d(CUtensorMap *map, const void *base, CUtensorMapDataType dtype, int elem_bytes, uint64_t inner,
                   uint64_t rows, uint64_t planes, uint32_t box_inner, uint32_t box_rows)
{
    return encode_tmap_3d_strided(map, base, dtype, elem_bytes, inner, rows, planes, inner * (uint64_t)elem_bytes,
                                  box_inner, box_rows);
}

namespace {

int encode_3d(CUtensorMap *map, const void *base, CUtensorMapDataType dtype, uint64_t inner, uint64_t rows,
              uint64_t planes, uint64_t row_stride, uint32_t box_inner, uint32_t box_rows, CUtensorMapSwizzle swz)
{
    EncodeTiledFn fn = encode_fn();
    if (!fn)
        return ERR_CUDA;
    const cuuint64_t dims[3] = {inner, rows, planes};
    const cuuint64_t strides[2] = {row_stride, rows * row_stride};
    const cuuint32_t box[3] = {box_inner, box_rows, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    const CUresult r = fn(map, dtype, 3, const_cast<void *>(base), dims, strides, box, estr,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, swz, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? OK : ERR_CUDA;
}

}  // namespace

int encode_tmap_3d_plain(CUtensorMap *map, const void *base, CUtensorMapDataType dtype, int elem_bytes,
                         uint64_t inner, uint64_t rows, uint64_t planes, uint32_t box_inner, uint32_t box_rows)
{
    return encode_3d(map, base, dtype, inner, rows, planes, inner * (uint64_t)elem_bytes, box_inner, box_rows,
                     CU_TENSOR_MAP_SWIZZLE_NONE);
}

int encode_tmap_3d_strided(CUtensorMap *map, const void *base, CUtensorMapDataType dtype, int elem_bytes,
                           uint64_t inner, uint64_t rows, uint64_t planes, uint64_t row_stride, uint32_t box_inner,
                           uint32_t box_rows)
{
    (void)elem_bytes;
    return encode_3d(map, base, dtype, inner, rows, planes, row_stride, box_inner, box_rows,
                     CU_TENSOR_MAP_SWIZZLE_128B);
}


int encode_tmap(CUtensorMap *map, const void *base, CUtensorMapDataType dtype, int rank, const uint64_t *dims,
                const uint64_t *strides, const uint32_t *box, CUtensorMapSwizzle swizzle)
{
    EncodeTiledFn fn = encode_fn();
    if (!fn || rank > 5)
        return ERR_CUDA;
    cuuint64_t gd[5], gs[5];
    cuuint32_t bx[5], es[5];
    for (int i = 0; i < rank; ++i) {
        gd[i] = dims[i];
        bx[i] = box[i];
        es[i] = 1;
        if (i + 1 < rank)
            gs[i] = strides[i];
    }
    return fn(map, dtype, (cuuint32_t)rank, const_cast<void *>(base), gd, gs, bx, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
              swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? OK
               : ERR_CUDA;
}

int device_sm_count()
{
    static int cache[kMaxDevices] = {0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return 1;
    if (dev >= 0 && dev < kMaxDevices && cache[dev] > 0)
        return cache[dev];
    int n = 1;
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    if (dev >= 0 && dev < kMaxDevices)
        cache[dev] = n;
    return n;
}

uint64_t wait_timeout_ns()
{
    static const uint64_t ns = [] {
        const char *e = std::getenv("FA_WAIT_TIMEOUT_MS");
        long ms = e ? std::strtol(e, nullptr, 10) : 0;
        if (ms <= 0)
            ms = 4000;
        return (uint64_t)ms * 1000000ull;
    }();
    return ns;
}

#if FA_TEST_WITHHOLD
namespace {
std::mutex g_withhold_mu;
int g_withhold = WITHHOLD_NONE;
}  // namespace

int test_withhold_take(int lo, int hi)
{
    std::lock_guard<std::mutex> lock(g_withhold_mu);
    const int w = g_withhold;
    if (w < lo || w > hi)
        return WITHHOLD_NONE;
    g_withhold = WITHHOLD_NONE;
    return w;
}
#endif

// ------------------------------------------------------------ fill kernel
// Rows with no key at all (Tk == 0): O = 0, lse = -inf.
__global__ void fill_empty_kernel(uint8_t *o, float *lse, size_t rows, int row_bytes)
{
    const size_t n16 = rows * (size_t)(row_bytes / 16);
    for (size_t i = blockIdx.x * (size_t)blockDim.x + threadIdx.x; i < n16; i += (size_t)gridDim.x * blockDim.x)
        reinterpret_cast<uint4 *>(o)[i] = make_uint4(0, 0, 0, 0);
    for (size_t i = blockIdx.x * (size_t)blockDim.x + threadIdx.x; i < rows; i += (size_t)gridDim.x * blockDim.x)
        lse[i] = -INFINITY;
}

int fill_empty_launch(void *o, float *lse, size_t rows, int d, int elem_bytes, cudaStream_t s)
{
    const int grid = device_sm_count() * 4;
    fill_empty_kernel<<<grid, 256, 0, s>>>(static_cast<uint8_t *>(o), lse, rows, d * elem_bytes);
    return cudaGetLastError() == cudaSuccess ? OK : ERR_CUDA;
}

// ------------------------------------------------------------ status words in use
namespace {
std::atomic<unsigned> g_status_in_use{0};   // a bit a StatusWords
#if FA_TEST_WITHHOLD
std::atomic<int> g_status_reads{0};         // of the cache kernels' words
#endif
bool status_is_in_use(StatusWords w)
{
    const bool in_use = g_status_in_use.load(std::memory_order_relaxed) >> w & 1u;
#if FA_TEST_WITHHOLD
    g_status_reads += in_use;
#endif
    return in_use;
}
}  // namespace

void status_in_use(StatusWords w)
{
    if (!(g_status_in_use.load(std::memory_order_relaxed) >> w & 1u))
        g_status_in_use.fetch_or(1u << w, std::memory_order_relaxed);
}

// ------------------------------------------------------------ validation
bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// A buffer of n elements: non-null and 16-byte aligned, or anything when n == 0.
bool present16(const void *p, size_t n) { return n == 0 || (p && aligned16(p)); }

bool overlaps(const void *a, size_t na, const void *b, size_t nb)
{
    if (!a || !b || na == 0 || nb == 0)
        return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
    return a0 < b0 + nb && b0 < a0 + na;
}

// sm_103 check of the current device (cached).
int check_device()
{
    static int cache[kMaxDevices] = {0};   // 0 unknown, 1 ok, 2 unsupported
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return ERR_CUDA;
    if (dev >= 0 && dev < kMaxDevices && cache[dev])
        return cache[dev] == 1 ? OK : ERR_UNSUPPORTED;
    int major = 0, minor = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
        return ERR_CUDA;
    const bool ok = (major == 10 && minor == 3);
    if (dev >= 0 && dev < kMaxDevices)
        cache[dev] = ok ? 1 : 2;
    return ok ? OK : ERR_UNSUPPORTED;
}

namespace {

// Shapes, flags and scale shared by every entry point.
int check_sizes(int B, int H, int Tq, int Tk, int d, int causal, float scale)
{
    if (B < 0 || H < 0 || Tq < 0 || Tk < 0)
        return ERR_INVALID_ARG;
    if (causal != 0 && causal != 1)
        return ERR_INVALID_ARG;
    if (!std::isfinite(scale) || !(scale > 0.0f))
        return ERR_INVALID_ARG;
    if (d != 64 && d != 128 && d != 256)
        return ERR_UNSUPPORTED;
    // every (b*H + h) * T + row index must fit in 32 bits
    const long long bh = (long long)B * H;
    if (bh * (long long)(Tq > Tk ? Tq : Tk) > INT_MAX)
        return ERR_INVALID_ARG;
    return OK;
}

int check_fwd(const void *q, const void *k, const void *v, const void *o, const float *lse, int B, int H,
              int Tq, int Tk, int d, int causal, float scale, int elem)
{
    int st = check_sizes(B, H, Tq, Tk, d, causal, scale);
    if (st != OK)
        return st;
    const size_t bh = (size_t)B * H;
    if (bh * Tq == 0)
        return OK;
    const size_t nq = bh * Tq * d * elem, nk = bh * Tk * d * elem, nl = bh * Tq * sizeof(float);
    if (!q || !o || !lse || (Tk > 0 && (!k || !v)))
        return ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse))
        return ERR_INVALID_ARG;
    if (overlaps(o, nq, q, nq) || overlaps(o, nq, k, nk) || overlaps(o, nq, v, nk) || overlaps(o, nq, lse, nl) ||
        overlaps(lse, nl, q, nq) || overlaps(lse, nl, k, nk) || overlaps(lse, nl, v, nk))
        return ERR_INVALID_ARG;
    return check_device();
}

size_t round256(size_t x) { return (x + 255) & ~(size_t)255; }

}  // namespace

size_t bwd_row_stride(int Tq) { return ((size_t)Tq + 127) / 128 * 128; }

size_t bwd_workspace_bytes(size_t BH, int Tq, int d)
{
    const size_t rows = BH * bwd_row_stride(Tq);
    return 2 * round256(rows * sizeof(float)) + round256(rows * d * sizeof(float)) +
           round256((size_t)BH * 2 * sizeof(float) + rows / 128 * sizeof(int));
}

BwdWorkspace bwd_workspace_carve(void *ws, int BH, int Tq, int d)
{
    const size_t rows = (size_t)BH * bwd_row_stride(Tq);
    uint8_t *p = static_cast<uint8_t *>(ws);
    BwdWorkspace w;
    w.lse2 = reinterpret_cast<float *>(p);
    w.delta = reinterpret_cast<float *>(p + round256(rows * sizeof(float)));
    w.dq_acc = reinterpret_cast<float *>(p + 2 * round256(rows * sizeof(float)));
    uint8_t *det = p + 2 * round256(rows * sizeof(float)) + round256(rows * d * sizeof(float));
    w.kvmax = reinterpret_cast<float *>(det);
    w.bound = reinterpret_cast<int *>(det + (size_t)BH * 2 * sizeof(float));
    return w;
}


// Every check of the backward's arguments except those of the workspace and the device:
// sizes, flags, scale, head width, and the tensors' presence, alignment and overlaps.
// Makes no CUDA call.  OK also when there is nothing to compute.
int bwd_check_args(const void *q, const void *k, const void *v, const void *o, const float *lse, const void *dO,
                   const void *dq, const void *dk, const void *dv, int B, int H, int Tq, int Tk, int d,
                   const MaskSpec &mask, float scale)
{
    int st = check_sizes(B, H, Tq, Tk, d, 0, scale);
    if (st != OK)
        return st;
    if (mask.left < -1 || mask.right < -1 || mask.per_head < 0 || mask.per_head > 1)
        return ERR_INVALID_ARG;
    if (d == 256)
        return ERR_UNSUPPORTED;
    const size_t bh = (size_t)B * H;
    if (bh == 0 || (Tq == 0 && Tk == 0))
        return OK;
    const size_t nq = bh * Tq * d * 2, nk = bh * Tk * d * 2, nl = bh * Tq * sizeof(float);
    if ((Tq > 0 && (!q || !o || !lse || !dO || !dq)) || (Tk > 0 && (!k || !v || !dk || !dv)))
        return ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse) || !aligned16(dO) ||
        !aligned16(dq) || !aligned16(dk) || !aligned16(dv))
        return ERR_INVALID_ARG;
    const void *ins[6] = {q, k, v, o, lse, dO};
    const size_t in_n[6] = {nq, nk, nk, nq, nl, nq};
    const void *outs[3] = {dq, dk, dv};
    const size_t out_n[3] = {nq, nk, nk};
    const size_t nm = (mask.per_head ? bh : 1) * (size_t)((Tq + 127) / 128) * ((Tk + 127) / 128);
    for (int i = 0; i < 3; ++i) {
        for (int j = 0; j < 6; ++j)
            if (overlaps(outs[i], out_n[i], ins[j], in_n[j]))
                return ERR_INVALID_ARG;
        for (int j = i + 1; j < 3; ++j)
            if (overlaps(outs[i], out_n[i], outs[j], out_n[j]))
                return ERR_INVALID_ARG;
        if (mask.block && overlaps(outs[i], out_n[i], mask.block, nm))
            return ERR_INVALID_ARG;
    }
    return OK;
}

}  // namespace fa

// ================================================================ C ABI
extern "C" {

int fa_fwd(const void *q, const void *k, const void *v, void *o, float *lse, int B, int H, int Tq, int Tk, int d,
           int causal, float scale, fa_stream_t stream)
{
    int st = fa::check_fwd(q, k, v, o, lse, B, H, Tq, Tk, d, causal, scale, 2);
    if (st != fa::OK)
        return st;
    const int BH = B * H;
    if ((size_t)BH * Tq == 0)
        return FA_OK;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (Tk == 0)
        return fa::fill_empty_launch(o, lse, (size_t)BH * Tq, d, 2, s);
    return fa::fwd_bf16_launch(q, k, v, o, lse, BH, Tq, Tk, d, fa::causal_spec(causal), scale, s);
}

int fa_fwd_masked(const void *q, const void *k, const void *v, void *o, float *lse, int B, int H, int Tq, int Tk,
                  int d, int window_left, int window_right, const unsigned char *block_mask, int mask_per_head,
                  float scale, fa_stream_t stream)
{
    if (window_left < -1 || window_right < -1 || mask_per_head < 0 || mask_per_head > 1)
        return FA_ERR_INVALID_ARG;
    int st = fa::check_fwd(q, k, v, o, lse, B, H, Tq, Tk, d, 0, scale, 2);
    if (st != fa::OK)
        return st;
    const int BH = B * H;
    if ((size_t)BH * Tq == 0)
        return FA_OK;
    if (block_mask) {
        const size_t nm = (size_t)(mask_per_head ? BH : 1) * ((Tq + 127) / 128) * ((Tk + 127) / 128);
        const size_t nq = (size_t)BH * Tq * d * 2, nl = (size_t)BH * Tq * sizeof(float);
        if (fa::overlaps(block_mask, nm, o, nq) || fa::overlaps(block_mask, nm, lse, nl))
            return FA_ERR_INVALID_ARG;
    }
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (Tk == 0)
        return fa::fill_empty_launch(o, lse, (size_t)BH * Tq, d, 2, s);
    const fa::MaskSpec m{window_left, window_right, block_mask, mask_per_head};
    return fa::fwd_bf16_launch(q, k, v, o, lse, BH, Tq, Tk, d, m, scale, s);
}

size_t fa_fp8_vt_stride(int Tk) { return Tk < 0 ? 0 : fa::fp8_vt_stride(Tk); }

int fa_fp8_quantize(const void *q, const void *k, const void *v, const float *signs, int B, int H, int Tq, int Tk,
                    int d, void *q8, void *k8, void *vt8, float *q_descale, float *k_descale, float *v_descale,
                    fa_stream_t stream)
{
    int st = fa::check_sizes(B, H, Tq, Tk, d, 0, 1.f);
    if (st != fa::OK)
        return st;
    const int BH = B * H;
    const size_t nq = (size_t)BH * Tq * d, nk = (size_t)BH * Tk * d, nvt = (size_t)BH * d * fa::fp8_vt_stride(Tk);
    // buffers of a tensor with no elements may be null
    if (!fa::present16(q, nq) || !fa::present16(q8, nq) || !fa::present16(q_descale, nq) ||
        !fa::present16(k, nk) || !fa::present16(v, nk) || !fa::present16(k8, nk) || !fa::present16(vt8, nk) ||
        !fa::present16(k_descale, nk) || !fa::present16(v_descale, nk) || (signs && !fa::aligned16(signs)))
        return FA_ERR_INVALID_ARG;
    const size_t nqd = (size_t)BH * ((Tq + 127) / 128) * 4, nkd = (size_t)BH * ((Tk + 127) / 128) * 4,
                 nvd = (size_t)BH * d * 4;
    const void *outs[6] = {q8, k8, vt8, q_descale, k_descale, v_descale};
    const size_t nouts[6] = {nq, nk, nvt, nqd, nkd, nvd};
    const void *ins[4] = {q, k, v, signs};
    const size_t nins[4] = {nq * 2, nk * 2, nk * 2, signs ? (size_t)d * 4 : 0};
    for (int i = 0; i < 6; ++i) {
        for (int j = 0; j < 4; ++j)
            if (fa::overlaps(outs[i], nouts[i], ins[j], nins[j]))
                return FA_ERR_INVALID_ARG;
        for (int j = i + 1; j < 6; ++j)
            if (fa::overlaps(outs[i], nouts[i], outs[j], nouts[j]))
                return FA_ERR_INVALID_ARG;
    }
    if ((size_t)BH * (Tq > Tk ? Tq : Tk) == 0)
        return FA_OK;
    if ((st = fa::check_device()) != fa::OK)
        return st;
    return fa::fp8_quantize_launch(q, k, v, signs, BH, Tq, Tk, d, q8, k8, vt8, q_descale, k_descale, v_descale,
                                   reinterpret_cast<cudaStream_t>(stream));
}

int fa_fwd_fp8(const void *q8, const void *k8, const void *vt8, const float *q_descale, const float *k_descale,
               const float *v_descale, void *o, float *lse, int B, int H, int Tq, int Tk, int d, int causal,
               float scale, fa_stream_t stream)
{
    int st = fa::check_sizes(B, H, Tq, Tk, d, causal, scale);
    if (st != fa::OK)
        return st;
    if (d != 128)
        return FA_ERR_UNSUPPORTED;
    const int BH = B * H;
    const size_t nqe = (size_t)BH * Tq, nke = (size_t)BH * Tk;
    if (!fa::present16(q8, nqe) || !fa::present16(o, nqe) || !fa::present16(lse, nqe) ||
        !fa::present16(q_descale, nqe) || !fa::present16(k8, nke * nqe) || !fa::present16(vt8, nke * nqe) ||
        !fa::present16(k_descale, nke * nqe) || !fa::present16(v_descale, nke * nqe))
        return FA_ERR_INVALID_ARG;
    const size_t no = (size_t)BH * Tq * d * 2, nl = (size_t)BH * Tq * 4;
    const void *ins[6] = {q8, k8, vt8, q_descale, k_descale, v_descale};
    const size_t nins[6] = {(size_t)BH * Tq * d, (size_t)BH * Tk * d, (size_t)BH * d * fa::fp8_vt_stride(Tk),
                            (size_t)BH * ((Tq + 127) / 128) * 4, (size_t)BH * ((Tk + 127) / 128) * 4,
                            (size_t)BH * d * 4};
    for (int j = 0; j < 6; ++j)
        if (fa::overlaps(o, no, ins[j], nins[j]) || fa::overlaps(lse, nl, ins[j], nins[j]))
            return FA_ERR_INVALID_ARG;
    if (fa::overlaps(o, no, lse, nl))
        return FA_ERR_INVALID_ARG;
    if ((size_t)BH * Tq == 0)
        return FA_OK;
    if ((st = fa::check_device()) != fa::OK)
        return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (Tk == 0)
        return fa::fill_empty_launch(o, lse, (size_t)BH * Tq, d, 2, s);
    return fa::fwd_fp8_launch(q8, k8, vt8, q_descale, k_descale, v_descale, o, lse, BH, Tq, Tk, d, causal, scale, s);
}

size_t fa_decode_workspace_bytes(int B, int H, int Tq, int Tk, int d)
{
    if (fa::check_sizes(B, H, Tq, Tk, d, 0, 1.f) != fa::OK || Tq > fa::decode_max_rows(d))
        return 0;
    const size_t n = fa::decode_workspace_bytes(B * H, Tq, Tk, d);
    return n > 256 ? n : 256;
}

int fa_decode(const void *q, const void *k, const void *v, void *o, float *lse, int B, int H, int Tq, int Tk, int d,
              int causal, float scale, void *workspace, size_t workspace_bytes, fa_stream_t stream)
{
    int st = fa::check_fwd(q, k, v, o, lse, B, H, Tq, Tk, d, causal, scale, 2);
    if (st != fa::OK)
        return st;
    if (Tq > fa::decode_max_rows(d))
        return FA_ERR_UNSUPPORTED;
    const int BH = B * H;
    if ((size_t)BH * Tq == 0)
        return FA_OK;
    const size_t need = fa::decode_workspace_bytes(BH, Tq, Tk, d);
    if (need > 0) {
        if (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
            return FA_ERR_INVALID_ARG;
        const size_t nq = (size_t)BH * Tq * d * 2, nk = (size_t)BH * Tk * d * 2, nl = (size_t)BH * Tq * sizeof(float);
        if (fa::overlaps(workspace, need, q, nq) || fa::overlaps(workspace, need, k, nk) ||
            fa::overlaps(workspace, need, v, nk) || fa::overlaps(workspace, need, o, nq) ||
            fa::overlaps(workspace, need, lse, nl))
            return FA_ERR_INVALID_ARG;
    }
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (Tk == 0)
        return fa::fill_empty_launch(o, lse, (size_t)BH * Tq, d, 2, s);
    return fa::decode_launch(q, k, v, o, lse, BH, Tq, Tk, d, causal, scale, workspace, s);
}

int fa_fwd_f32(const float *q, const float *k, const float *v, float *o, float *lse, int B, int H, int Tq, int Tk,
               int d, int causal, float scale, fa_stream_t stream)
{
    int st = fa::check_fwd(q, k, v, o, lse, B, H, Tq, Tk, d, causal, scale, 4);
    if (st != fa::OK)
        return st;
    const int BH = B * H;
    if ((size_t)BH * Tq == 0)
        return FA_OK;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (Tk == 0)
        return fa::fill_empty_launch(o, lse, (size_t)BH * Tq, d, 4, s);
    return fa::fwd_f32_launch(q, k, v, o, lse, BH, Tq, Tk, d, causal, scale, s);
}

size_t fa_bwd_workspace_bytes(int B, int H, int Tq, int Tk, int d)
{
    if (B < 0 || H < 0 || Tq < 0 || Tk < 0 || (d != 64 && d != 128 && d != 256))
        return 0;
    if ((long long)B * H > INT_MAX)   // the kernels index heads with 32-bit integers
        return 0;
    return fa::bwd_workspace_bytes((size_t)B * H, Tq, d);
}


static int bwd_common(const void *q, const void *k, const void *v, const void *o, const float *lse, const void *dO,
                      void *dq, void *dk, void *dv, int B, int H, int Tq, int Tk, int d, const fa::MaskSpec &mask,
                      float scale, void *workspace, size_t workspace_bytes, int stages, fa_stream_t stream)
{
    int st = fa::bwd_check_args(q, k, v, o, lse, dO, dq, dk, dv, B, H, Tq, Tk, d, mask, scale);
    if (st != fa::OK)
        return st;
    const size_t bh = (size_t)B * H;
    if (bh == 0 || (Tq == 0 && Tk == 0))
        return FA_OK;
    const size_t nq = bh * Tq * d * 2, nk = bh * Tk * d * 2, nl = bh * Tq * sizeof(float);
    const size_t need = fa::bwd_workspace_bytes(bh, Tq, d);
    if (need > 0 && (!workspace || workspace_bytes < need))
        return FA_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
        return FA_ERR_INVALID_ARG;
    const void *ins[6] = {q, k, v, o, lse, dO};
    const size_t in_n[6] = {nq, nk, nk, nq, nl, nq};
    void *outs[4] = {dq, dk, dv, workspace};
    const size_t out_n[4] = {nq, nk, nk, need};
    for (int i = 0; i < 4; ++i) {
        for (int j = 0; j < 6; ++j)
            if (fa::overlaps(outs[i], out_n[i], ins[j], in_n[j]))
                return FA_ERR_INVALID_ARG;
        for (int j = i + 1; j < 4; ++j)
            if (fa::overlaps(outs[i], out_n[i], outs[j], out_n[j]))
                return FA_ERR_INVALID_ARG;
        if (mask.block) {
            const size_t nm = (mask.per_head ? bh : 1) * (size_t)((Tq + 127) / 128) * ((Tk + 127) / 128);
            if (fa::overlaps(outs[i], out_n[i], mask.block, nm))
                return FA_ERR_INVALID_ARG;
        }
    }
    st = fa::check_device();
    if (st != fa::OK)
        return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const fa::BwdWorkspace ws = fa::bwd_workspace_carve(workspace, (int)bh, Tq, d);
    return fa::bwd_launch(q, k, v, o, lse, dO, dq, dk, dv, (int)bh, Tq, Tk, d, mask, scale, ws, stages, s);
}

static int causal_ok(int causal) { return causal == 0 || causal == 1; }

int fa_bwd(const void *q, const void *k, const void *v, const void *o, const float *lse, const void *dO, void *dq,
           void *dk, void *dv, int B, int H, int Tq, int Tk, int d, int causal, float scale, void *workspace,
           size_t workspace_bytes, fa_stream_t stream)
{
    if (!causal_ok(causal))
        return FA_ERR_INVALID_ARG;
    return bwd_common(q, k, v, o, lse, dO, dq, dk, dv, B, H, Tq, Tk, d, fa::causal_spec(causal), scale, workspace,
                      workspace_bytes, 7, stream);
}

int fa_bwd_masked(const void *q, const void *k, const void *v, const void *o, const float *lse, const void *dO,
                  void *dq, void *dk, void *dv, int B, int H, int Tq, int Tk, int d, int window_left, int window_right,
                  const unsigned char *block_mask, int mask_per_head, int deterministic, float scale,
                  void *workspace, size_t workspace_bytes, fa_stream_t stream)
{
    if (deterministic < 0 || deterministic > 1)
        return FA_ERR_INVALID_ARG;
    const fa::MaskSpec m{window_left, window_right, block_mask, mask_per_head};
    return bwd_common(q, k, v, o, lse, dO, dq, dk, dv, B, H, Tq, Tk, d, m, scale, workspace, workspace_bytes,
                      7 | (deterministic ? fa::kBwdDeterministic : 0), stream);
}

int fa_bwd_deterministic(const void *q, const void *k, const void *v, const void *o, const float *lse,
                         const void *dO, void *dq, void *dk, void *dv, int B, int H, int Tq, int Tk, int d,
                         int causal, float scale, void *workspace, size_t workspace_bytes, fa_stream_t stream)
{
    if (!causal_ok(causal))
        return FA_ERR_INVALID_ARG;
    return bwd_common(q, k, v, o, lse, dO, dq, dk, dv, B, H, Tq, Tk, d, fa::causal_spec(causal), scale, workspace,
                      workspace_bytes, 7 | fa::kBwdDeterministic, stream);
}

int fa_bwd_stage(int stage, const void *q, const void *k, const void *v, const void *o, const float *lse,
                 const void *dO, void *dq, void *dk, void *dv, int B, int H, int Tq, int Tk, int d, int causal,
                 float scale, void *workspace, size_t workspace_bytes, fa_stream_t stream)
{
    if (stage < 1 || stage > 3 || !causal_ok(causal))
        return FA_ERR_INVALID_ARG;
    return bwd_common(q, k, v, o, lse, dO, dq, dk, dv, B, H, Tq, Tk, d, fa::causal_spec(causal), scale, workspace,
                      workspace_bytes, 1 << (stage - 1), stream);
}

// The status word of the first kernel file that has one (all are read and cleared): those with waits come
// before those that report indexes alone, so that a timeout is told first.
static int fetch_status(cudaStream_t s, int *word)
{
    int w[5] = {0, 0, 0, 0, 0};
    if (fa::fwd_status_fetch_clear(s, &w[0]) != fa::OK || fa::bwd_status_fetch_clear(s, &w[1]) != fa::OK ||
        fa::dec_status_fetch_clear(s, &w[2]) != fa::OK)
        return fa::ERR_CUDA;
    if (fa::status_is_in_use(fa::STATUS_PAGED) && fa::paged_status_fetch_clear(s, &w[3]) != fa::OK)
        return fa::ERR_CUDA;
    if (fa::status_is_in_use(fa::STATUS_CACHE) && fa::cache_status_fetch_clear(s, &w[4]) != fa::OK)
        return fa::ERR_CUDA;
    for (int i = 0; i < 5 && *word == 0; ++i)
        *word = w[i];
    return fa::OK;
}

int fa_sync_status(fa_stream_t stream)
{
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (cudaStreamSynchronize(s) != cudaSuccess)
        return FA_ERR_CUDA;
    int word = 0;
    return fetch_status(s, &word) == fa::OK ? (word & 0xFF) : FA_ERR_CUDA;
}

const char *fa_status_string(int status)
{
    switch (status) {
    case FA_OK:
        return "ok";
    case FA_ERR_INVALID_ARG:
        return "invalid argument (null or misaligned pointer, bad size or flag, overlapping output, bad scale)";
    case FA_ERR_UNSUPPORTED:
        return "unsupported (head width, backward d=256, or a device other than sm_103)";
    case FA_ERR_CUDA:
        return "CUDA runtime or driver error";
    case FA_ERR_TIMEOUT:
        return "a device-side bounded wait timed out; outputs of that call are invalid";
    case FA_ERR_BAD_INDEX:
        return "a length, count or page number in device memory is out of range; that sequence or page was left out";
    default:
        return "unknown status";
    }
}

#if FA_TEST_WITHHOLD
// Test-only exports (absent from the product library): arm one withheld arrive for the
// next matching launch, count the reads of the cache kernels' status words, and read the raw status word
// (wait site << 8 | status).
void fa_test_withhold(int which)
{
    std::lock_guard<std::mutex> lock(fa::g_withhold_mu);
    fa::g_withhold = which;
}

int fa_test_status_reads(void) { return fa::g_status_reads; }

int fa_test_status_word(fa_stream_t stream)
{
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (cudaStreamSynchronize(s) != cudaSuccess)
        return -1;
    int word = 0;
    return fetch_status(s, &word) == fa::OK ? word : -1;
}
#endif

}  // extern "C"
