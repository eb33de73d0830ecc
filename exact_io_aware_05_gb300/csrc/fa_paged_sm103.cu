// fa_paged_sm103.cu -- attention of a few new rows over all entries of the paged key/value cache
// (kernels in fa_paged.cuh).
#include "fa_paged.cuh"

namespace fa {

size_t paged_workspace_bytes(int B, int Hq, int Hkv, int Tq, int max_len, int d, int accumulate)
{
    return where_bytes(B) + part_bytes(Hq / Hkv * Tq, d) + (accumulate ? round256((size_t)B * Hq * Tq * max_len * sizeof(float)) : 0);
}

int paged_launch(const fa_kv_cache &c, const void *q, void *o, float *lse, int Hq, int Tq, int causal, float scale,
                 int accumulate, void *workspace, cudaStream_t s, const int *first_pages, int n_first)
{
    status_in_use(STATUS_PAGED);
    PagedArgs a = paged_args(c, q, o, lse, Hq, Tq, causal, scale, workspace);
    a.first_pages = first_pages;
    a.n_first = n_first;
    // several row blocks of a unit: only the join can add their weights
    const bool can = !accumulate || a.RB == 1;
    a.whole = can && a.cap <= (c.d == 256 ? kWholeSlots / 2 : kWholeSlots);
    a.may_whole = can;
    a.scores = accumulate ? reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + where_bytes(c.B) + part_bytes(a.M, c.d)) : nullptr;
#if FA_TEST_WITHHOLD
    a.withhold = test_withhold_take(WITHHOLD_PAGED_FULL, WITHHOLD_PAGED_FULL);
#endif
    return c.d == 64 ? paged_run<64, false>(c, a, s) : c.d == 128 ? paged_run<128, false>(c, a, s) : paged_run<256, false>(c, a, s);
}

int paged_status_fetch_clear(cudaStream_t s, int *host_word) { return paged_words_fetch_clear(s, host_word); }

}  // namespace fa
