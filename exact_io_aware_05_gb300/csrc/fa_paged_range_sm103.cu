// fa_paged_range_sm103.cu -- attention of a few new rows over a part of the paged key/value cache: a
// sliding window and the first entries (sinks), or the entries behind a shared prefix (kernels in fa_paged.cuh).
//
// The tiles of a sequence are those that any of its rows sees, numbered without the ones between, and are
// shared out like the others': a batch's time goes with its visible entries and not with its lengths. The bytes bound
// it: 64 sequences of 200 to 8000 entries, 8 KV heads of 128, under a window of 1024 with 4 sinks 51 us (265 MB, 5.2 TB/s;
// without the window 164); 16 of 1001 to 65536 in e4m3, 4 KV heads of 64, 4096 and 4: 16 us, of them 3 the start and 4 the
// join.
#include "fa_paged.cuh"

namespace fa {

namespace {

// Units whose rows see at most `span` slots: whole ones as in a table of so many (kWholeSlots).
int run(const fa_kv_cache &c, PagedArgs &a, cudaStream_t s)
{
    a.whole = a.span <= (c.d == 256 ? kWholeSlots / 2 : kWholeSlots);
    a.may_whole = 1;
    a.scores = nullptr;
#if FA_TEST_WITHHOLD
    a.withhold = test_withhold_take(WITHHOLD_RANGE_FULL, WITHHOLD_RANGE_FULL);
#endif
    return c.d == 64 ? paged_run<64, true>(c, a, s) : c.d == 128 ? paged_run<128, true>(c, a, s) : paged_run<256, true>(c, a, s);
}

}  // namespace

int paged_window_launch(const fa_kv_cache &c, const void *q, void *o, float *lse, int Hq, int Tq, int left, int sinks,
                        float scale, void *workspace, cudaStream_t s)
{
    status_in_use(STATUS_RANGE);
    PagedArgs a = paged_args(c, q, o, lse, Hq, Tq, 1, scale, workspace);
    a.left = std::min(left, 1 << 30);
    a.sinks = std::min(sinks, a.cap);
    a.span = (int)std::min<long long>(a.cap, (long long)a.left + Tq + a.sinks);
    return run(c, a, s);
}

// The entries from slot `base` on: o in fp32, and no join.
int paged_behind_launch(const fa_kv_cache &c, const void *q, float *o, float *lse, int Hq, int Tq, int causal, int base, float scale,
                        void *workspace, OwnStates *states, cudaStream_t s)
{
    status_in_use(STATUS_RANGE);
    PagedArgs a = paged_args(c, q, nullptr, lse, Hq, Tq, causal, scale, workspace);
    a.left = -1;
    a.sinks = 0;
    a.base = std::min(base, a.cap);
    a.span = a.cap - a.base;
    a.o32 = o;
    const int st = run(c, a, s);
    *states = OwnStates{o, lse, a.part, a.where, a.lens, a.whole, a.rows, a.RB, a.Hkv, a.kt, a.base, a.cap};
    return st;
}

int paged_range_status_fetch_clear(cudaStream_t s, int *host_word) { return paged_words_fetch_clear(s, host_word); }

}  // namespace fa
