"""Child process of test_more_timeout_gpu.py (not collected by pytest: no test_ prefix).

The paged decode under a window and over a shared prefix with the test-only library, in which one launch may leave
out the loader's arrive for its first tile (see paged_timeout_child.py).  For each case: arm it, make the call, read
the raw status word, then make the same call normally and compare it with the product library's.  The
parent sets FA_WAIT_TIMEOUT_MS.  Prints one JSON line.
"""
import ctypes
import json
import os
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, os.path.dirname(HERE))
sys.path.insert(0, HERE)

import torch  # noqa: E402

from exact_io_aware_05_gb300 import build, fa  # noqa: E402
from test_cache_gpu import gen, make_cache, randn  # noqa: E402
from test_shared_gpu import shared_cache  # noqa: E402

WITHHOLD_RANGE_FULL, WITHHOLD_PREFIX_FULL = 5, 6


def main():
    lib = ctypes.CDLL(build.TEST_SO)
    for name in ("fa_decode_paged_window", "fa_decode_paged_shared", "fa_sync_status"):
        getattr(lib, name).argtypes = getattr(fa.lib(), name).argtypes
    lib.fa_test_withhold.argtypes = [ctypes.c_int]
    lib.fa_test_status_word.argtypes = [ctypes.c_void_p]
    stream = torch.cuda.current_stream().cuda_stream
    assert lib.fa_sync_status(stream) == 0
    out = {}
    for name, shared, lens, Hq, d, fp8 in (("window", False, [40], 4, 128, False), ("long_window_e4m3", False, [9000, 5000], 4, 128, True),
                                           ("prefix", True, [5, 9], 8, 128, False), ("prefix_d256", True, [5, 0], 4, 256, False),
                                           ("prefix_e4m3", True, [5, 9], 8, 64, True), ("prefix_one_tile", True, [5], 2, 64, False)):
        P = 64 if name == "prefix_one_tile" else 4096
        if shared:
            cache, pages = shared_cache(fa, 5, P, lens, 2, d, 16, fp8)
        else:
            cache = make_cache(fa, 5, lens, 2, d, 16, fp8)
        q = randn(gen(6), len(lens), Hq, 1, d)
        o, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
        n = fa.fa_decode_paged_shared_workspace_bytes(cache, Hq, 1, pages) if shared else fa.fa_decode_paged_window_workspace_bytes(cache, Hq)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")

        def call():
            if shared:
                return lib.fa_decode_paged_shared(cache._ref, q.data_ptr(), o.data_ptr(), lse.data_ptr(), Hq, 1, 1, pages.data_ptr(), pages.numel(),
                                                  0.1, ws.data_ptr(), n, stream)
            return lib.fa_decode_paged_window(cache._ref, q.data_ptr(), o.data_ptr(), lse.data_ptr(), Hq, 1, 4000, 4, 0.1, ws.data_ptr(), n, stream)
        res = {}
        lib.fa_test_withhold(WITHHOLD_PREFIX_FULL if shared else WITHHOLD_RANGE_FULL)
        res["launch"] = call()
        res["word"] = lib.fa_test_status_word(stream)
        o.fill_(7)
        res["again_launch"] = call()
        res["again_status"] = lib.fa_sync_status(stream)
        first = o.clone(), lse.clone()
        call()
        res["repeats"] = bool(torch.equal(first[0], o) and torch.equal(first[1], lse)) and lib.fa_sync_status(stream) == 0
        want = fa.attention_decode_paged(cache, q, 0.1) if shared else fa.attention_decode_paged(cache, q, 0.1, window=(4000, 0), sinks=4)
        # a prefix's probabilities have 8 bits, the decode's 16: 2^-8 of sums of |v| < 6 and a bf16 step
        res["off"] = float((o.float() - want[0].float()).abs().max())
        res["off_lse"] = float((lse - want[1]).abs().max())
        out[name] = res
    print(json.dumps(out))


if __name__ == "__main__":
    main()
