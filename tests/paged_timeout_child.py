"""Child process of test_paged_timeout_gpu.py (not collected by pytest: no test_ prefix).

Runs the paged decode with the test-only library libfa_waittest.so, in which one launch may leave out
the loader's arrive for its first tile (the copies are made; the phase is never completed).  For each
case: arm it, make the call, read the raw status word, then make the same call normally and return how
far it is from the 64-bit reference.  The parent sets FA_WAIT_TIMEOUT_MS.  Prints one JSON line.
"""
import ctypes
import json
import os
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, os.path.dirname(HERE))
sys.path.insert(0, HERE)

import numpy as np  # noqa: E402
import torch  # noqa: E402

import paged_ref as R  # noqa: E402
from exact_io_aware_05_gb300 import build, fa  # noqa: E402
from gpu_util import to64  # noqa: E402
from test_cache_gpu import entries, gen, make_cache, randn  # noqa: E402

WITHHOLD_PAGED_FULL = 4
# lengths, query heads, e4m3, a length out of range too
CASES = {"fits_the_ring": ([40], 4, False, False), "last_tiles": ([100, 30], 8, True, False),
         "longer_than_the_ring": ([9000, 5000], 4, False, False), "in_shares_e4m3": ([70000], 40, True, False),
         "beside_a_bad_length": ([40, 50], 4, False, True)}


def main():
    lib = ctypes.CDLL(build.TEST_SO)
    for name in ("fa_decode_paged", "fa_sync_status"):
        getattr(lib, name).argtypes = getattr(fa.lib(), name).argtypes
    lib.fa_test_withhold.argtypes = [ctypes.c_int]
    lib.fa_test_status_word.argtypes = [ctypes.c_void_p]
    stream = torch.cuda.current_stream().cuda_stream
    assert lib.fa_sync_status(stream) == 0
    out = {"reads_before_any_cache_call": lib.fa_test_status_reads()}
    for name, (lens, Hq, fp8, bad) in CASES.items():
        cache = make_cache(fa, 5, lens, 2, 128, 16, fp8)
        q = randn(gen(6), len(lens), Hq, 1, 128)
        o, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
        ws = torch.empty(fa.fa_decode_paged_workspace_bytes(cache, Hq), dtype=torch.uint8, device="cuda")

        def call():
            return lib.fa_decode_paged(cache._ref, q.data_ptr(), o.data_ptr(), lse.data_ptr(), Hq, 1, 1, 0.1, 0, ws.data_ptr(),
                                       ws.numel(), stream)

        res = {}
        if bad:
            cache.lens[1] = -1
        lib.fa_test_withhold(WITHHOLD_PAGED_FULL)
        res["launch"] = call()
        if bad:
            res["status"] = lib.fa_sync_status(stream)
            cache.lens[1] = lens[1]
        else:
            res["word"] = lib.fa_test_status_word(stream)
        o.fill_(7)
        res["again_launch"] = call()
        res["again_status"] = lib.fa_sync_status(stream)
        excess = -1.0
        for b in range(len(lens)):
            k, v = entries(cache, b)
            ro, rl, _, to, tl, _ = R.attend(to64(q[b]), k, v, 0.1, True, Hq // 2, fp8)
            excess = max(excess, float((np.abs(to64(o[b]) - ro) - to - 2.0 ** -8 * np.abs(ro)).max()),
                         float((np.abs(to64(lse[b]) - rl) - tl).max()))
        res["again_excess"] = excess
        out[name] = res
    n = lib.fa_test_status_reads()
    assert lib.fa_sync_status(stream) == 0
    out["reads_after_decodes"] = lib.fa_test_status_reads() - n
    print(json.dumps(out))


if __name__ == "__main__":
    main()
