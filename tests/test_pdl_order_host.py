"""The order that csrc/fa_pdl.cuh asks of kernels that may start while the one before them runs, read from their source:
pdl_wait() in front of every access to device memory, but for the lengths that the joins read past the L1; and in the
kernels whose states are joined pdl_launch() behind pdl_wait(), on which those reads rest.  No GPU is needed."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "exact_io_aware_05_gb300", "csrc")
ACCESS = re.compile(r"a(?:\.own)?\.\w+\[|__ld\w+\(|\*reinterpret_cast<|tma_load|length_of\(|tiles_of<|place_of<")
JOINED = {"paged_kernel", "prefix_kernel"}


def kernels():
    out = {}
    for f in sorted(os.listdir(CSRC)):
        text = open(os.path.join(CSRC, f)).read()
        if "fa_pdl.cuh" not in text:
            continue
        for m in re.finditer(r"__global__.*?(\w+_kernel)\(", text, re.S):
            at = text.index("{", m.end())
            depth, end = 1, at + 1
            while depth:
                depth += {"{": 1, "}": -1}.get(text[end], 0)
                end += 1
            out[m.group(1)] = re.sub(r"//.*", "", text[at:end])
    return out


KERNELS = kernels()


def test_the_kernels_are_found():
    assert JOINED | {"norm_rope_kernel", "norm_bwd_kernel", "append_kernel", "range_join_kernel", "prefix_join_kernel"} <= set(KERNELS)


@pytest.mark.parametrize("name", sorted(KERNELS))
def test_the_wait_comes_first(name):
    body = KERNELS[name]
    if "pdl_launch" not in body and "pdl_wait" not in body:
        pytest.skip("does not overlap")
    before = body[:body.index("pdl_wait()")]
    if name.endswith("join_kernel"):
        before = re.sub(r"__ldcg\(a\.(own\.)?lens \+ b\)", "len", before)
    # tensor memory's base lies in shared memory
    assert not ACCESS.search(before.replace("*reinterpret_cast<uint32_t *>(smem", "").replace("*tmem_slot", "")), name


@pytest.mark.parametrize("name", sorted(JOINED))
def test_joined_kernels_let_the_join_start_behind_their_wait(name):
    assert KERNELS[name].index("pdl_wait()") < KERNELS[name].index("pdl_launch()")
