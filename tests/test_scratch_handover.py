"""The kernels that run two roles in one grid first plan in shared memory that the roles then fill by TMA.
Nothing that a run shows tells whether the two are ordered, so the sources are looked at: the last barrier
before the roles is the one with the proxy fence, and the fence stands before it."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "pagedattention_paged_kv_gb300", "csrc")


def text(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_the_barrier_has_the_fence():
    body = re.search(r"void hand_over_smem\(\) \{(.*?)\}", text("tcgen05.cuh"), re.S).group(1)
    assert re.sub(r"\s", "", body) == "fence_async_smem();__syncthreads();"


@pytest.mark.parametrize("name,kernel", [("paged_shared.cu", "paged_shared_kernel"), ("paged_varlen.cu", "cta_sum")])
def test_scratch_goes_over_to_the_copies(name, kernel):
    src = text(name)
    plan = src[src.index(kernel + "("):]
    plan = plan[:re.search(r"\bdecode_cta<|\n\}", plan).start()]
    barriers = re.findall(r"__syncthreads\w*|hand_over_smem", plan)
    assert barriers[-1] == "hand_over_smem"
