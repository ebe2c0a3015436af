"""CPU checks of the kernels' sources: orders of instructions that no run can
be relied on to show."""
import glob
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "moe_grouped_gemm_fp8_gb300", "csrc")
# a store or an arrival in another CTA's shared memory; the second half of a cluster barrier
REMOTE = r"\b(?:st_shared_cluster_\w+|gd_send_v4|st_async_v4|mbar_arrive_cluster|mapa_shared)\("
BARRIER = r"\b(?:cluster_sync_all|cluster_wait|gd_cluster_wait|cluster_wait_acquire)\(\)"


def _kernels():
    """(file name, text from one `__global__` to the next) of every kernel."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        parts = re.split(r"(?=\b__global__\b)", text)
        for i, part in enumerate(parts[1:]):
            yield "%s:%d" % (os.path.basename(path), i), part


FOUND = [k for k in _kernels() if re.search(REMOTE, k[1])]


@pytest.mark.parametrize("name,text", FOUND, ids=[n for n, _ in FOUND])
def test_remote_shared_memory_is_touched_only_after_a_cluster_barrier(name, text):
    """Another CTA's shared memory exists once that CTA runs, which only a
    cluster barrier tells: one is completed before the first remote access."""
    barrier = re.search(BARRIER, text)
    assert barrier and barrier.start() < re.search(REMOTE, text).start(), name


def test_the_search_finds_the_kernels_with_remote_accesses():
    found = {n.split(":")[0] for n, _ in FOUND}
    assert {"gated_gemv.cu", "gated_decode.cu", "gemm_decode.cu", "gemm_kernel.cuh", "gemm2_kernel.cuh"} <= found
