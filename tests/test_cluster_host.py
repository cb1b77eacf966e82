"""Clusters of thread blocks, from the kernels' sources (no GPU needed)."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "tiered_sparse_mla_gb300", "csrc")

# what reaches another CTA's shared memory, or barriers in it
REMOTE = re.compile(r"\b(?:dsmem_(?:st|ld|st64|atom_add)|mbar_arrive_(?:peer|remote)|st_cluster_v4|tma_load_pair|bulk_push|commit_both)\("
                    r"|(?:st|ld|atom|red)[\w.]*\.shared::cluster")
WAIT = re.compile(r"\bcluster_(?:wait|sync_all|sync_relaxed)\(|barrier\.cluster\.wait")


def kernels(source):
    with open(os.path.join(CSRC, source)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    for kernel in re.split(r"__global__|__device__ __forceinline__ void (?=\w+_body\()", text)[1:]:
        name = re.search(r"(\w+)\s*\((?!\()", re.sub(r"__launch_bounds__\([^;{]*?\)\s*\n?", "", kernel)).group(1)
        yield name, kernel[kernel.index("{"):]


SOURCES = sorted(f for f in os.listdir(CSRC) if f.endswith(".cu"))


@pytest.mark.parametrize("source", SOURCES)
def test_no_cta_reaches_another_before_all_of_the_cluster_run(source):
    """A CTA's shared memory is there from when the CTA has begun: a cluster barrier has to lie before the
    first access from another one."""
    found = 0
    for name, body in kernels(source):
        remote = REMOTE.search(body)
        if not remote:
            continue
        found += 1
        wait = WAIT.search(body)
        # a wait on the way out (a return behind it) does not count
        while wait and re.match(r"[^{}]*\breturn;", body[wait.end():]):
            wait = WAIT.search(body, wait.end())
        assert wait and wait.start() < remote.start(), f"{source}: {name}"
    assert found or source not in ("hs_resolve.cu", "hs_select.cu", "hs_page_decode.cu", "hs_weights.cu", "hs_evict.cu", "hs_verify.cu")
