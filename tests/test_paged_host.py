"""The paged cache's host side and what can be read off its kernels' source (no GPU needed)."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def hstu():
    import hstu_sequential_transduction_layer_b200 as m
    return m


def kernel_body(name):
    """A kernel's definition, comments taken out."""
    path = os.path.join(ROOT, "hstu_sequential_transduction_layer_b200", "csrc", "paged_kernels.cuh")
    text = re.sub(r"//[^\n]*", "", open(path).read())
    at = re.search(r"__global__[^;{]*\b%s\(" % name, text).start()
    return text[at:text.index("\n}\n", at)]


def test_a_cluster_has_started_before_its_shared_memory_is_touched():
    """A CTA's shared memory may be accessed by its cluster only once it runs: the selection waits for a
    cluster barrier before the search, whose first step stores to the other CTAs, and arrives on it
    behind the return of sequences that are short enough (all of the cluster's CTAs return there)."""
    body = kernel_body("evict_select_kernel")
    arrive, wait = body.find("cluster_arrive()"), body.find("cluster_wait()")
    search = body.index("for (; pass < 3 && in_bin != want; pass++)")
    assert 0 <= arrive < wait < search
    assert body.index("return;") < arrive
    assert "map_shared_rank" not in body[:wait]
