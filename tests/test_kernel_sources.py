"""Host test: the hash that ties a committed profile to its kernel covers every source that the kernel is compiled from."""
import os
import re

import pytest

import bench

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "structured_sparse_long_gb300", "csrc")


def compiled_from(name):
    """A source and the headers of its folder that it includes, directly or not."""
    seen, todo = set(), [name]
    while todo:
        at = todo.pop()
        if at not in seen and os.path.exists(os.path.join(CSRC, at)):
            seen.add(at)
            with open(os.path.join(CSRC, at), encoding="utf-8") as fh:
                todo += re.findall(r'^\s*#include "([^"]+)"', fh.read(), flags=re.M)
    return seen


@pytest.mark.parametrize("kind", sorted(bench.KERNEL_SOURCES))
def test_profile_hash_covers_the_kernels_headers(kind):
    sources = bench.KERNEL_SOURCES[kind]
    assert set(sources) == compiled_from(sources[0])
