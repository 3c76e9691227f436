"""The files that the bench's traffic figures and its library hash go by."""

from __future__ import annotations

import glob
import os
import re

import bench

CSRC = os.path.join("sparse_latent_attention_gb300", "csrc")


def test_every_timed_workload_has_a_traffic_figure():
    """A change to the attention kernels' sources takes the captured figures away: they are captured again."""
    key = bench.kernel_source_hash()
    for name in bench.TIMED_WORKLOADS:
        assert bench.NCU_TRAFFIC.get((key, name), 0) > 0, (key, name)


def test_the_attention_sources_have_their_headers():
    """Every header of the library that they include, directly or through another, is among them."""
    seen, todo = set(), [p for p in bench.ATTN_SOURCES if p.endswith(".cu")]
    while todo:
        path = todo.pop()
        if path in seen:
            continue
        seen.add(path)
        with open(os.path.join(bench.ROOT, path)) as f:
            for name in re.findall(r'^#include "([^"]+)"', f.read(), re.M):
                found = [d for d in (CSRC, "include") if os.path.exists(os.path.join(bench.ROOT, d, name))]
                assert found, (path, name)
                todo.append(os.path.join(found[0], name))
    assert seen == set(bench.ATTN_SOURCES)


def test_the_library_hash_covers_every_header():
    files = {os.path.join(bench.ROOT, p) for p in bench.library_sources()}
    for pattern in ("include/**/*.h", os.path.join(CSRC, "*.cu"), os.path.join(CSRC, "*.cuh")):
        want = set(glob.glob(os.path.join(bench.ROOT, pattern), recursive=True))
        assert want and want <= files, pattern
