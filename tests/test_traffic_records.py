"""The bench's records of DRAM traffic hold for the decode step's sources, and for nothing else."""

import os
import re

import bench
from moe_decode_layer_gb300 import build

PROFILES = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "profiles")


def test_digest_is_of_the_decode_step():
    names = build.sources_of(build.DECODE_SOURCES)
    assert {"api.cu", "moe_kernels.cuh", "ptx.cuh", "moe_params.h"} <= set(names)
    assert not any(n.startswith("rows_") for n in names)
    # no source is in neither part
    every = set(names) | set(build.sources_of(build.ROWS_SOURCES))
    assert every == {n for n in os.listdir(build.CSRC) if n.endswith((".cu", ".cuh", ".h"))}


def test_records_are_of_the_present_sources():
    """Every recorded row reports its traffic."""
    found = 0
    for name in os.listdir(PROFILES):
        text = open(os.path.join(PROFILES, name)).read()
        if "sources_sha256_16:" not in text or "traffic_bytes_per_launch:" not in text:
            continue
        kernel, workload = re.fullmatch(r"(\w+_kernel)_(\w+)\.md", name).groups()
        traffic, digest = bench.traffic_record(kernel, workload)
        assert traffic and digest in text, name
        found += 1
    assert found == 8
