"""Kernels that may be on the GPU while the one before them still writes (those launched through
follow.cuh) read no global memory by non-coherent loads, which promise that nothing writes it."""
from __future__ import annotations

import os
import re

import attention_cached_kv_gb300 as pkg

CSRC = os.path.join(os.path.dirname(pkg.__file__), "csrc")


def code(name):
    """A source without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


def test_no_non_coherent_loads_behind_wait_before():
    following = [n for n in os.listdir(CSRC) if n.endswith(".cu") and "launch_following(" in code(n)]
    assert {"paged_bf16.cu", "paged_pages.cu", "proj_w4.cu", "proj_w4_tc.cu"} <= set(following)
    for name in following + ["follow.cuh", "proj_w4.cuh"]:
        assert not re.search(r"global\.nc|__ldg\b|\bldg16\b|__restrict__", code(name)), name
        if name in following:
            kernels, waits = (len(re.findall(p, code(name))) for p in (r"__global__", r"\bwait_before\(\);"))
            assert kernels == waits, name  # each of them waits
