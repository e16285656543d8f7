"""Calls of the ragged serving step at the edges of what its documentation allows."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import paged_utils as pu
from attention_cached_kv_gb300 import binding
from test_paged_range_gpu import check

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    binding.load_library()
    yield
    torch.cuda.empty_cache()


def test_many_chunks_that_see_no_key():
    """Hundreds of prompt chunks that were not served, one after another in a block of the
    grid, among a few that were."""
    served = [0, 150, 399]
    pb = pu.Problem([30 if r in served else 0 for r in range(400)], [17] * 400, 2, 1, 64, 16, seed=3)
    pb.kv_len = np.array([47 if r in served else 0 for r in range(400)])
    check(pb, "unserved")
