"""The ragged serving step's entry points from several threads and on other streams
than the current one."""
from __future__ import annotations

import threading

import pytest
import torch

from attention_cached_kv_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    binding.load_library()
    yield
    torch.cuda.empty_cache()


def test_plans_of_unlike_sizes_from_two_threads():
    """Neither call takes the other's shared memory away."""
    failed = []

    def calls(B):
        try:
            zeros = torch.zeros(B, dtype=torch.int32, device=DEV)
            table = torch.zeros((B, 1), dtype=torch.int32, device=DEV)
            free, rng = zeros[:4].clone(), torch.tensor([0, 4], dtype=torch.int32, device=DEV)
            dims = dict(num_requests=B, num_tokens=4, max_new=1, num_q_heads=1, num_kv_heads=1, head_dim=64, block_len=16,
                        max_blocks=1, num_blocks=4, num_layers=1, layer=0, rope_theta=1e4, softmax_scale=0.0)
            out = [torch.empty(n, dtype=torch.int32, device=DEV) for n in (B + 1, B, 4, 4, 2)]
            s = torch.cuda.Stream()
            torch.cuda.synchronize()
            for _ in range(3000):
                binding.gist_paged_plan(zeros, zeros, table, free, rng, out, dims=dims, stream=s)
            s.synchronize()
        except Exception as e:  # noqa: BLE001 - reported by the test's own thread
            failed.append((B, e))

    threads = [threading.Thread(target=calls, args=(B,)) for B in (16384, 5000, 9000)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
