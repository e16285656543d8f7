"""gist_paged_plan on the GPU against a request-by-request construction: whole
numbers, so every output is equal."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import paged_utils as pu
from attention_cached_kv_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    binding.load_library()


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def check(cached, new, bl, free, free_range, T, W, num_blocks, seed=0):
    rng = np.random.default_rng(seed)
    B = len(cached)
    table = rng.integers(0, num_blocks, (B, W)).astype(np.int64)
    ref = pu.plan(cached, new, table, free, free_range, T, bl, num_blocks)
    dims = dict(num_requests=B, num_tokens=T, max_new=max(list(new) + [1]), num_q_heads=1, num_kv_heads=1, head_dim=64,
                block_len=bl, max_blocks=W, num_blocks=num_blocks, num_layers=1, layer=0, rope_theta=1e4, softmax_scale=0.0)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    t = i32(table)
    got = binding.gist_paged_plan(i32(cached), i32(new), t, i32(free), i32(free_range), dims=dims, status=status)
    torch.cuda.synchronize()
    for name in binding.PagedPlan._fields:
        np.testing.assert_array_equal(getattr(got, name).cpu().numpy(), ref[name], err_msg=name)
    np.testing.assert_array_equal(t.cpu().numpy(), ref["block_table"])
    assert int(status.item()) == ref["status"]
    return ref


@pytest.mark.parametrize("B,bl,cached,new,seed", [
    (1, 16, 100, 1, 0), (3, 1, 9, 4, 1), (32, 256, 4096, 1, 2), (70, 16, 300, 40, 3), (1025, 32, 200, 9, 4),
    (4100, 64, 500, 3, 5), (16384, 16, 20, 2, 6), (5, 48, 500, 3000 // 7, 7), (2, 100, 5, 20000, 8),
])
@pytest.mark.parametrize("pad", [0, 37])
def test_random_lengths(B, bl, cached, new, seed, pad):
    rng = np.random.default_rng(seed)
    c = rng.integers(0, cached + 1, B)
    n = rng.integers(0, new + 1, B)
    c[0] = bl  # ends on a block's edge
    W = -(-int((c + n).max()) // bl) + 2
    need = int((-(-(c + n) // bl) - -(-c // bl)).sum())
    free = rng.permutation(need + 50)[:need + 20]
    ref = check(c, n, bl, free, [5, need + 5 + 3], int(n.sum()) + pad, W, need + 50, seed)
    assert ref["status"] == 0 and ref["free_range"][0] == need + 5


def test_free_list_runs_out():
    """Requests that need blocks are served from the front until the free blocks
    end; requests that need none always are."""
    ref = check([16, 10, 16, 3, 31], [1, 2, 40, 1, 2], 16, [9, 8, 7, 6, 5, 4], [1, 4], 46, 4, 12)
    assert ref["status"] == 8 and list(ref["kv_len"]) == [17, 12, 0, 4, 0]


def test_refused_requests():
    check([-1, 5, 5, 60, 5], [2, -3, 4, 10, 1], 16, list(range(8)), [0, 8], 17, 4, 9)   # lengths, table
    check([5, 5, 5], [4, 4, 4], 16, list(range(8)), [0, 8], 10, 4, 9)                   # token rows
    check([0, 5], [4, 4], 16, [99, 1, 2], [0, 3], 8, 4, 9)                              # a bad free id
    check([0, 5], [4, 4], 16, [1, 2, 3], [2, 99], 8, 4, 9)                              # a range past the list


def test_nothing_to_do():
    check([], [], 16, [1, 2], [0, 2], 5, 4, 9)
    check([7, 0], [0, 0], 16, [1, 2], [0, 2], 0, 4, 9)
    check([7, 0], [0, 0], 16, [1, 2], [0, 2], 3, 4, 9)


@pytest.mark.parametrize("free_range", [[5, -2 ** 31], [2 ** 31 - 1, 3], [-4, 2], [3, 3], [2 ** 31 - 1, -2 ** 31]])
def test_free_ranges_without_a_block(free_range):
    """Ends before the list, before their begin, or far outside give no blocks but
    those in both the range and the list."""
    ref = check([0, 15, 16], [4, 1, 4], 16, [6, 7, 8, 9, 5, 4], free_range, 9, 4, 12)
    if free_range == [-4, 2]:
        assert ref["status"] == 0 and ref["free_range"][0] == 2  # never handed out again
    else:
        assert ref["status"] == 8 and list(ref["kv_len"]) == [0, 16, 0]
