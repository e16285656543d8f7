"""Attention of single tokens for a server that keeps many slots, few of which have a token in a step:
q_start as the plan leaves it."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import serving_utils as su
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


def spread_out(pb, slots, active):
    """The problem's requests at the slots `active` of so many; the others hold caches of their own,
    which nothing may read (no block of theirs is in the pool)."""
    q, pool, table, kv = pb.args()
    W = table.shape[1]
    big = torch.full((slots, W), 1 << 30, dtype=torch.int32, device=DEV)
    lens = torch.full((slots,), W * pb.bl, dtype=torch.int32, device=DEV)
    at = torch.tensor(active, device=DEV)
    big[at], lens[at] = table, kv
    has = np.zeros(slots, np.int64)
    has[active] = 1
    start = pb.i32(np.concatenate([[0], np.cumsum(has)]))
    return (q, pool, big, lens, start), dict(pb.dims, num_requests=slots)


SLOTS = {
    "first and last": (16384, [0, 16383]),
    "last alone": (16384, [16383]),
    "a few": (5000, [3, 4, 5, 2500, 2501, 4998]),
    "one in a thousand": (16384, list(range(7, 16384, 1000))),
    "one in forty": (4000, list(range(0, 4000, 40))),
    "all but a few": (300, [i for i in range(300) if i % 7]),
    "two runs": (16384, list(range(100, 130)) + list(range(16000, 16040))),
    "fewer than threads": (200, [0, 199]),
}


@pytest.mark.parametrize("name", SLOTS)
@pytest.mark.parametrize("Hq,Hkv,d", [(14, 2, 64), (8, 8, 128), (16, 1, 128)])
def test_scattered_requests(name, Hq, Hkv, d):
    slots, active = SLOTS[name]
    rng = np.random.default_rng(slots + len(active))
    lens = [int(x) for x in rng.integers(1, 2500 if len(active) < 20 else 200, len(active))]
    lens[0] = 0  # one with a token and no key
    pb = su.Decode(lens, Hq, Hkv, d, 32, seed=len(active))
    args, dims = spread_out(pb, slots, active)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = binding.gist_attn_paged_decode(*args, dims=dims, status=status)
    assert int(status) == 0
    su.near(got, *pb.expected(), name)
    # (the bits of the call without empty slots only where the join goes by the same num_requests)
    assert torch.equal(got, binding.gist_attn_paged_decode(*args, dims=dims))


@pytest.mark.parametrize("lens", [[40, 900], [9000, 9000]])
def test_empty_slots_cost_little(lens):
    """Two requests 16 k slots apart.  Every CTA reads all slots (three words each, 43 a thread, some 30 us
    at worst); a walk over them one after another took several hundred us."""
    pb = su.Decode(lens, 8, 2, 64, 64, seed=1)
    args, dims = spread_out(pb, 16384, [0, 16383])
    out, ws = torch.empty_like(args[0]), torch.empty(binding.paged_decode_workspace_bytes(dims), dtype=torch.uint8, device=DEV)
    g = torch.cuda.CUDAGraph()
    binding.gist_attn_paged_decode(*args, out, ws, dims=dims)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        binding.gist_attn_paged_decode(*args, out, ws, dims=dims)
    best = float("inf")
    for _ in range(20):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        g.replay()
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b) * 1e3)
    print(f"{lens}: {best:.1f} us")
    assert best < 100
