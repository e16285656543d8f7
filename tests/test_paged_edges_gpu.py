"""Calls of the ragged serving step at the edges of what its documentation allows."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import paged_utils as pu
from attention_cached_kv_gb300 import binding
from test_paged_range_gpu import check, expected

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


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new", [3, 33])
@pytest.mark.parametrize("which,value", [("K", float("nan")), ("V", float("nan")), ("V", float("inf")), ("V", float("-inf"))])
def test_scales_that_are_not_finite_reach_the_tokens_that_see_them(d, new, which, value):
    """The last block's scale, which only the last token of one request sees: that token's
    rows are not finite and reported, all others are what they would be."""
    pb = pu.Problem([48 - new + 1, 200], [new, new], 4, 2, d, 16, seed=6)
    assert pb.kv_len[0] == 49
    ref, tol = expected(pb, False)
    args = list(pb.args())
    args[2][int(pb.table[0, 3]), pb.layer, "KV".index(which)] = value
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = binding.gist_attn_paged_fp8kv(*args, dims=pb.dims, status=st).float().cpu().numpy().astype(np.float64)
    last = new - 1
    assert int(st.item()) == binding.STATUS_RANGE
    assert not np.isfinite(got[last]).any()
    rest = np.arange(len(got)) != last
    assert (np.abs(got - ref) <= tol)[rest].all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("start", [-5, -4096, -2 ** 31])
def test_append_turns_keys_at_negative_positions(d, start):
    """Backwards, as far as forwards."""
    from test_paged_append_gpu import check as check_append, fresh, places
    pb = pu.Problem([3, 9], [9, 2], 2, 2, d, 16, seed=4)
    k, v = fresh(pb, 7)
    slot, position = places(pb)
    check_append(pb, k, v, slot, [p - 3 + start for p in position])


def test_plan_of_the_largest_number_of_token_rows():
    """2^31 - 1 rows, nearly all of them padding: counted past the last without a wrap."""
    T = 2 ** 31 - 1
    i32 = dict(dtype=torch.int32, device=DEV)
    out = [torch.zeros(n, **i32) for n in (3, 2, T, T, 2)]
    dims = dict(num_requests=2, num_tokens=T, max_new=8, num_q_heads=1, num_kv_heads=1, head_dim=64, block_len=16, max_blocks=2,
                num_blocks=9, num_layers=1, layer=0, rope_theta=1e4, softmax_scale=0.0)
    table = torch.tensor([[5, -1], [-1, -1]], **i32)
    st = torch.zeros(1, **i32)
    p = binding.gist_paged_plan(torch.tensor([14, 0], **i32), torch.tensor([4, 3], **i32), table, torch.tensor([7, 8], **i32),
                                torch.tensor([0, 2], **i32), out, dims=dims, status=st)
    assert int(st.item()) == 0 and p.kv_len.tolist() == [18, 3] and p.free_range.tolist() == [2, 2]
    assert p.slot[:8].tolist() == [94, 95, 112, 113, 128, 129, 130, -1]
    for x in (p.slot, p.position):
        for a in range(7, T, 1 << 29):
            assert int(x[a:a + (1 << 29)].max()) == -1 == int(x[a:a + (1 << 29)].min())
