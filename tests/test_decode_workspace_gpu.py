"""The workspace of the single tokens' attention: as many bytes as are asked for are enough, none
behind them is written, and what it held before does not matter."""
from __future__ import annotations

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


# groups of up to 2, 4, 8 and 16 heads and of more, whose parts and warps differ
@pytest.mark.parametrize("G", [1, 2, 4, 7, 16, 40])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,Hkv", [([6000], 1), ([700, 30, 0, 5000, 17] * 12, 2)])
def test_no_more_than_it_asks_for(G, d, lens, Hkv):
    pb = su.Decode(lens, G * Hkv, Hkv, d, 16, seed=G)
    need, guard = binding.paged_decode_workspace_bytes(pb.dims), 1 << 16
    assert need > 0
    ref, tol = pb.expected()
    for fill in (0, 0xFF, 0x7F):  # zeros, NaNs, huge values
        buf = torch.full((need + guard,), fill, dtype=torch.uint8, device=DEV)
        buf[need:] = 0xA5
        got = binding.gist_attn_paged_decode(*pb.args(), workspace=buf[:need], dims=pb.dims)
        su.near(got, ref, tol)
        assert (buf[need:] == 0xA5).all()


def test_refusals_are_of_the_workspace():
    pb = su.Decode([40], 8, 2, 64, 16)
    need = binding.paged_decode_workspace_bytes(pb.dims)
    buf = torch.empty(need + 512, dtype=torch.uint8, device=DEV)
    for ws in (buf[:need - 1], buf[16:], buf[128:], buf[:0]):
        with pytest.raises(binding.GistAttnError) as e:
            binding.gist_attn_paged_decode(*pb.args(), workspace=ws, dims=pb.dims)
        assert e.value.code == binding.ERR_SCRATCH
    binding.gist_attn_paged_decode(*pb.args(), workspace=buf[256:256 + need], dims=pb.dims)
