"""4-bit projections around the sizes where one kernel takes over from the other: right on both sides,
and more tokens take about as long as one more or one less."""
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


def dims_of(T, Hq):
    return dict(num_requests=T, num_tokens=T, max_new=1, num_q_heads=Hq, num_kv_heads=1, head_dim=64, block_len=16, max_blocks=1,
                num_blocks=1, num_layers=1, layer=0, rope_theta=1e4, softmax_scale=0.0)


# inputs / 64, outputs, group: small weights, some around each border, few rows of long inputs, large ones
SIZES = [(4, 256, 32), (16, 1040, 64), (16, 2064, 128), (16, 4112, 64), (64, 2000, 32), (512, 48, 128), (128, 1040, 128), (1024, 16, 128),
         (48, 4096, 64)]


@pytest.mark.parametrize("Hq,N,group", SIZES)
def test_both_sides(Hq, N, group):
    K = Hq * 64
    w = su.W4(N, K, group, seed=Hq)
    x = su.bf16(np.random.default_rng(N).standard_normal((65, Hq, 64)))
    xd, wd, sd = x.to(DEV), w.w.to(DEV), w.scale.to(DEV)
    ref, off = w.times(x.double().numpy().reshape(65, K))
    for T in (1, 2, 3, 7, 8, 9, 15, 16, 17, 24, 25, 32, 33, 40, 64, 65):
        y = torch.full((T + 1, N), 7.0, dtype=torch.bfloat16, device=DEV)
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        binding.gist_out_proj_w4(xd[:T], wd, sd, y[:T], group=group, dims=dims_of(T, Hq), status=status)
        su.near(y[:T], ref[:T], off[:T] + su.BF16 * 1.01 * np.abs(ref[:T]), f"{T} tokens")
        assert int(status) == 0 and (y[T:] == 7.0).all()


@pytest.mark.parametrize("Hq,N", [(64, 4096), (64, 6144), (128, 8192), (16, 1024), (14, 1152), (64, 1536)])
def test_a_token_more_is_no_cliff(Hq, N):
    """The time of a call may double from a number of tokens to the next one tried, with a us for launches: where
    the rule between the kernels stood at 16 tokens, 17 took a quarter to a seventh of 16's time."""
    K = Hq * 64
    w, s = (torch.zeros((N, n), dtype=t, device=DEV) for n, t in ((K // 2, torch.uint8), (K // 64, torch.bfloat16)))

    def us(T):
        x, y = torch.zeros((T, Hq, 64), dtype=torch.bfloat16, device=DEV), torch.empty((T, N), dtype=torch.bfloat16, device=DEV)
        g = torch.cuda.CUDAGraph()
        binding.gist_out_proj_w4(x, w, s, y, group=64, dims=dims_of(T, Hq))
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            for _ in range(20):
                binding.gist_out_proj_w4(x, w, s, y, group=64, dims=dims_of(T, Hq))
        best = float("inf")
        for _ in range(6):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            g.replay()
            b.record()
            b.synchronize()
            best = min(best, a.elapsed_time(b) * 1e3 / 20)
        return best

    tokens = [1, 2, 3, 8, 9, 16, 17, 32, 33, 64]
    took = [us(T) for T in tokens]
    print(N, K, [f"{T}: {t:.1f}" for T, t in zip(tokens, took)])
    for a, b in zip(took, took[1:]):
        assert max(a, b) <= 2 * min(a, b) + 1
    assert max(took) <= 4 * min(took) + 1
