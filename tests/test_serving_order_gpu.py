"""4-bit projections right behind what writes their inputs, in buffers that are used again: a kernel
may be set up while the one before it still runs, and has to read what that one left."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import serving_utils as su
from attention_cached_kv_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda"
TOKENS = [1, 5, 12, 40, 64, 100]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    binding.load_library()
    yield
    torch.cuda.empty_cache()


def dims_of(T, Hq, **kw):
    return dict(num_requests=T, num_tokens=T, max_new=1, num_q_heads=Hq, num_kv_heads=1, head_dim=64, block_len=16, max_blocks=1,
                num_blocks=1, num_layers=1, layer=0, rope_theta=1e4, softmax_scale=0.0) | kw


@pytest.mark.parametrize("T", TOKENS)
@pytest.mark.parametrize("Hq", [4, 32])
def test_two_buffers_in_turn(T, Hq):
    """a = b w1, b = a w2, ...: each projection's x is what the one before wrote over older values that
    the one before that has read; eagerly and captured."""
    D = Hq * 64
    dims = dims_of(T, Hq)
    ws = [su.W4(D, D, 32, seed=s) for s in range(4)]
    dev = [(w.w.to(DEV), w.scale.to(DEV) * 2) for w in ws]
    x = su.bf16(np.random.default_rng(T).standard_normal((T, D))).to(DEV)
    want, at = [], x
    for w, s in dev * 3:  # one at a time, a buffer each
        torch.cuda.synchronize()
        want.append(binding.gist_out_proj_w4(at, w, s, group=32, dims=dims))
        torch.cuda.synchronize()
        at = want[-1]
    a, b, kept = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)

    def chain():
        src, dst = a, b
        src.copy_(x)
        for w, s in dev * 3:
            binding.gist_out_proj_w4(src, w, s, dst, group=32, dims=dims)
            src, dst = dst, src
        kept.copy_(src)

    for _ in range(30):
        chain()
        assert torch.equal(kept, want[-1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        chain()
    for _ in range(30):
        kept.zero_()
        g.replay()
        assert torch.equal(kept, want[-1])


@pytest.mark.parametrize("T", TOKENS)
def test_weights_and_scales_right_behind_what_writes_them(T):
    """Codes and scales that gist_pages_copy (which may overlap in the same way) writes before each call:
    those of one weight and another in turn."""
    D = 256
    dims = dims_of(T, 4)
    ws = [su.W4(D, D, 32, seed=s) for s in range(2)]
    x = su.bf16(np.random.default_rng(T).standard_normal((T, 4, 64))).to(DEV)
    # pools of three blocks: two weights, and the one in use.  256 x 8 scales are a block of bf16 with one
    # head, 256 x 128 bytes of codes one of bytes with four and 64 rows
    scales = torch.cat([w.scale for w in ws] + [torch.zeros_like(ws[0].scale)]).view(3, 1, 2, 1, 16, 64).to(DEV)
    codes = torch.cat([w.w for w in ws] + [torch.zeros_like(ws[0].w)]).view(3, 1, 2, 4, 64, 64).to(DEV)
    sd, cd = dims_of(1, 1, num_blocks=3), dims_of(1, 4, num_blocks=3, num_kv_heads=4, block_len=64)
    src = [torch.tensor([i], dtype=torch.int32, device=DEV) for i in range(3)]
    w, s = codes[2].view(D, D // 2), scales[2].view(D, D // 32)
    want = [binding.gist_out_proj_w4(x, a.w.to(DEV), a.scale.to(DEV), group=32, dims=dims) for a in ws]
    assert not torch.equal(*want)
    y = [torch.empty_like(want[0]) for _ in range(8)]

    def calls():
        for i, out in enumerate(y):
            binding.gist_pages_copy(codes, None, src[i % 2], src[2], dims=cd)
            binding.gist_pages_copy(scales, None, src[i % 2], src[2], dims=sd)
            binding.gist_out_proj_w4(x, w, s, out, group=32, dims=dims)

    g = torch.cuda.CUDAGraph()
    calls()
    with torch.cuda.graph(g):
        calls()
    for again in (calls, g.replay):
        for _ in range(20):
            for out in y:
                out.zero_()
            again()
            assert all(torch.equal(out, want[i % 2]) for i, out in enumerate(y))
