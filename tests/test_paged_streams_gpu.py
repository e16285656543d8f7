"""The ragged serving step's entry points from several threads and on other streams
than the current one."""
from __future__ import annotations

import threading

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


STREAMS = ["stream", "handle"]


def problem():
    pb = pu.Problem([3000, 700, 20], [1, 40, 3], 8, 2, 64, 16, seed=1)
    return pb, pb.args()


@pytest.mark.parametrize("kind", STREAMS)
def test_what_a_call_allocates_belongs_to_its_stream(kind, monkeypatch):
    """Workspace, output and plan buffers come from the memory of the stream that the call
    runs on, so that no other stream's work can still be using them, or get them while
    the call runs."""
    pb, args = problem()
    s = torch.cuda.Stream()
    given = s if kind == "stream" else s.cuda_stream
    seen = []
    for name in ("empty", "empty_like"):
        def alloc(*a, _f=getattr(torch, name), **kw):
            seen.append(torch.cuda.current_stream().cuda_stream)
            return _f(*a, **kw)
        monkeypatch.setattr(torch, name, alloc)
    torch.cuda.synchronize()
    binding.gist_attn_paged_fp8kv(*args, dims=pb.dims, stream=given)
    assert seen == [s.cuda_stream] * 2
    i = pb.i32([0, 5])
    dims = dict(pb.dims, num_requests=1, num_tokens=4)
    binding.gist_paged_plan(i[:1], i[1:], pb.i32(pb.table), i, pb.i32([0, 0]), dims=dims, stream=given)
    assert seen == [s.cuda_stream] * 7
    torch.cuda.synchronize()


@pytest.mark.parametrize("kind", STREAMS)
def test_memory_that_other_streams_use_is_not_taken(kind):
    """Calls on two streams without workspaces, the memory between them freed and used
    again on the current one: every answer is the one of a call alone."""
    pb, args = problem()
    want = binding.gist_attn_paged_fp8kv(*args, dims=pb.dims)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    need = binding.paged_workspace_bytes(pb.dims)
    outs = []
    for i in range(20):
        here = torch.zeros(need, dtype=torch.uint8, device=DEV)  # current stream: work on memory of that size,
        here.fill_(0x7F)
        del here                                                   # then free while the work may be under way
        s = streams[i % 2]
        outs.append(binding.gist_attn_paged_fp8kv(*args, dims=pb.dims, stream=s if kind == "stream" else s.cuda_stream))
        outs.append(binding.gist_attn_paged_fp8kv(*args, dims=pb.dims))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


def test_a_raw_handle_of_the_default_stream():
    pb, args = problem()
    want = binding.gist_attn_paged_fp8kv(*args, dims=pb.dims)
    got = binding.gist_attn_paged_fp8kv(*args, dims=pb.dims, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("kind", STREAMS)
def test_outputs_of_the_other_calls_belong_to_their_stream(kind, monkeypatch):
    """Attention over bf16 and E4M3 pools, block mass, gather and projections."""
    P, Hq, Hkv, d, bl, nblk = 2, 4, 2, 64, 16, 9
    dims = dict(num_pairs=P, n_new=1, num_q_heads=Hq, num_kv_heads=Hkv, head_dim=d, block_len=bl, blocks_per_pair=nblk,
                num_blocks=P * nblk, num_layers=1, layer=0, rope_theta=1e4, softmax_scale=0.0, flags=0)
    bf = dict(dtype=torch.bfloat16, device=DEV)
    q, k, v = (torch.randn((P, 1, h, d), **bf) for h in (Hq, Hkv, Hkv))
    pool = torch.randn((P * nblk, 1, 2, Hkv, bl, d), **bf)
    codes, scale = pool.to(torch.float8_e4m3fn), torch.ones((P * nblk, 1, 2, Hkv), device=DEV)
    table = torch.arange(P * nblk, dtype=torch.int32, device=DEV).view(P, nblk)
    rows = dict(dims, num_pairs=3, n_new=64, num_q_heads=14, block_len=8, blocks_per_pair=1, num_blocks=1)
    x, w = torch.randn((3, 64, 256), **bf), torch.randn(((14 + 2 * Hkv) * d, 256), **bf)
    wo, attn = torch.randn((256, 14 * d), **bf), torch.randn((3, 64, 14, d), **bf)
    s = torch.cuda.Stream()
    given = s if kind == "stream" else s.cuda_stream
    calls = [lambda **kw: binding.gist_attn_fwd(q, k, v, pool, None, table, dims=dims, **kw),
             lambda **kw: binding.gist_attn_fwd_fp8kv(q, k, v, codes, scale, None, table, dims=dims, **kw),
             lambda **kw: binding.gist_attn_fwd_block_mass(q, k, v, pool, table, dims=dims, **kw),
             lambda **kw: binding.gist_attn_gather_debug(pool, None, table, dims=dims, **kw),
             lambda **kw: binding.gist_qkv_rope(x, w, dims=rows, **kw),
             lambda **kw: binding.gist_out_proj(attn, wo, dims=rows, **kw)]
    want = [call() for call in calls]
    torch.cuda.synchronize()
    seen = []
    for name in ("empty", "empty_like"):
        def alloc(*a, _f=getattr(torch, name), **kw):
            seen.append(torch.cuda.current_stream().cuda_stream)
            return _f(*a, **kw)
        monkeypatch.setattr(torch, name, alloc)
    got = [call(stream=given) for call in calls]
    torch.cuda.synchronize()
    assert seen == [s.cuda_stream] * 9
    flat = lambda xs: [t for x in xs for t in (x if isinstance(x, tuple) else (x,))]  # noqa: E731
    assert all(torch.equal(a, b) for a, b in zip(flat(got), flat(want)))
