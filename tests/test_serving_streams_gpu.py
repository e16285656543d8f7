"""The single-token step's calls one right behind another, on other streams than the current one,
captured, and from several threads."""
from __future__ import annotations

import threading

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


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def page_dims(nb, L, Hkv, bl, d, B=1, W=1):
    return dict(num_requests=B, num_tokens=B, max_new=1, num_q_heads=Hkv, num_kv_heads=Hkv, head_dim=d, block_len=bl, max_blocks=W,
                num_blocks=nb, num_layers=L, layer=0, rope_theta=1e4, softmax_scale=0.0)


@pytest.mark.parametrize("bl,L", [(16, 1), (256, 12)])
def test_copies_that_depend_on_each_other(bl, L):
    """Each call reads what the one before it wrote, small and large ones, nothing waited for."""
    nb, Hkv, d = 40, 4, 64
    pool = torch.zeros((nb, L, 2, Hkv, bl, d), dtype=torch.bfloat16, device=DEV)
    dims, ids = page_dims(nb, L, Hkv, bl, d), i32(range(nb))
    for turn in range(5):
        pool[0] = torch.randn(pool[0].shape, device=DEV)
        for i in range(nb - 1):
            binding.gist_pages_copy(pool, None, ids[i:i + 1], ids[i + 1:i + 2], dims=dims)
        assert torch.equal(pool[nb - 1], pool[0])


def test_tables_and_copies_in_a_row():
    """Free list, fork, copy, compaction, copy: each takes what the one before left on the device."""
    rng = np.random.default_rng(0)
    B, W, bl, nb, L, Hkv, d = 24, 5, 16, 260, 1, 2, 64
    dims = page_dims(nb, L, Hkv, bl, d, B, W)
    for turn in range(20):
        cached = np.concatenate([rng.integers(1, W * bl + 1, 8), np.zeros(16, np.int64)])
        table = np.full((B, W), -1)
        table[:8] = rng.permutation(nb)[:8 * W].reshape(8, W)
        parent = np.concatenate([np.full(8, -1), rng.integers(0, 8, 16)])
        pool = torch.randn((nb, L, 2, Hkv, bl, d), device=DEV).to(torch.bfloat16)
        before = pool.clone()
        lens, t, par = i32(cached), i32(table), i32(parent)
        f = binding.gist_pages_free(lens, t, dims=dims)
        k = binding.gist_pages_fork(lens, par, t, f.free_blocks, f.free_range, dims=dims)
        binding.gist_pages_copy(pool, None, k.copy_src, k.copy_dst, k.copy_rows, k.num_copies, dims=dims)
        c = binding.gist_pages_compact(k.cached_len, t, dims=dims)
        binding.gist_pages_copy(pool, None, c.copy_src, c.copy_dst, None, c.num_copies, dims=dims)
        out = c.block_table.cpu().numpy()
        for r in range(B):
            p = parent[r] if r >= 8 else r
            n, ids = int(cached[p]), torch.tensor(table[p, :-(-int(cached[p]) // bl)], device=DEV)
            want = before[ids].permute(1, 2, 3, 0, 4, 5).reshape(L, 2, Hkv, -1, d)[:, :, :, :n]
            got = pool[torch.tensor(out[r, :len(ids)], device=DEV)].permute(1, 2, 3, 0, 4, 5).reshape(L, 2, Hkv, -1, d)[:, :, :, :n]
            assert torch.equal(want, got)


def test_attention_right_behind_what_writes_its_cache():
    """Lengths, table and keys written by the call before, which another call follows at once."""
    pb = su.Decode([600, 40, 3000], 8, 2, 64, 16, seed=1)
    q, pool, table, kv = pb.args()
    nb = pb.dims["num_blocks"]
    far = torch.cat([torch.full_like(pool, float("nan")), pool])  # the cache, one pool on
    dims = dict(pb.dims, num_blocks=2 * nb)
    want = binding.gist_attn_paged_decode(q, pool, table, kv, dims=pb.dims)
    src, dst = i32(range(nb, 2 * nb)), i32(range(nb))
    ws = torch.empty(binding.paged_decode_workspace_bytes(dims), dtype=torch.uint8, device=DEV)
    out = torch.empty_like(q)
    for _ in range(20):
        far[:nb] = float("nan")
        out.zero_()
        binding.gist_pages_copy(far, None, src, dst, dims=dims)
        binding.gist_attn_paged_decode(q, far, table, kv, None, out, ws, dims=dims)
        assert torch.equal(out, want)


@pytest.mark.parametrize("T", [1, 12, 40, 64, 100])
def test_projections_in_a_row(T):
    """y1 = x w1, y2 = y1 w2, ...: each reads the one before's result; eagerly and captured."""
    d = 256
    dims = dict(page_dims(1, 1, 4, 16, 64, T), num_q_heads=4, num_kv_heads=1)
    ws = [su.W4(d, d, 32, seed=s) for s in range(6)]
    dev = [(w.w.to(DEV), w.scale.to(DEV)) for w in ws]
    x = su.bf16(np.random.default_rng(T).standard_normal((T, d))).to(DEV)
    bufs = [torch.zeros((T, d), dtype=torch.bfloat16, device=DEV) for _ in ws]

    def chain():
        at = x
        for (w, s), y in zip(dev, bufs):
            binding.gist_out_proj_w4(at, w, s, y, group=32, dims=dims)
            at = y

    chain()
    want = [b.clone() for b in bufs]
    at = x
    for (w, s), b in zip(dev, want):  # one at a time
        torch.cuda.synchronize()
        assert torch.equal(binding.gist_out_proj_w4(at, w, s, group=32, dims=dims), b)
        torch.cuda.synchronize()
        at = b
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        chain()
    for _ in range(10):
        for b in bufs:
            b.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(bufs, want))


@pytest.mark.parametrize("kind", ["stream", "handle"])
def test_what_a_call_allocates_belongs_to_its_stream(kind, monkeypatch):
    pb = su.Decode([300, 20], 8, 2, 64, 16, seed=2)
    q, pool, table, kv = pb.args()
    d = dict(pb.dims, num_q_heads=8)
    w = su.W4((8 + 4) * 64, 128, 32)
    wo = su.W4(64, 512, 32)
    x, ww, wsc = torch.zeros((2, 128), dtype=torch.bfloat16, device=DEV), w.w.to(DEV), w.scale.to(DEV)
    wo_w, wo_s = wo.w.to(DEV), wo.scale.to(DEV)
    s = torch.cuda.Stream()
    given = s if kind == "stream" else s.cuda_stream
    seen = []
    for name in ("empty", "empty_like"):
        def alloc(*a, _f=getattr(torch, name), **kw):
            seen.append(torch.cuda.current_stream().cuda_stream)
            return _f(*a, **kw)
        monkeypatch.setattr(torch, name, alloc)
    torch.cuda.synchronize()
    binding.gist_attn_paged_decode(q, pool, table, kv, dims=d, stream=given)
    f = binding.gist_pages_free(kv, table, dims=d, stream=given)
    binding.gist_pages_compact(kv, table, dims=d, stream=given)
    binding.gist_pages_fork(kv, kv.new_full((2,), -1), table, f.free_blocks, f.free_range, dims=d, stream=given)
    binding.gist_qkv_rope_w4(x, ww, wsc, kv, group=32, dims=d, stream=given)
    binding.gist_out_proj_w4(q, wo_w, wo_s, group=32, dims=d, stream=given)
    assert seen == [s.cuda_stream] * (2 + 3 + 7 + 6 + 3 + 1)
    s.synchronize()


def test_strided_and_short_tensors_are_refused():
    pb = su.Decode([300, 20], 8, 2, 64, 16, seed=2)
    q, pool, table, kv = pb.args()
    with pytest.raises(TypeError, match="contiguous"):
        binding.gist_attn_paged_decode(q.transpose(1, 2).contiguous().transpose(1, 2), pool, table, kv, dims=pb.dims)
    with pytest.raises(ValueError, match="kv_len"):
        binding.gist_attn_paged_decode(q, pool, table, kv[:1], dims=pb.dims)
    with pytest.raises(ValueError, match="kv_pool"):
        binding.gist_attn_paged_decode(q, pool[:-1], table, kv, dims=pb.dims)
    with pytest.raises(TypeError, match="kv_pool"):
        binding.gist_attn_paged_decode(q, pool.half(), table, kv, dims=pb.dims)
    with pytest.raises(TypeError, match="kv_pool"):
        binding.gist_pages_copy(pool.half(), None, kv, kv, dims=pb.dims)
    with pytest.raises(ValueError, match="kv_scale"):
        binding.gist_pages_copy(pool, torch.zeros(3, device=DEV), kv, kv, dims=pb.dims)
    with pytest.raises(ValueError, match="copy_dst"):
        binding.gist_pages_copy(pool, None, kv, kv[:1], dims=pb.dims)
    with pytest.raises(ValueError, match="free_blocks"):
        binding.gist_pages_free(kv, table, [i32([0] * n) for n in (pb.dims["num_blocks"], 1, 2)], dims=pb.dims)
    w = su.W4((8 + 4) * 64, 128, 32)
    with pytest.raises(ValueError, match="w_scale"):
        binding.gist_qkv_rope_w4(torch.zeros((2, 128), dtype=torch.bfloat16, device=DEV), w.w.to(DEV), w.scale.to(DEV)[:, :-1].contiguous(), kv,
                                 group=32, dims=pb.dims)
    with pytest.raises(ValueError, match="group"):
        binding.gist_out_proj_w4(q, w.w.to(DEV), w.scale.to(DEV), group=48, dims=pb.dims)


def test_calls_from_threads_of_unlike_sizes():
    """Projections on both kernels, tables and forks from four threads at once."""
    jobs, failed = [], []
    for T, K in ((3, 8192), (40, 1024)):
        w = su.W4(256, K, 64, seed=T)
        x = su.bf16(np.random.default_rng(T).standard_normal((T, K // 64, 64))).to(DEV)
        a = (x, w.w.to(DEV), w.scale.to(DEV))
        dims = dict(page_dims(1, 1, 1, 16, 64, T), num_q_heads=K // 64)
        jobs.append(lambda s, a=a, dims=dims: binding.gist_out_proj_w4(*a, group=64, dims=dims, stream=s))
    for B in (16384, 40):
        dims = page_dims(3 * B, 1, 1, 16, 64, B, 2)
        lens = i32(np.random.default_rng(B).integers(0, 33, B))
        par = i32(np.where(np.arange(B) % 2, np.arange(B) - 1, -1))
        free = i32(range(2 * B, 3 * B))
        tab = i32(np.arange(2 * B).reshape(B, 2))

        def job(s, dims=dims, lens=lens, par=par, free=free, tab=tab, span=i32([0, B])):
            with torch.cuda.stream(s):
                t = tab.clone()
            f = binding.gist_pages_fork(lens, par, t, free, span, dims=dims, stream=s)
            c = binding.gist_pages_compact(f.cached_len, t, dims=dims, stream=s)
            with torch.cuda.stream(s):
                return torch.cat([t.view(-1), f.cached_len, c.block_table.view(-1), c.new_id])
        jobs.append(job)
    here = torch.cuda.current_stream()
    want = [j(here).clone() for j in jobs]
    torch.cuda.synchronize()

    def calls(i):
        try:
            s = torch.cuda.Stream()
            for _ in range(60):
                got = jobs[i](s)
                s.synchronize()
                assert torch.equal(got, want[i])
        except Exception as e:  # noqa: BLE001 - reported by the test's own thread
            failed.append((i, e))

    threads = [threading.Thread(target=calls, args=(i,)) for i in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
