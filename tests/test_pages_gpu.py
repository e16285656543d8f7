"""The blocks of a paged cache between steps against loops over requests and entries: free
lists, renaming, forks, and the copies, all bit for bit."""
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


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def make(B, W, bl, nb, seed, most=None):
    """Tables with shared prefixes, ended requests, and entries past the live ones."""
    rng = np.random.default_rng(seed)
    cached = rng.integers(0, W * bl + 1 if most is None else most + 1, B)
    cached[rng.random(B) < 0.2] = 0
    table = rng.integers(-3, nb + 3, (B, W))
    perm, at = rng.permutation(nb), 0
    for r in range(B):
        n = su.blocks(cached[r], bl, W)
        share = min(n, su.blocks(cached[r - 1], bl, W)) // 2 if r % 2 else 0
        table[r, :share] = table[r - 1, :share]
        for j in range(share, n):
            table[r, j] = perm[at % nb]
            at += 1
    dims = dict(num_requests=B, num_tokens=B, max_new=1, num_q_heads=2, num_kv_heads=2, head_dim=64, block_len=bl, max_blocks=W,
                num_blocks=nb, num_layers=2, layer=0, rope_theta=1e4, softmax_scale=0.0)
    return cached, table, dims


SIZES = [(1, 1, 16, 1), (1, 1, 16, 2), (3, 5, 1, 7), (40, 9, 16, 300), (5, 700, 3, 5000), (700, 3, 64, 2500), (0, 4, 16, 33),
         (17, 130, 16, 2049), (300, 40, 256, 20000)]


@pytest.mark.parametrize("B,W,bl,nb", SIZES)
def test_free(B, W, bl, nb):
    cached, table, dims = make(B, W, bl, nb, B + W)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = binding.gist_pages_free(i32(cached), i32(table), dims=dims, status=status)
    want = su.free(cached, table, bl, nb)
    su.same(got._asdict(), want)
    assert int(status) == want["status"]


@pytest.mark.parametrize("B,W,bl,nb", SIZES)
@pytest.mark.parametrize("in_place", [False, True])
def test_compact(B, W, bl, nb, in_place):
    cached, table, dims = make(B, W, bl, nb, B + W, most=max(1, W * bl // 2))
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    t = i32(table)
    out = None
    if in_place:
        out = [t] + [torch.full((n,), 99, dtype=torch.int32, device=DEV) for n in (nb, nb // 2, nb // 2, 1, nb, 2)]
    got = binding.gist_pages_compact(i32(cached), t, out, dims=dims, status=status)
    want = su.compact(cached, table, bl, nb)
    su.same(got._asdict(), want)
    assert int(status) == want["status"]


def test_full_and_empty_pools():
    for cached in ([64, 64], [0, 0]):
        table = np.arange(8).reshape(2, 4)[:, ::-1].copy()
        _, _, dims = make(2, 4, 16, 8, 0)
        for call, want in ((binding.gist_pages_free, su.free), (binding.gist_pages_compact, su.compact)):
            su.same(call(i32(cached), i32(table), dims=dims)._asdict(), want(cached, table, 16, 8))


def test_bad_entries_and_lengths():
    cached, table, dims = make(30, 6, 16, 200, 4)
    cached[3], cached[4], cached[5] = 6 * 16 + 1, 2 ** 31 - 1, -(2 ** 31)
    table[6, 0], table[7, 1] = -1, 200
    cached[6], cached[7] = 50, 50
    for call, want in ((binding.gist_pages_free, su.free), (binding.gist_pages_compact, su.compact)):
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        su.same(call(i32(cached), i32(table), dims=dims, status=status)._asdict(), want(cached, table, 16, 200))
        assert int(status) == binding.STATUS_BAD_BLOCK


@pytest.mark.parametrize("B,W,bl", [(1, 1, 16), (8, 3, 16), (50, 40, 16), (4000, 3, 64), (16384, 2, 1), (33, 300, 7)])
@pytest.mark.parametrize("short", [False, True])
def test_fork(B, W, bl, short):
    nb = 2 * B * W + 8
    rng = np.random.default_rng(B)
    cached, table, dims = make(B, W, bl, nb, B)
    parent = np.where(rng.random(B) < 0.5, -1, rng.integers(0, B, B))
    parent[:1] = -1
    if B > 4:
        parent[2], parent[3] = 3, 3      # of itself: unchanged, and 2 its fork
        parent[4] = B + 5                # no such row
    free = rng.permutation(nb)
    rng_ = [3, 3 + (2 if short else B)]
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    t = i32(table)
    out = [torch.full((n,), 99, dtype=torch.int32, device=DEV) for n in (B, B, B, B, 1, 2)]
    got = binding.gist_pages_fork(i32(cached), i32(parent), t, i32(free), i32(rng_), out, dims=dims, status=status)
    want = su.fork(cached, parent, table, free, rng_, bl, nb)
    su.same(got._asdict() | {"block_table": t}, want)
    assert int(status) == want["status"]


def test_fork_of_bad_blocks_and_lengths():
    cached, table, dims = make(10, 4, 16, 50, 2)
    cached[:5] = [20, 20, 65, -3, 64]
    table[0, 1], table[4] = 50, [4, 3, 2, 1]
    parent = np.array([-1] * 5 + [0, 1, 2, 3, 4])
    for free, rng_ in (([7, 8, 9], [0, 3]), ([7, -1, 9], [-4, 9]), ([], [0, 0])):
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        t = i32(table)
        got = binding.gist_pages_fork(i32(cached), i32(parent), t, i32(free), i32(rng_), dims=dims, status=status)
        want = su.fork(cached, parent, table, free, rng_, 16, 50)
        su.same(got._asdict() | {"block_table": t}, want)
        assert int(status) == want["status"]


def pools(nb, L, Hkv, bl, d, fp8, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    shape = (nb, L, 2, Hkv, bl, d)
    if fp8:
        return (torch.randint(0, 256, shape, generator=g, device=DEV, dtype=torch.uint8),
                torch.randn(shape[:4], generator=g, device=DEV))
    return torch.randn(shape, generator=g, device=DEV).to(torch.bfloat16), None


@pytest.mark.parametrize("L,Hkv,bl,d", [(1, 1, 1, 64), (3, 2, 16, 64), (2, 5, 7, 128), (2, 8, 256, 128), (1, 3, 33, 64)])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n", [1, 9, 60])
def test_copy(L, Hkv, bl, d, fp8, n):
    nb = 2 * n + 3
    pool, scale = pools(nb, L, Hkv, bl, d, fp8)
    rng = np.random.default_rng(n)
    ids = rng.permutation(nb)
    src, dst = ids[:n], ids[n:2 * n]
    rows = rng.integers(0, bl + 1, n)
    dims = dict(num_requests=1, num_tokens=1, max_new=1, num_q_heads=Hkv, num_kv_heads=Hkv, head_dim=d, block_len=bl, max_blocks=1,
                num_blocks=nb, num_layers=L, layer=0, rope_theta=1e4, softmax_scale=0.0)
    for given in (None, rows):
        for count in (None, n // 2, n, n + 5, -1):
            p, s = pool.clone(), None if scale is None else scale.clone()
            status = torch.zeros(1, dtype=torch.int32, device=DEV)
            binding.gist_pages_copy(p, s, i32(src), i32(dst), None if given is None else i32(given),
                                    None if count is None else i32([count]), dims=dims, status=status)
            want, ws = pool.clone(), None if scale is None else scale.clone()
            for i in range(n if count is None else max(0, min(count, n))):
                k = bl if given is None else int(given[i])
                want[dst[i], :, :, :, :k] = pool[src[i], :, :, :, :k]
                if ws is not None:
                    ws[dst[i]] = scale[src[i]]
            assert torch.equal(p.view(torch.uint8), want.view(torch.uint8)) and int(status) == 0
            assert s is None or torch.equal(s, ws)


def test_copy_passes_over_what_is_not_there():
    nb = 12
    pool, scale = pools(nb, 2, 2, 16, 64, True)
    dims = dict(num_requests=1, num_tokens=1, max_new=1, num_q_heads=2, num_kv_heads=2, head_dim=64, block_len=16, max_blocks=1,
                num_blocks=nb, num_layers=2, layer=0, rope_theta=1e4, softmax_scale=0.0)
    good = ([0, -1, 4, 6, 1], [5, 7, -9, 6, 2])
    want = pool.clone()
    want[5], want[2] = pool[0], pool[1]
    for more, rows, bits in (([], [16] * 5, 0), ([(nb, 8)], [16] * 6, 1), ([(3, nb)], [16] * 6, 1), ([(3, 9)], [16] * 5 + [17], 1),
                             ([(3, 9)], [16] * 5 + [-1], 1), ([(2 ** 31 - 1, 8)], [16] * 6, 1)):
        p, s, status = pool.clone(), scale.clone(), torch.zeros(1, dtype=torch.int32, device=DEV)
        src, dst = good[0] + [a for a, _ in more], good[1] + [b for _, b in more]
        binding.gist_pages_copy(p, s, i32(src), i32(dst), i32(rows), dims=dims, status=status)
        assert torch.equal(p, want) and int(status) == bits


def test_copy_past_4_gib_and_of_a_float8_pool():
    L, Hkv, bl, d = 4, 8, 256, 128
    nb = (9 << 29) // (L * 2 * Hkv * bl * d)
    pool = torch.zeros((nb, L, 2, Hkv, bl, d), dtype=torch.uint8, device=DEV)
    pool[2] = torch.randint(0, 256, pool[2].shape, dtype=torch.uint8, device=DEV)
    pool[nb - 1] = torch.randint(0, 256, pool[2].shape, dtype=torch.uint8, device=DEV)
    dims = dict(num_requests=1, num_tokens=1, max_new=1, num_q_heads=8, num_kv_heads=Hkv, head_dim=d, block_len=bl, max_blocks=1,
                num_blocks=nb, num_layers=L, layer=0, rope_theta=1e4, softmax_scale=0.0)
    binding.gist_pages_copy(pool.view(torch.float8_e4m3fn), None, i32([2, nb - 1]), i32([nb - 2, 5]), i32([bl, 100]), dims=dims)
    assert torch.equal(pool[nb - 2], pool[2])
    assert torch.equal(pool[5, :, :, :, :100], pool[nb - 1, :, :, :, :100]) and not pool[5, :, :, :, 100:].any()
    assert not pool[3].any() and not pool[nb - 3].any()


def test_a_fork_and_a_compaction_keep_what_requests_see():
    """Fork, copy, end some requests, compact, copy: every request's rows are the same bits."""
    rng = np.random.default_rng(3)
    L, Hkv, bl, d, B, W, nb = 2, 2, 16, 64, 12, 6, 90
    pool, scale = pools(nb, L, Hkv, bl, d, True)
    cached = np.concatenate([rng.integers(1, W * bl, 4), np.zeros(8, np.int64)])
    table, perm = np.full((B, W), -1), rng.permutation(nb)
    for r in range(4):
        table[r] = perm[6 * r:6 * r + 6]
    parent = np.array([-1] * 4 + [0, 0, 0, 1, 1, 2, 3, 3])
    dims = dict(num_requests=B, num_tokens=B, max_new=1, num_q_heads=2, num_kv_heads=Hkv, head_dim=d, block_len=bl, max_blocks=W,
                num_blocks=nb, num_layers=L, layer=0, rope_theta=1e4, softmax_scale=0.0)

    def seen(r, length, tab):
        ids = tab[r, :-(-length // bl)].long()
        return (pool[ids].permute(1, 2, 3, 0, 4, 5).reshape(L, 2, Hkv, -1, d)[:, :, :, :length].clone(), scale[ids].clone())

    t = i32(table)
    before = {r: seen(parent[r] if parent[r] >= 0 else r, int(cached[max(parent[r], r if parent[r] < 0 else 0)]), t) for r in range(B)}
    got = binding.gist_pages_free(i32(cached), t, dims=dims)
    f = binding.gist_pages_fork(i32(cached), i32(parent), t, got.free_blocks, got.free_range, dims=dims)
    binding.gist_pages_copy(pool, scale, f.copy_src, f.copy_dst, f.copy_rows, f.num_copies, dims=dims)
    lens = f.cached_len.cpu().numpy()
    for r in range(B):
        assert all(torch.equal(a, b) for a, b in zip(before[r], seen(r, int(lens[r]), t)))
    lens[[0, 5, 8]] = 0
    c = binding.gist_pages_compact(i32(lens), t, dims=dims)
    binding.gist_pages_copy(pool, scale, c.copy_src, c.copy_dst, None, c.num_copies, dims=dims)
    for r in range(B):
        if lens[r]:
            assert all(torch.equal(a, b) for a, b in zip(before[r], seen(r, int(lens[r]), c.block_table)))
    n = nb - int(c.free_range[1])
    assert (c.block_table[torch.arange(B), 0].cpu().numpy()[lens > 0] < n).all()


def test_captured_and_on_another_stream():
    cached, table, dims = make(40, 9, 16, 300, 1)
    lens, t = i32(cached), i32(table)
    out = list(binding.gist_pages_compact(lens, t, dims=dims))
    free = list(binding.gist_pages_free(lens, t, dims=dims))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        binding.gist_pages_compact(lens, t, out, dims=dims)
        binding.gist_pages_free(lens, t, free, dims=dims)
    for seed in (5, 6):
        c2, t2, _ = make(40, 9, 16, 300, seed)
        lens.copy_(i32(c2))
        t.copy_(i32(t2))
        g.replay()
        torch.cuda.synchronize()
        su.same(binding.PagesCompact(*out)._asdict(), su.compact(c2, t2, 16, 300))
        su.same(binding.PagesFree(*free)._asdict(), su.free(c2, t2, 16, 300))
    s = torch.cuda.Stream()
    got = binding.gist_pages_free(lens, t, dims=dims, stream=s)
    s.synchronize()
    su.same(got._asdict(), su.free(c2, t2, 16, 300))
