"""A decoding layer as a server runs it (projection, plan, append, attention, projection; forks and a
compaction between steps), each stage against its definition in 64 bits on what the stage before
left on the device, and the cache bit for bit."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import serving_utils as su
from attention_cached_kv_gb300 import binding

DEV = "cuda"
Hq, Hkv, d, D, bl, W, nb, group = 14, 2, 64, 896, 16, 6, 60, 32
B = 6


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def weights():
    return su.W4((Hq + 2 * Hkv) * d, D, group, seed=1), su.W4(D, Hq * d, group, seed=2)


def check_projection(w, x, position, q, k, v):
    """q, k, v [n][heads][d] of tokens x [n][D]."""
    n = len(x)
    y, off = (a.reshape(n, -1, d) for a in w.times(x))
    yr, offr = su.rotated(y[:, :Hq + Hkv], off[:, :Hq + Hkv], position)
    mag = np.abs(y[:, :Hq + Hkv])  # a position t is t theta_j / 2 pi turns to 2^-53 t and 2^-32 turns
    offr = offr + (2.0 ** -31 + position[:, None, None] * 2.0 ** -52) * 2 * np.pi * (mag + np.roll(mag, d // 2, -1))
    su.near(q, yr[:, :Hq], offr[:, :Hq] + su.BF16 * 1.01 * np.abs(yr[:, :Hq]), "q")
    su.near(k, yr[:, Hq:], offr[:, Hq:] + su.BF16 * 1.01 * np.abs(yr[:, Hq:]), "k")
    su.near(v, y[:, Hq + Hkv:], off[:, Hq + Hkv:] + su.BF16 * 1.01 * np.abs(y[:, Hq + Hkv:]), "v")


@pytest.mark.parametrize("C", [2, 21, 27, 33])
def test_the_attention_bound_notices_any_one_key(C):
    """On the CPU: leaving out a key, or seeing the one before it twice, passes the bound that the layer is
    held to."""
    rng = np.random.default_rng(C)
    wq, _ = weights()
    y = wq.times(rng.standard_normal((C, D)))[0].reshape(C, -1, d)
    pos = np.arange(C)
    q = su.bf16(su.rotate(y[-1:, :Hq], pos[-1:])).double().numpy()
    kv = [su.bf16(a).double().numpy() for a in (su.rotate(y[:, Hq:Hq + Hkv], pos), y[:, Hq + Hkv:])]

    def attend(rows):
        n = -(-len(rows) // bl)
        pool = np.zeros((n, 2, Hkv, bl, d))
        for j, r in enumerate(rows):
            for i in (0, 1):
                pool[j // bl, i, :, j % bl] = kv[i][r]
        return su.attend(q, pool, np.arange(n)[None], [len(rows)], bl, Hq // Hkv, rotated=True)

    ref, tol = attend(list(range(C)))
    for j in range(C):
        for rows in ([r for r in range(C) if r != j], [r if r != j else (j or C) - 1 for r in range(C)]):
            assert (np.abs(attend(rows)[0] - ref) > 4 * tol).any(), j


@pytest.mark.gpu
def test_a_layer_stage_by_stage():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    dims = dict(num_requests=B, num_tokens=B, max_new=1, num_q_heads=Hq, num_kv_heads=Hkv, head_dim=d, block_len=bl, max_blocks=W,
                num_blocks=nb, num_layers=2, layer=1, rope_theta=1e4, softmax_scale=0.0, flags=binding.FLAG_PREROTATED)
    pair = dict(num_pairs=B, n_new=1, num_q_heads=Hq, num_kv_heads=Hkv, head_dim=d, block_len=bl, blocks_per_pair=W, num_blocks=nb,
                num_layers=2, layer=1, rope_theta=1e4, softmax_scale=0.0, flags=binding.FLAG_PREROTATED)
    wq, wo = weights()
    dev = [t.to(DEV) for t in (wq.w, wq.scale, wo.w, wo.scale)]
    pool = torch.full((nb, 2, 2, Hkv, bl, d), float("nan"), dtype=torch.bfloat16, device=DEV)
    table = torch.full((B, W), -1, dtype=torch.int32, device=DEV)
    cached, new = torch.zeros(B, dtype=torch.int32, device=DEV), i32([1, 1, 0, 1, 0, 0])
    f = binding.gist_pages_free(cached, table, dims=dims)
    free, span = f.free_blocks, f.free_range
    x = torch.zeros((B, D), dtype=torch.bfloat16, device=DEV)
    plan = [torch.zeros(n, dtype=torch.int32, device=DEV) for n in (B + 1, B, B, B, 2)]
    q = torch.zeros((B, Hq, d), dtype=torch.bfloat16, device=DEV)
    k, v = (torch.zeros((B, Hkv, d), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    attn, y = torch.zeros_like(q), torch.zeros_like(x)
    ws = torch.empty(binding.paged_decode_workspace_bytes(dims), dtype=torch.uint8, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)

    def step():
        p = binding.gist_paged_plan(cached, new, table, free, span, plan, dims=dims, status=status)
        binding.gist_qkv_rope_w4(x, dev[0], dev[1], p.position, q, k, v, group=group, dims=dims, status=status)
        # the append takes a token a request: request r's is row q_start[r] (a slot of -1 has none)
        at = p.q_start[:-1].long().clamp(max=B - 1)
        slot = torch.where(new > 0, p.position[at], torch.full_like(new, -1))
        binding.gist_kv_append(k[at][:, None].contiguous(), v[at][:, None].contiguous(), pool, table, slot, dims=pair)
        binding.gist_attn_paged_decode(q, pool, table, p.kv_len, p.q_start, attn, ws, dims=dims, status=status)
        binding.gist_out_proj_w4(attn, dev[2], dev[3], y, group=group, dims=dims, status=status)
        cached.copy_(p.kv_len)
        span.copy_(p.free_range)

    history = [[] for _ in range(B)]  # of each request: the k and v of its tokens, as the projection left them

    def check(live):
        torch.cuda.synchronize()
        assert int(status) == 0
        n, lens = len(live), [len(history[r]) + 1 for r in live]
        assert [int(c) for c in cached[live]] == lens and [int(s) for s in plan[0]][-1] == n
        xs, pos = x[:n].cpu().double().numpy(), np.array(lens) - 1
        check_projection(wq, xs, pos, q[:n], k[:n], v[:n])
        for i, r in enumerate(live):
            history[r].append(torch.stack([k[i], v[i]]).clone())  # [2][Hkv][d]
        tab = table.cpu().numpy()
        for r in range(B):  # the cache, bit for bit, of requests without a token too
            if history[r]:
                want = torch.stack(history[r], 2)
                ids = torch.tensor(tab[r, :-(-len(history[r]) // bl)].astype(np.int64), device=DEV)
                got = pool[ids, 1].permute(1, 2, 0, 3, 4).reshape(2, Hkv, -1, d)[:, :, :len(history[r])]
                assert torch.equal(got, want), r
        su.near(attn[:n], *su.attend(q[:n].cpu().double().numpy(), pool[:, 1].cpu().double().numpy(), tab[live], lens, bl, Hq // Hkv,
                                     rotated=True), "attention")
        ref, off = wo.times(attn[:n].cpu().double().numpy().reshape(n, -1))
        su.near(y[:n], ref, off + su.BF16 * 1.01 * np.abs(ref), "output")

    g = torch.Generator(device=DEV).manual_seed(0)
    step()  # outside the capture, then undone: the cache is empty again
    cached.zero_()
    table.fill_(-1)
    span.copy_(i32([0, nb]))
    pool.fill_(float("nan"))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    x.zero_()  # (a graph's capture runs nothing)

    def run(live, steps):
        for _ in range(steps):
            x.copy_(torch.randn((B, D), generator=g, device=DEV))
            graph.replay()
            check(live)

    run([0, 1, 3], 21)
    for kids, steps in (([2, 4, 5], 9), ([2, 5, 1], 20)):
        # rows `kids` go on from rows 0, 3 and 0; all run; two end, the others are moved together
        parent = np.full(B, -1)
        parent[kids] = [0, 3, 0]
        fk = binding.gist_pages_fork(cached, i32(parent), table, free, span, dims=dims, status=status)
        binding.gist_pages_copy(pool, None, fk.copy_src, fk.copy_dst, fk.copy_rows, fk.num_copies, dims=dims, status=status)
        cached.copy_(fk.cached_len)
        span.copy_(fk.free_range)
        for r in kids:
            history[r] = list(history[parent[r]])
        live = [r for r in range(B) if history[r]]
        new.copy_(i32([int(r in live) for r in range(B)]))
        run(live, steps)
        live = [r for r in live if r not in (1, 5)]
        cached[[1, 5]] = 0
        history[1], history[5] = [], []
        new.copy_(i32([int(r in live) for r in range(B)]))
        c = binding.gist_pages_compact(cached, table, dims=dims, status=status)
        binding.gist_pages_copy(pool, None, c.copy_src, c.copy_dst, None, c.num_copies, dims=dims, status=status)
        table.copy_(c.block_table)
        free.copy_(c.free_blocks)
        span.copy_(c.free_range)
        run(live, 4)
        new.copy_(i32([0, 0, 0, 1, 0, 0]))  # one alone, the others keep theirs
        run([3], 2)
        new.copy_(i32([int(r in live) for r in range(B)]))
