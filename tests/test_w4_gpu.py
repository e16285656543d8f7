"""4-bit projections of few tokens against the definition in 64 bits, and a decoding layer
as a server runs it: projection, plan, append, attention, projection, with forks between."""
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


def dims_of(T, Hq, Hkv, d, **kw):
    return dict(num_requests=T, num_tokens=T, max_new=1, num_q_heads=Hq, num_kv_heads=Hkv, head_dim=d, block_len=16, max_blocks=1,
                num_blocks=1, num_layers=1, layer=0, rope_theta=1e4, softmax_scale=0.0) | kw


TOKENS = [1, 2, 7, 8, 9, 16, 17, 32, 33, 64, 65, 130]


@pytest.mark.parametrize("T", TOKENS)
@pytest.mark.parametrize("Hq,Hkv,d,K,group", [(14, 2, 64, 896, 32), (1, 1, 64, 32, 32), (4, 1, 128, 96, 32), (8, 8, 128, 1088, 64), (2, 1, 64, 4096, 128)])
def test_qkv(T, Hq, Hkv, d, K, group):
    N = (Hq + 2 * Hkv) * d
    w = su.W4(N, K, group, seed=T)
    rng = np.random.default_rng(T)
    x = su.bf16(rng.standard_normal((T, K)))
    pos = rng.integers(0, 2 ** 31 - 1, T) if T % 2 else rng.integers(0, 5000, T)
    q, k, v = binding.gist_qkv_rope_w4(x.to(DEV), w.w.to(DEV), w.scale.to(DEV), i32(pos), group=group, dims=dims_of(T, Hq, Hkv, d))
    y, off = w.times(x.double().numpy())
    y, off = y.reshape(T, -1, d), off.reshape(T, -1, d)
    yr, offr = su.rotated(y[:, :Hq + Hkv], off[:, :Hq + Hkv], pos)
    # a position t is t theta_j / 2 pi turns to 2^-53 t and 2^-32 turns
    turn = (2.0 ** -31 + pos[:, None, None] * 2.0 ** -52) * 2 * np.pi
    mag = np.abs(y[:, :Hq + Hkv])
    offr = offr + turn * (mag + np.roll(mag, d // 2, -1))
    su.near(q, yr[:, :Hq], offr[:, :Hq] + su.BF16 * 1.01 * np.abs(yr[:, :Hq]), "q")
    su.near(k, yr[:, Hq:], offr[:, Hq:] + su.BF16 * 1.01 * np.abs(yr[:, Hq:]), "k")
    su.near(v, y[:, Hq + Hkv:], off[:, Hq + Hkv:] + su.BF16 * 1.01 * np.abs(y[:, Hq + Hkv:]), "v")


@pytest.mark.parametrize("T", TOKENS)
@pytest.mark.parametrize("Hq,d,N,group", [(14, 64, 896, 128), (1, 64, 16, 32), (32, 128, 1040, 64), (3, 128, 400, 32)])
def test_out(T, Hq, d, N, group):
    w = su.W4(N, Hq * d, group, seed=T)
    x = su.bf16(np.random.default_rng(T).standard_normal((T, Hq, d)))
    y = binding.gist_out_proj_w4(x.to(DEV), w.w.to(DEV), w.scale.to(DEV), group=group, dims=dims_of(T, Hq, 1, d))
    ref, off = w.times(x.double().numpy().reshape(T, -1))
    su.near(y, ref, off + su.BF16 * 1.01 * np.abs(ref))
    again = binding.gist_out_proj_w4(x.to(DEV), w.w.to(DEV), w.scale.to(DEV), group=group, dims=dims_of(T, Hq, 1, d))
    assert torch.equal(y, again)  # sums in a fixed order


@pytest.mark.parametrize("T,Hq", [(3, 512), (40, 256), (64, 128)])
def test_long_inputs(T, Hq):
    """K of 16 k to 64 k: x is split over a cluster, the tokens over passes."""
    w = su.W4(32, Hq * 128, 128, seed=T)
    x = su.bf16(np.random.default_rng(T).standard_normal((T, Hq, 128)))
    y = binding.gist_out_proj_w4(x.to(DEV), w.w.to(DEV), w.scale.to(DEV), group=128, dims=dims_of(T, Hq, 1, 128))
    ref, off = w.times(x.double().numpy().reshape(T, -1))
    su.near(y, ref, off + su.BF16 * 1.01 * np.abs(ref))


def test_padding_rows_are_left_as_they_were():
    T, Hq, Hkv, d, K = 6, 4, 2, 64, 256
    w = su.W4((Hq + 2 * Hkv) * d, K, 64)
    x = su.bf16(np.random.default_rng(0).standard_normal((T, K)))
    pos = i32([5, -1, 0, 9, -1, -7])
    out = [torch.full((T, h, d), 3.0, dtype=torch.bfloat16, device=DEV) for h in (Hq, Hkv, Hkv)]
    got = binding.gist_qkv_rope_w4(x.to(DEV), w.w.to(DEV), w.scale.to(DEV), pos, *out, group=64, dims=dims_of(T, Hq, Hkv, d))
    for t in got:
        assert (t[[1, 4, 5]] == 3.0).all() and (t[[0, 2, 3]] != 3.0).any()


def test_values_that_are_not_finite_stay_with_their_token_or_row():
    T, N, Hq, d = 9, 64, 4, 64
    w = su.W4(N, Hq * d, 32)
    x = su.bf16(np.random.default_rng(0).standard_normal((T, Hq, d)))
    x[3, 1, 7] = float("inf")
    w.scale[17, 2] = float("nan")
    y = binding.gist_out_proj_w4(x.to(DEV), w.w.to(DEV), w.scale.to(DEV), group=32, dims=dims_of(T, Hq, 1, d)).float()
    good = torch.isfinite(y)
    assert not good[3].any() and not good[:, 17].any()
    good[3], good[:, 17] = True, True
    assert good.all()


def test_a_decoding_layer_with_forks():
    """qkv -> plan -> append -> attention -> out, five steps of three conversations from one captured
    graph; then each is forked, and the forks go on with tokens of their own."""
    Hq, Hkv, d, D, bl, W, nb, group = 14, 2, 64, 896, 16, 6, 60, 32
    B = 6
    dims = dims_of(B, Hq, Hkv, d, block_len=bl, max_blocks=W, num_blocks=nb, num_layers=2, layer=1, flags=binding.FLAG_PREROTATED)
    pair = dict(num_pairs=B, n_new=1, num_q_heads=Hq, num_kv_heads=Hkv, head_dim=d, block_len=bl, blocks_per_pair=W, num_blocks=nb,
                num_layers=2, layer=1, rope_theta=1e4, softmax_scale=0.0, flags=binding.FLAG_PREROTATED)
    wq, wo = su.W4((Hq + 2 * Hkv) * d, D, group, seed=1), su.W4(D, Hq * d, group, seed=2)
    dev = [t.to(DEV) for t in (wq.w, wq.scale, wo.w, wo.scale)]
    pool = torch.full((nb, 2, 2, Hkv, bl, d), float("nan"), dtype=torch.bfloat16, device=DEV)
    table = torch.full((B, W), -1, dtype=torch.int32, device=DEV)
    cached, new = torch.zeros(B, dtype=torch.int32, device=DEV), i32([1, 1, 1, 0, 0, 0])
    f = binding.gist_pages_free(cached, table, dims=dims)
    free, span = f.free_blocks, f.free_range
    x = torch.zeros((B, D), dtype=torch.bfloat16, device=DEV)
    plan = [torch.zeros(n, dtype=torch.int32, device=DEV) for n in (B + 1, B, B, B, 2)]
    q = torch.zeros((B, Hq, d), dtype=torch.bfloat16, device=DEV)
    k, v = (torch.zeros((B, Hkv, d), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    attn, y = torch.zeros_like(q), torch.zeros_like(x)
    ws = torch.empty(binding.paged_decode_workspace_bytes(dims), dtype=torch.uint8, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    rows = torch.zeros(B, dtype=torch.int64, device=DEV)  # token row of each request

    def step():
        p = binding.gist_paged_plan(cached, new, table, free, span, plan, dims=dims, status=status)
        binding.gist_qkv_rope_w4(x, dev[0], dev[1], p.position, q, k, v, group=group, dims=dims)
        # the append takes a token a request: request r's is row q_start[r] (a slot of -1 has none)
        at = p.q_start[:-1].long().clamp(max=B - 1)
        slot = torch.where(new > 0, p.position[at], torch.full_like(new, -1))
        binding.gist_kv_append(k[at][:, None].contiguous(), v[at][:, None].contiguous(), pool, table, slot, dims=pair)
        binding.gist_attn_paged_decode(q, pool, table, p.kv_len, p.q_start, attn, ws, dims=dims, status=status)
        binding.gist_out_proj_w4(attn, dev[2], dev[3], y, group=group, dims=dims)
        cached.copy_(p.kv_len)
        span.copy_(p.free_range)
        rows.copy_(at)

    history = [[] for _ in range(B)]

    def check(live):
        torch.cuda.synchronize()
        assert int(status) == 0
        xs = x.cpu().double().numpy()
        for i, r in enumerate(live):
            assert int(rows[r]) == i
            history[r].append(xs[i])
            H = np.array(history[r])
            qkv, _ = wq.times(H)
            qkv = qkv.reshape(len(H), -1, d)
            pos = np.arange(len(H))
            qr = su.rotate(qkv[:, :Hq], pos)[-1]
            kk = su.bf16(su.rotate(qkv[:, Hq:Hq + Hkv], pos)).double().numpy()
            vv = su.bf16(qkv[:, Hq + Hkv:]).double().numpy()
            out = np.empty((Hq, d))
            for h in range(Hq):
                s = kk[:, h // 7] @ qr[h] / 8
                p = np.exp(s - s.max())
                out[h] = p / p.sum() @ vv[:, h // 7]
            ref, _ = wo.times(out.reshape(1, -1))
            # q, k, v and the attention's output are each rounded to bf16, and a k or v of the kernel
            # may round the other way: 2^-8 each of |v|, of scores of up to `top` twice that
            top = (np.abs(kk[:, 0]).sum(-1).max() * np.abs(qr).max()) / 8
            tol = 2.0 ** -8 * (3 + 2 * min(top, 8.0)) * np.abs(vv).max() * np.abs(wo.value).sum(1) / np.sqrt(wo.value.shape[1])
            su.near(y[i], ref[0], np.maximum(tol, 2.0 ** -8 * np.abs(ref[0])), f"request {r}")

    g = torch.Generator(device=DEV).manual_seed(0)
    step()  # outside the capture, then undone: the cache is empty again
    cached.zero_()
    table.fill_(-1)
    span.copy_(f.free_range.new_tensor([0, nb]))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    for _ in range(21):
        x.copy_(torch.randn((B, D), generator=g, device=DEV))
        graph.replay()
        check([0, 1, 2])
    fk = binding.gist_pages_fork(cached, i32([-1, -1, -1, 0, 1, 2]), table, free, span, dims=dims, status=status)
    binding.gist_pages_copy(pool, None, fk.copy_src, fk.copy_dst, fk.copy_rows, fk.num_copies, dims=dims, status=status)
    cached.copy_(fk.cached_len)
    span.copy_(fk.free_range)
    for r in range(3):
        history[3 + r] = list(history[r])
    new.fill_(1)
    for i in range(12):
        if i == 6:  # two end; what they held is given back and the rest moved together
            live = [0, 2, 3, 4]
            cached[[1, 5]] = 0
            new[[1, 5]] = 0
            c = binding.gist_pages_compact(cached, table, [table] + list(binding.gist_pages_compact(cached, table, dims=dims))[1:],
                                           dims=dims, status=status)
            binding.gist_pages_copy(pool, None, c.copy_src, c.copy_dst, None, c.num_copies, dims=dims, status=status)
            free.copy_(c.free_blocks)
            span.copy_(c.free_range)
        x.copy_(torch.randn((B, D), generator=g, device=DEV))
        graph.replay()
        check(list(range(6)) if i < 6 else live)
