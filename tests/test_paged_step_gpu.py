"""The ragged serving step as a server runs it: plan, append and attention one
after another, step by step, eagerly and from one captured graph; two calls at
once; pools past 4 GiB; the E4M3 pool shared with gist_attn_fwd_fp8kv."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import paged_utils as pu
from attention_cached_kv_gb300 import binding
from test_paged_attn_gpu import close

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


class Server:
    """Static buffers of a batch and its cache; a step reads `new_len`, q, k, v and
    leaves the output, the table and the lengths of the next step."""

    def __init__(self, B, T, Hq, Hkv, d, bl, W, num_blocks, max_new, seed, layers=2):
        g = np.random.default_rng(seed)
        self.dims = dict(num_requests=B, num_tokens=T, max_new=max_new, num_q_heads=Hq, num_kv_heads=Hkv, head_dim=d,
                         block_len=bl, max_blocks=W, num_blocks=num_blocks, num_layers=layers, layer=0, rope_theta=1e4,
                         softmax_scale=0.0)
        self.pool = torch.full((num_blocks, layers, 2, Hkv, bl, d), 0x7F, dtype=torch.uint8, device=DEV)  # NaN: never seen
        self.scale = torch.ones((num_blocks, layers, 2, Hkv), device=DEV)
        self.table = torch.full((B, W), -1, dtype=torch.int32, device=DEV)
        self.free = i32(g.permutation(num_blocks))
        self.range = i32([0, num_blocks])
        self.cached = torch.zeros(B, dtype=torch.int32, device=DEV)
        self.new = torch.zeros(B, dtype=torch.int32, device=DEV)
        self.plan = [torch.zeros(n, dtype=torch.int32, device=DEV) for n in (B + 1, B, T, T, 2)]
        self.q = torch.zeros((T, Hq, d), dtype=torch.bfloat16, device=DEV)
        self.k = torch.zeros((layers, T, Hkv, d), dtype=torch.bfloat16, device=DEV)
        self.v = torch.zeros_like(self.k)
        self.out = torch.zeros((layers, T, Hq, d), dtype=torch.bfloat16, device=DEV)
        self.ws = torch.empty(binding.paged_workspace_bytes(self.dims), dtype=torch.uint8, device=DEV)
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)

    def step(self):
        kw = dict(status=self.status)
        p = binding.gist_paged_plan(self.cached, self.new, self.table, self.free, self.range, self.plan, dims=self.dims, **kw)
        for layer in range(self.dims["num_layers"]):
            d = dict(self.dims, layer=layer)
            binding.gist_kv_append_fp8(self.k[layer], self.v[layer], self.pool, self.scale, p.slot, p.position, dims=d, **kw)
            binding.gist_attn_paged_fp8kv(self.q, self.pool, self.scale, self.table, p.q_start, p.kv_len, self.out[layer],
                                          self.ws, dims=d, **kw)
        self.cached.copy_(p.kv_len)
        self.range.copy_(p.free_range)

    def feed(self, new, rng):
        self.new.copy_(i32(new))
        for t in (self.q, self.k, self.v):
            t.copy_(torch.from_numpy(rng.standard_normal(t.shape).astype(np.float32)))

    def check(self, new):
        """The outputs against the definition on what the cache holds."""
        torch.cuda.synchronize()
        assert int(self.status.item()) == 0
        q_start, kv_len = self.plan[0].cpu().numpy(), self.plan[1].cpu().numpy()
        n = int(sum(new))
        codes, scale, table = self.pool.cpu().numpy(), self.scale.cpu().numpy().astype(np.float64), self.table.cpu().numpy()
        G = self.dims["num_q_heads"] // self.dims["num_kv_heads"]
        for layer in range(self.dims["num_layers"]):
            ref = pu.attend(self.q.cpu().double().numpy(), codes, scale, table, q_start, kv_len, self.dims["block_len"], layer, G)
            got = self.out[layer].float().cpu().numpy().astype(np.float64)
            close(got[:n], ref[:n], f"layer {layer}")


STEPS = [[40, 0, 17, 100], [1, 30, 1, 1], [1, 1, 1, 1], [3, 1, 0, 5], [1, 1, 1, 1], [0, 64, 1, 1]]


@pytest.mark.parametrize("Hq,Hkv,d", [(14, 2, 64), (16, 4, 128)])
def test_a_conversation_of_steps(Hq, Hkv, d):
    rng = np.random.default_rng(0)
    s = Server(4, 160, Hq, Hkv, d, 16, 12, 40, 100, seed=d)
    for step, new in enumerate(STEPS):
        s.feed(new, rng)
        s.step()
        s.check(new)
    # the cache holds what was fed, to E4M3's half step at its scale (2^-4 of a value, 2^-10
    # of the scale for subnormals) and twice that where a block's scale grew
    last = STEPS[-1]
    slot, position = s.plan[2].cpu().numpy(), s.plan[3].cpu().numpy()
    for layer in range(2):
        want = pu.rotate(s.k[layer].cpu().double().numpy(), np.maximum(position, 0))
        for t in range(sum(last)):
            blk, off = divmod(int(slot[t]), 16)
            sc = s.scale[blk, layer, 0].cpu().double().numpy()[:, None]
            got = pu.E4M3[s.pool[blk, layer, 0, :, off].cpu().numpy()] * sc
            assert (np.abs(got - want[t]) <= 2.0 ** -4 * np.abs(want[t]) * 1.001 + 2.0 ** -10 * sc).all()


def test_one_captured_graph_serves_every_step():
    eager, graphed = (Server(4, 160, 16, 4, 128, 32, 8, 30, 100, seed=3) for _ in range(2))
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):  # warm-up outside the capture, on an empty step
        graphed.step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        graphed.step()
    for step, new in enumerate(STEPS):
        for s in (eager, graphed):
            s.feed(new, np.random.default_rng(step))
        eager.step()
        g.replay()
        torch.cuda.synchronize()
        n = sum(new)
        assert torch.equal(eager.out[:, :n], graphed.out[:, :n])
        for a, b in zip(eager.plan + [eager.pool, eager.scale, eager.table], graphed.plan + [graphed.pool, graphed.scale, graphed.table]):
            assert torch.equal(a, b)
    eager.check(STEPS[-1])


def test_two_calls_at_once():
    """Two streams, a workspace each: the answers of the calls one after another."""
    pbs = [pu.Problem([3000, 700, 20], [1, 2, 3], 8, 2, 64, 16, seed=1), pu.Problem([500, 900], [200, 90], 8, 2, 128, 32, seed=2)]
    args = [pb.args() for pb in pbs]
    alone = []
    for pb, a in zip(pbs, args):
        alone.append(binding.gist_attn_paged_fp8kv(*a, dims=pb.dims))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in pbs]
    for round in range(5):
        outs = [torch.empty_like(a[0]) for a in args]
        ws = [torch.empty(binding.paged_workspace_bytes(pb.dims), dtype=torch.uint8, device=DEV) for pb in pbs]
        torch.cuda.synchronize()
        for pb, a, o, w, st in zip(pbs, args, outs, ws, streams):
            binding.gist_attn_paged_fp8kv(*a, o, w, dims=pb.dims, stream=st)
        torch.cuda.synchronize()
        for o, ref in zip(outs, alone):
            assert torch.equal(o, ref)


def test_parts_of_an_earlier_call_do_not_matter():
    """A workspace full of NaN, of another call's parts, of zeros: the same answer."""
    pb = pu.Problem([3000, 900, 40], [1, 150, 33], 16, 2, 128, 16, seed=4)
    a = pb.args()
    n = binding.paged_workspace_bytes(pb.dims)
    outs = []
    for fill in (0xFF, 0x00, 0x7F):
        ws = torch.full((n,), fill, dtype=torch.uint8, device=DEV)
        for _ in range(2):
            outs.append(binding.gist_attn_paged_fp8kv(*a, None, ws, dims=pb.dims))
    torch.cuda.synchronize()
    n = int(pb.q_start[-1])
    assert all(torch.equal(o[:n], outs[0][:n]) for o in outs)


def test_pool_past_four_gib():
    """The last blocks of a pool of more than 2^32 bytes: what a small pool gives."""
    pb = pu.Problem([300, 90, 5], [1, 40, 3], 16, 8, 128, 256, seed=5, layers=8, layer=7)
    q, pool, scale, table, q_start, kv_len = pb.args()
    small = binding.gist_attn_paged_fp8kv(q, pool, scale, table, q_start, kv_len, dims=pb.dims)
    nb = pb.dims["num_blocks"]
    shift = 2 ** 32 // (pool[0].numel()) + 3
    big = torch.zeros((shift + nb,) + pool.shape[1:], dtype=torch.uint8, device=DEV)
    big[shift:] = pool
    big_scale = torch.zeros((shift + nb,) + scale.shape[1:], device=DEV)
    big_scale[shift:] = scale
    moved = torch.where(table >= 0, table + shift, table)
    dims = dict(pb.dims, num_blocks=shift + nb)
    out = binding.gist_attn_paged_fp8kv(q, big, big_scale, moved.contiguous(), q_start, kv_len, dims=dims)
    torch.cuda.synchronize()
    assert torch.equal(out, small)
    k = torch.randn((44, 8, 128), device=DEV).to(torch.bfloat16)
    slot, position = [], []
    for r, (c, n) in enumerate(zip(pb.cached, pb.new)):
        for p in range(c, c + n):
            slot.append(int(pb.table[r, p // 256]) * 256 + p % 256)
            position.append(p)
    binding.gist_kv_append_fp8(k, k, pool, scale, i32(slot), i32(position), dims=pb.dims)
    binding.gist_kv_append_fp8(k, k, big, big_scale, i32(np.array(slot) + shift * 256), i32(position), dims=dims)
    torch.cuda.synchronize()
    assert torch.equal(big[shift:], pool) and torch.equal(big_scale[shift:], scale) and not big[:shift].any()


def test_the_pool_is_the_one_that_gist_attn_fwd_fp8kv_reads():
    """A decode step over full blocks: the cache and the new token apart
    (gist_attn_fwd_fp8kv), or the token appended first.  The token's values are E4M3
    values, so that appending it rounds nothing; both kernels round within the
    tolerance of close()."""
    Hq, Hkv, d, bl, nblk, B = 16, 4, 128, 64, 5, 3
    pb = pu.Problem([nblk * bl] * B, [1] * B, Hq, Hkv, d, bl, seed=6)
    q, pool, scale, table, q_start, kv_len = pb.args()
    rng = np.random.default_rng(7)
    kv = [torch.from_numpy(rng.integers(-14, 15, (B, Hkv, d)) / 8.0).to(torch.bfloat16).to(DEV) for _ in range(2)]
    old = dict(num_pairs=B, n_new=1, num_q_heads=Hq, num_kv_heads=Hkv, head_dim=d, block_len=bl, blocks_per_pair=nblk,
               num_blocks=pb.dims["num_blocks"], num_layers=2, layer=1, rope_theta=1e4, softmax_scale=0.0,
               flags=binding.FLAG_PREROTATED)
    want = binding.gist_attn_fwd_fp8kv(q.view(B, 1, Hq, d), kv[0].view(B, 1, Hkv, d), kv[1].view(B, 1, Hkv, d), pool, scale, None,
                                       table[:, :nblk].contiguous(), dims=old)
    dims = dict(pb.dims, flags=binding.FLAG_PREROTATED)
    slot = [int(pb.table[r, nblk]) * bl for r in range(B)]
    binding.gist_kv_append_fp8(kv[0], kv[1], pool, scale, i32(slot), dims=dims)
    got = binding.gist_attn_paged_fp8kv(q, pool, scale, table, q_start, kv_len, dims=dims)
    torch.cuda.synchronize()
    a, b = (x.float().cpu().numpy().astype(np.float64).reshape(B, Hq, d) for x in (got, want))
    top = np.abs(b).max()
    assert (np.abs(a - b) <= 2 * (2.0 ** -8 * np.abs(b) + 2.0 ** -10 * top)).all()


def test_rows_of_q_that_are_not_finite():
    for new in (1, 40):
        pb = pu.Problem([200, 30], [new, new], 8, 2, 64, 16, seed=8)
        ref = pb.expected()
        pb.q[0, 3, 5] = float("inf")
        pb.q[new, 1, 9] = float("nan")
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        got = binding.gist_attn_paged_fp8kv(*pb.args(), dims=pb.dims, status=st).float().cpu().numpy().astype(np.float64)
        assert int(st.item()) == binding.STATUS_RANGE
        assert np.isnan(got[0, 3]).all() and np.isnan(got[new, 1]).all()
        got[0, 3], got[new, 1] = ref[0, 3], ref[new, 1]
        close(got, ref, f"new={new}")


def test_the_binding_refuses_what_does_not_fit():
    pb = pu.Problem([40], [2], 8, 2, 64, 16, seed=9)
    a = list(pb.args())
    with pytest.raises(ValueError, match="q holds"):
        binding.gist_attn_paged_fp8kv(a[0][:1].contiguous(), *a[1:], dims=pb.dims)
    with pytest.raises(TypeError, match="contiguous"):
        binding.gist_attn_paged_fp8kv(a[0].transpose(0, 1), *a[1:], dims=pb.dims)
    with pytest.raises(TypeError, match="float8"):
        binding.gist_attn_paged_fp8kv(a[0], a[1].float(), *a[2:], dims=pb.dims)
    with pytest.raises(binding.GistAttnError) as e:
        binding.gist_attn_paged_fp8kv(*a, None, torch.empty(16, dtype=torch.uint8, device=DEV), dims=pb.dims)
    assert e.value.code == binding.ERR_SCRATCH
    with pytest.raises(ValueError, match="block_table holds"):
        binding.gist_attn_paged_fp8kv(*a, dims=dict(pb.dims, block_len=8, max_blocks=2 * pb.dims["max_blocks"], num_blocks=1))
    with pytest.raises(binding.GistAttnError) as e:
        binding.gist_attn_paged_fp8kv(*a, dims=dict(pb.dims, block_len=8))
    assert e.value.code == binding.ERR_UNSUPPORTED
