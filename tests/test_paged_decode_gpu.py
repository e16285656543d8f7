"""Attention of one new token a request over a bf16 paged cache against the definition in 64
bits: head layouts, lengths from none to long, block sizes, bad inputs, streams, graphs."""
from __future__ import annotations

import math
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


HEADS = [(1, 1, 64), (4, 1, 128), (6, 2, 64), (14, 2, 64), (16, 2, 128), (9, 1, 128), (16, 1, 64), (32, 2, 128), (34, 2, 64),
         (40, 1, 128), (32, 32, 128)]
EDGES = [1, 15, 16, 17, 0, 31, 33, 255, 64, 500]


@pytest.mark.parametrize("Hq,Hkv,d", HEADS)
@pytest.mark.parametrize("bl", [16, 48, 256])
def test_head_layouts_and_lengths(Hq, Hkv, d, bl):
    pb = su.Decode(EDGES, Hq, Hkv, d, bl, seed=Hq + bl, extra_width=1)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = binding.gist_attn_paged_decode(*pb.args(), dims=pb.dims, status=status)
    su.near(got, *pb.expected(), f"{Hq}/{Hkv} {d} {bl}")
    assert int(status) == 0
    assert not got[4].any()  # no key: zeros


@pytest.mark.parametrize("lens", [[1], [20000], [30000, 1, 5], [1] * 700, list(range(1, 200)), [4096] * 9 + [7]])
@pytest.mark.parametrize("Hq,Hkv,d", [(14, 2, 64), (8, 4, 128)])
def test_batches_cut_anywhere(lens, Hq, Hkv, d):
    """One long request over all CTAs, many short ones in a warp, and both."""
    pb = su.Decode(lens, Hq, Hkv, d, 32, seed=len(lens))
    got = binding.gist_attn_paged_decode(*pb.args(), dims=pb.dims)
    su.near(got, *pb.expected(), str(lens[:3]))
    assert torch.equal(got, binding.gist_attn_paged_decode(*pb.args(), dims=pb.dims))  # the same bits again


@pytest.mark.parametrize("lens,Hq,Hkv,d,bl", [
    ([70000, 3, 71001], 8, 4, 64, 64),                        # few units, each over all CTAs
    ([150000, 40], 16, 4, 128, 256),
    ([int(x) for x in np.random.default_rng(0).integers(1, 2200, 140)], 16, 4, 64, 32),
    ([int(x) for x in np.random.default_rng(1).integers(300, 2000, 40)], 32, 16, 128, 16),
    ([5000] * 8 + [0, 1] + [4999] * 7, 64, 8, 64, 64),
    ([9000] * 9 + [17], 96, 8, 128, 64),
])
def test_large_batches(lens, Hq, Hkv, d, bl):
    """Runs of many tiles a warp, units over many CTAs; the same bits every time."""
    pb = su.Decode(lens, Hq, Hkv, d, bl, seed=3, layers=1, layer=0)
    args = pb.args()
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = binding.gist_attn_paged_decode(*args, dims=pb.dims, status=status)
    for _ in range(20):
        assert torch.equal(got, binding.gist_attn_paged_decode(*args, dims=pb.dims))
    assert int(status) == 0
    su.near(got, *pb.expected(), str(lens[:4]))
    # a bad block near the end of the last request of some length
    r = max(i for i, n in enumerate(lens) if n > bl)
    bad = args[2].clone()
    bad[r, lens[r] // bl - 1] = -1
    out = binding.gist_attn_paged_decode(*args[:2], bad, args[3], dims=pb.dims, status=status)
    assert not out[r].any() and int(status) == binding.STATUS_BAD_BLOCK
    keep = [i for i in range(len(lens)) if i != r]
    assert torch.equal(out[keep], got[keep])


def test_scale_and_rotation_given():
    pb = su.Decode([300, 40], 8, 2, 128, 16, seed=5)
    pb.dims |= dict(softmax_scale=0.3, flags=binding.FLAG_PREROTATED)
    got = binding.gist_attn_paged_decode(*pb.args(), dims=pb.dims)
    su.near(got, *pb.expected(rotated=True))


@pytest.mark.parametrize("Hq,Hkv", [(4, 1), (8, 1), (16, 1)])
def test_large_scores(Hq, Hkv):
    """Scores of some hundreds: the maximum moves often and most weights vanish."""
    pb = su.Decode([777, 90, 3000], Hq, Hkv, 128, 16, seed=6, spread=20.0)
    su.near(binding.gist_attn_paged_decode(*pb.args(), dims=pb.dims), *pb.expected())


def test_rows_of_the_plan():
    """q_start as the plan leaves it: requests without a token, padding rows left alone."""
    pb = su.Decode([50, 60, 70, 80], 14, 2, 64, 16, seed=7)
    q, pool, table, kv = pb.args()
    dims = dict(pb.dims, num_tokens=5)
    q = torch.cat([q[[0, 2, 3]], q[:2]])
    out = torch.full_like(q, 7.0)
    got = binding.gist_attn_paged_decode(q, pool, table, kv, pb.i32([0, 1, 1, 2, 3]), out, dims=dims)
    ref, tol = pb.expected()
    su.near(got[:3], ref[[0, 2, 3]], tol[[0, 2, 3]])
    assert (got[3:] == 7.0).all()


def test_bad_rows_blocks_and_lengths():
    pb = su.Decode([50, 600, 70, 80, 5000, 30], 8, 2, 64, 16, seed=8)
    q, pool, table, kv = pb.args()
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    ref, tol = pb.expected()
    for bad in (-1, pb.dims["num_blocks"], 1 << 30):
        t = table.clone()
        t[1, 20], t[4, 300] = bad, bad
        status.zero_()
        got = binding.gist_attn_paged_decode(q, pool, t, kv, dims=pb.dims, status=status)
        assert int(status) == binding.STATUS_BAD_BLOCK
        assert not got[1].any() and not got[4].any()
        su.near(got[[0, 2, 3, 5]], ref[[0, 2, 3, 5]], tol[[0, 2, 3, 5]])
    k = kv.clone()
    k[0], k[2] = pb.dims["max_blocks"] * 16 + 1, -5
    status.zero_()
    got = binding.gist_attn_paged_decode(q, pool, table, k, dims=pb.dims, status=status)
    assert int(status) == binding.STATUS_BAD_BLOCK and not got[0].any() and not got[2].any()
    su.near(got[3:], ref[3:], tol[3:])
    for start in ([0, 1, 2, 4, 4, 5, 6], [0, 1, 2, 1, 2, 3, 4], [0, 1, 2, 3, 4, 5, 7], [-1, 0, 1, 2, 3, 4, 5]):
        out = torch.full_like(q, 7.0)
        status.zero_()
        binding.gist_attn_paged_decode(q, pool, table, kv, pb.i32(start), out, dims=pb.dims, status=status)
        assert int(status) == binding.STATUS_BAD_BLOCK
        for r, (a, b) in enumerate(zip(start, start[1:])):
            if b == a + 1 and 0 <= a < 6 and b <= 6 and start.count(a) == 1:
                want = su.attend(q[[a]].cpu().double().numpy(), pb.pool[:, 1].double().numpy(), pb.table[[r]], [pb.lens[r]], 16, 4)
                su.near(out[[a]], *want)


def test_values_that_are_not_finite():
    """A NaN or infinity that a request sees reaches its rows alone and is reported with the sum."""
    pb = su.Decode([100, 40, 2000], 8, 2, 64, 16, seed=9)
    pb.pool[pb.table[0, 2], 1, 0, 1, 3, 5] = math.nan   # a key of request 0, head 1
    pb.pool[pb.table[2, 50], 1, 1, 0, 3, 5] = math.inf  # a value of request 2, head 0: one column
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = binding.gist_attn_paged_decode(*pb.args(), dims=pb.dims, status=status).float()
    assert int(status) == binding.STATUS_RANGE
    assert torch.isnan(got[0, 4:]).all() and torch.isfinite(got[0, :4]).all() and torch.isfinite(got[1]).all()
    hit = ~torch.isfinite(got[2])
    assert hit[:4, 5].all() and hit.sum() == 4
    pb = su.Decode([100], 4, 1, 64, 16, seed=9)
    pb.pool[:, :, 0] = -math.inf
    pb.q.fill_(1.0)
    pb.dims["flags"] = binding.FLAG_PREROTATED
    status.zero_()
    got = binding.gist_attn_paged_decode(*pb.args(), dims=pb.dims, status=status)
    assert torch.isnan(got).all() and int(status) == binding.STATUS_RANGE


def test_a_pool_past_4_gib():
    d, bl, Hkv = 128, 256, 8
    nb = (5 << 30) // (2 * 2 * Hkv * bl * d)
    pool = torch.zeros((nb, 1, 2, Hkv, bl, d), dtype=torch.bfloat16, device=DEV)
    pb = su.Decode([700, 256], 16, Hkv, d, bl, seed=10, layers=1, layer=0)
    ids = torch.tensor([nb - 1, 3, nb - 2, nb - 7], device=DEV)
    table = torch.full((2, 3), -1, dtype=torch.int32, device=DEV)
    for i, (r, j) in enumerate([(0, 0), (0, 1), (0, 2), (1, 0)]):
        pool[ids[i]] = pb.pool[pb.table[r, j]].to(DEV)
        table[r, j] = ids[i]
    got = binding.gist_attn_paged_decode(pb.q.to(DEV), pool, table, pb.i32(pb.lens), dims=dict(pb.dims, num_blocks=nb))
    su.near(got, *pb.expected())


def test_the_uniform_call_agrees():
    """gist_attn_fwd over the cached keys, with the new token given apart."""
    pb = su.Decode([64 + 1] * 3, 8, 2, 128, 16, seed=11)
    q, pool, table, kv = pb.args()
    dims = dict(num_pairs=3, n_new=1, num_q_heads=8, num_kv_heads=2, head_dim=128, block_len=16, blocks_per_pair=4,
                num_blocks=pb.dims["num_blocks"], num_layers=2, layer=1, rope_theta=1e4, softmax_scale=0.0,
                flags=binding.FLAG_PREROTATED)
    last = pool[table[:, 4].long(), 1][:, :, :, 0]  # [3][2][Hkv][d]
    want = binding.gist_attn_fwd(q[:, None], last[:, 0][:, None].contiguous(), last[:, 1][:, None].contiguous(), pool, None,
                                 table[:, :4].contiguous(), None, dims=dims)
    got = binding.gist_attn_paged_decode(q, pool, table, kv, dims=dict(pb.dims, flags=binding.FLAG_PREROTATED))
    ref, tol = pb.expected(rotated=True)
    su.near(got, ref, tol)
    assert (got.float() - want[:, 0].float()).abs().max() <= 2e-2


def test_one_graph_serves_other_lengths():
    """Captured once; lengths, table and q change between replays, on the device."""
    pb = su.Decode([900, 30, 1, 400], 14, 2, 64, 16, seed=12)
    q, pool, table, kv = pb.args()
    out, ws = torch.empty_like(q), torch.empty(binding.paged_decode_workspace_bytes(pb.dims), dtype=torch.uint8, device=DEV)
    binding.gist_attn_paged_decode(q, pool, table, kv, None, out, ws, dims=pb.dims)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        binding.gist_attn_paged_decode(q, pool, table, kv, None, out, ws, dims=pb.dims)
    for lens in ([900, 30, 1, 400], [1, 0, 1, 399], [899, 16, 1, 17]):
        kv.copy_(pb.i32(lens))
        out.fill_(9.0)
        g.replay()
        torch.cuda.synchronize()
        ref = su.attend(pb.q.double().numpy(), pb.pool[:, 1].double().numpy(), pb.table, lens, 16, 7)
        su.near(out, *ref, str(lens))


def test_calls_at_once_on_two_streams():
    pbs = [su.Decode([3000, 5, 70], 8, 2, 128, 16, seed=s) for s in (1, 2)]
    args = [pb.args() for pb in pbs]
    want = [binding.gist_attn_paged_decode(*a, dims=pb.dims) for a, pb in zip(args, pbs)]
    torch.cuda.synchronize()
    failed = []

    def calls(i):
        try:
            s = torch.cuda.Stream()
            for _ in range(50):
                got = binding.gist_attn_paged_decode(*args[i], dims=pbs[i].dims, stream=s)
                s.synchronize()
                assert torch.equal(got, want[i])
        except Exception as e:  # noqa: BLE001 - reported by the test's own thread
            failed.append(e)

    threads = [threading.Thread(target=calls, args=(i % 2,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed


def test_a_workspace_is_asked_for():
    pb = su.Decode([40], 8, 2, 64, 16)
    need = binding.paged_decode_workspace_bytes(pb.dims)
    small = torch.empty(need - 1, dtype=torch.uint8, device=DEV)
    with pytest.raises(binding.GistAttnError) as e:
        binding.gist_attn_paged_decode(*pb.args(), workspace=small, dims=pb.dims)
    assert e.value.code == binding.ERR_SCRATCH
    off = torch.empty(need + 256, dtype=torch.uint8, device=DEV)[16:]
    with pytest.raises(binding.GistAttnError):
        binding.gist_attn_paged_decode(*pb.args(), workspace=off, dims=pb.dims)
    assert np.isfinite(need)
