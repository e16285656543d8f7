"""gist_attn_paged_fp8kv over its whole range: V scales of one sequence far apart, q
of large logits, far positions.  Every element has a tolerance of its own, summed
from the roundings of one token and head:

  output    2^-8 |out|, its rounding to bf16
  weights   each off by 2^-10 of itself at most (11 bits and the sums), and by
            2^-24 of the largest weight x scale where they are smaller than that:
            2^-10 sum_j p_j |v_j| + keys 2^-24 448 max_j(p_j scale_j)
  scores    q element i carried to 2^-15.8 of itself and 2^-17 of the row's largest,
            the errors independent and uniform: six deviations of their sum over
            i; and 2^-20 of the products' magnitudes for sums and angles in fp32.
            An error e_j of score j moves the output by sum_j p_j |v_j| (e_j + sum p e)
            (with many rows q is carried to 2^-11 where scores stay below 160 in any
            case: six deviations of that are below the other terms)
"""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import paged_utils as pu
from attention_cached_kv_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda"
SENTINEL = -77.0


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    binding.load_library()
    yield
    torch.cuda.empty_cache()


def expected(pb, rotated):
    """The definition in 64 bits and the tolerance of each element."""
    q, d = pb.q.double().numpy(), pb.dims["head_dim"]
    scale = pb.scale.astype(np.float32).astype(np.float64)
    sc = 1 / math.sqrt(d)
    out, tol = np.full(q.shape, np.nan), np.full(q.shape, np.nan)
    for r, C in enumerate(pb.kv_len):
        a, b = pb.q_start[r], pb.q_start[r + 1]
        ids = pb.table[r, :-(-C // pb.bl)]
        pos = C - (b - a) + np.arange(b - a)
        x = q[a:b] if rotated else pu.rotate(q[a:b], pos)
        for h in range(q.shape[1]):
            g = h // pb.G
            kk, vv = ((pu.E4M3[pb.codes[ids, pb.layer, kv, g]] * scale[ids, pb.layer, kv, g][:, None, None]).reshape(-1, d)[:C]
                      for kv in (0, 1))
            vs = np.repeat(np.abs(scale[ids, pb.layer, 1, g]), pb.bl)[:C]
            for i, p in enumerate(pos):
                if p < 0:  # sees no key
                    out[a + i, h] = tol[a + i, h] = 0.0
                    continue
                k, v, y, s_v = kk[:p + 1], vv[:p + 1], x[i, h], vs[:p + 1]
                s = k @ y * sc
                w = np.exp(s - s.max())
                w /= w.sum()
                dq = 2.0 ** -15.8 * np.abs(y) + 2.0 ** -17 * np.abs(y).max()
                e = sc * (6 / math.sqrt(3) * np.sqrt((k * k) @ (dq * dq)) + 2.0 ** -20 * (np.abs(k) @ np.abs(y)))
                o = w @ v
                mag = np.abs(v) * w[:, None]
                out[a + i, h] = o
                tol[a + i, h] = (2.0 ** -8 * np.abs(o) + 2.0 ** -10 * mag.sum(0) + len(s) * 2.0 ** -24 * 448 * (w * s_v).max()
                                 + (mag * (e + w @ e)[:, None]).sum(0))
    return out, tol


def check(pb, what, rotated=False, status=0):
    args = pb.args()
    out = torch.full_like(args[0], SENTINEL)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    binding.gist_attn_paged_fp8kv(*args, out, dims=dict(pb.dims, flags=binding.FLAG_PREROTATED if rotated else 0), status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == status, what
    got = out.float().cpu().numpy().astype(np.float64)
    ref, tol = expected(pb, rotated)
    written = ~np.isnan(ref)
    assert (got[~written] == SENTINEL).all(), f"{what}: padding rows were written"
    assert np.isfinite(got[written]).all(), what
    worst = (np.abs(got - ref)[written] / np.maximum(tol[written], 1e-37)).max()
    assert worst <= 1.0, f"{what}: worst error / tolerance {worst:.3f}"


def outlier(pb, r, block, k, low):
    """Block `block` of request r gets V scales 2^k, and keys that score about -2 low (in
    a head whose q has 4 as its first element, prerotated)."""
    blk = pb.table[r, block]
    d = pb.dims["head_dim"]
    pb.scale[blk, pb.layer, 1] = 2.0 ** k
    pb.codes[blk, pb.layer, 0] = 0
    pb.codes[blk, pb.layer, 0, ..., 0] = pu.encode(np.array(-448.0))
    pb.scale[blk, pb.layer, 0] = 2.0 * low * math.sqrt(d) / (4 * 448.0)


# new tokens, heads, d: 4, 12, 1 and 32 rows (of which d = 64 takes 16 at most)
FEW = [(n, Hq, Hkv, d) for n, Hq, Hkv in ((1, 8, 2), (3, 8, 2), (1, 4, 4)) for d in (64, 128)] + [(2, 32, 2, 128), (1, 32, 2, 64)]


@pytest.mark.parametrize("new,Hq,Hkv,d", FEW)
@pytest.mark.parametrize("k", [4, 10, 16, 24, 60])
@pytest.mark.parametrize("block", [0, 7, -1])
def test_few_rows_beside_a_block_of_large_v_scale(new, Hq, Hkv, d, k, block):
    """A block of hardly any weight, met first, in the middle or last, takes no bits from
    the others; in the last block it is one that earlier drafted tokens do not see."""
    pb = pu.Problem([300, 40], [new] * 2, Hq, Hkv, d, 16, seed=k + new)
    pb.q[..., 0] = 4.0
    n = -(-int(pb.kv_len[0]) // 16)
    outlier(pb, 0, block % n, k - 7, k)
    check(pb, f"k={k} block={block}", rotated=True)


@pytest.mark.parametrize("d", [64, 128])
def test_few_rows_with_v_scales_in_every_order(d):
    """Scales that fall, rise and alternate by 2^30 along the sequence, weights alike; a
    sequence long enough to be joined from parts."""
    for kind in range(3):
        pb = pu.Problem([3000, 90], [1, 2], 8, 2, d, 16, seed=kind)
        n = -(-int(pb.kv_len[0]) // 16)
        ramp = np.linspace(-15, 15, n).round()
        e = [ramp, -ramp, np.where(np.arange(n) % 2, 15.0, -15.0)][kind]
        pb.scale[pb.table[0, :n], pb.layer, 1] = (2.0 ** e)[:, None]
        check(pb, f"kind {kind}")


@pytest.mark.parametrize("d", [64, 128])
def test_few_rows_with_v_scales_at_the_ends_of_their_range(d):
    """Blocks of zeros at append's smallest scale, blocks of scale zero and of negative
    scale among ordinary ones; sequences of nothing else."""
    pb = pu.Problem([100, 50, 33, 20], [1, 2, 1, 1], 4, 2, d, 16, seed=4)
    t, V = pb.table, (pb.layer, 1)
    for r, blocks in ((0, [0, 3]), (2, [0, 1, 2])):
        for b in blocks:
            pb.codes[t[r, b]][V] = 0
            pb.scale[t[r, b]][V] = 2.0 ** -100
    pb.scale[t[0, 1]][V] = 0.0
    pb.scale[t[0, 4]][V] *= -1
    pb.scale[t[1, :4], pb.layer, 1] = 0.0
    pb.scale[t[3, :2], pb.layer, 1] = 2.0 ** 100
    check(pb, "ends")


def spread(pb, r, e, rng):
    """Request r's V scales 2^e (repeated along its blocks), and a fifth of the blocks zeros
    at the smallest scale."""
    n = -(-int(pb.kv_len[r]) // pb.bl)
    e = np.resize(np.asarray(e, dtype=np.float64), n)
    for b in range(n):
        at = (pb.table[r, b], pb.layer, 1)
        pb.scale[at] = 2.0 ** e[b]
        if rng.random() < 0.2:
            pb.codes[at] = 0
            pb.scale[at] = 2.0 ** -100


SPREADS = [[-90, 0, 90], [90, -90], [60, 20, -20, -60, -95], [-95, -90, -60, 0, 60, 99], [-95] * 3 + [50]]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("e", SPREADS)
def test_few_rows_with_v_scales_over_their_whole_range(d, e):
    """From 2^-95 to 2^99 in one sequence, rising, falling and alternating along it."""
    pb = pu.Problem([330, 2000, 100], [1, 2, 1], 4, 2, d, 16, seed=len(e))
    rng = np.random.default_rng(2)
    for r in range(3):
        spread(pb, r, e if r != 1 else np.repeat(e, 126 // len(e) + 1), rng)
    check(pb, f"{e}")


@pytest.mark.parametrize("new", [1, 2])
def test_few_rows_report_v_scales_past_the_range(new):
    pb = pu.Problem([100, 50], [new, new], 4, 2, 64, 16, seed=4)
    pb.scale[pb.table[1, 1], pb.layer, 1] = 2.0 ** 110
    check(pb, "past", status=binding.STATUS_RANGE)


MANY = [(n, Hq, Hkv, d) for n, Hq, Hkv in ((40, 8, 2), (35, 4, 4), (150, 16, 2), (9, 40, 1)) for d in (64, 128)] + [(2, 32, 2, 64)]


@pytest.mark.parametrize("new,Hq,Hkv,d", MANY)
@pytest.mark.parametrize("k", [4, 16, 24, 30, 60])
@pytest.mark.parametrize("block", [0, 7, -1])
def test_many_rows_beside_a_block_of_large_v_scale(new, Hq, Hkv, d, k, block):
    """As with few rows; in the last block it is one that most new tokens do not see."""
    pb = pu.Problem([300, 40], [new] * 2, Hq, Hkv, d, 16, seed=k + new)
    pb.q[..., 0] = 4.0
    n = -(-int(pb.kv_len[0]) // 16)
    outlier(pb, 0, block % n, k - 7, k)
    check(pb, f"k={k} block={block}", rotated=True)


@pytest.mark.parametrize("d", [64, 128])
def test_many_rows_with_v_scales_in_every_order(d):
    for kind in range(3):
        pb = pu.Problem([1500, 90], [33, 70], 4, 2, d, 16, seed=kind)
        n = -(-int(pb.kv_len[0]) // 16)
        ramp = np.linspace(-15, 15, n).round()
        e = [ramp, -ramp, np.where(np.arange(n) % 2, 15.0, -15.0)][kind]
        pb.scale[pb.table[0, :n], pb.layer, 1] = (2.0 ** e)[:, None]
        check(pb, f"kind {kind}")


@pytest.mark.parametrize("d", [64, 128])
def test_many_rows_with_v_scales_at_the_ends_of_their_range(d):
    pb = pu.Problem([100, 50, 33, 20, 300], [40, 39, 65, 38, 40], 4, 2, d, 16, seed=4)
    t, V = pb.table, (pb.layer, 1)
    for r, blocks in ((0, [0, 3]), (2, range(7)), (4, [2, 17])):
        for b in blocks:
            pb.codes[t[r, b]][V] = 0
            pb.scale[t[r, b]][V] = 2.0 ** -100
    pb.scale[t[0, 1]][V] = 0.0
    for r, b in ((0, 4), (4, 3), (4, 10)):
        pb.scale[t[r, b]] *= -1  # keys too
    pb.scale[t[1, :6], pb.layer, 1] = 0.0
    pb.scale[t[3, :4], pb.layer, 1] = 2.0 ** 100
    check(pb, "ends")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("e", SPREADS)
def test_many_rows_with_v_scales_over_their_whole_range(d, e):
    pb = pu.Problem([330, 1500, 100], [40, 33, 70], 2, 1, d, 16, seed=len(e))
    rng = np.random.default_rng(2)
    for r in range(3):
        spread(pb, r, e if r != 1 else np.repeat(e, 96 // len(e) + 1), rng)
    check(pb, f"{e}")


def test_many_rows_report_v_scales_past_the_range():
    pb = pu.Problem([100, 50], [40, 39], 4, 2, 64, 16, seed=4)
    pb.scale[pb.table[1, 1], pb.layer, 1] = 2.0 ** 110
    check(pb, "past", status=binding.STATUS_RANGE)


@pytest.mark.parametrize("new,Hq,Hkv,d", FEW)
@pytest.mark.parametrize("times", [1, 4, 16, 64])
def test_few_rows_of_large_logits(new, Hq, Hkv, d, times):
    """q whose logits are up to hundreds, rotated here."""
    pb = pu.Problem([300, 77], [new] * 2, Hq, Hkv, d, 16, seed=times)
    pb.q.mul_(float(times))
    check(pb, f"x {times}")


@pytest.mark.parametrize("d", [64, 128])
def test_few_rows_far_from_the_start(d):
    pb = pu.Problem([30011, 20000], [1, 3], 4, 2, d, 64, seed=5)
    pb.q.mul_(8.0)
    check(pb, "far")


@pytest.mark.parametrize("new,Hq,Hkv,d", MANY)
@pytest.mark.parametrize("times", [1, 1.25, 2, 4, 16, 64])
def test_many_rows_of_large_logits(new, Hq, Hkv, d, times):
    pb = pu.Problem([300, 77], [new] * 2, Hq, Hkv, d, 16, seed=int(times))
    pb.q.mul_(float(times))
    check(pb, f"x {times}")


@pytest.mark.parametrize("d", [64, 128])
def test_many_rows_far_from_the_start(d):
    pb = pu.Problem([30011], [35], 2, 1, d, 64, seed=5)
    pb.q.mul_(8.0)
    check(pb, "far")


HEADS = [(14, 2, 64), (32, 8, 128), (8, 8, 128), (16, 1, 64), (16, 1, 128), (6, 2, 128)]
BATCHES = {"decode": ([0, 1, 15, 63, 64, 127, 128, 255, 256, 700], [1] * 10, 0),
           "room for long ones": ([0, 126, 129, 383, 700], [1, 2, 5, 3, 2], 300),
           "mixed": ([0, 77, 400, 0, 130, 20], [130, 1, 65, 33, 1, 150], 0),
           "one chunk behind many keys": ([3000, 5], [37, 2], 0)}


@pytest.mark.parametrize("Hq,Hkv,d", HEADS)
@pytest.mark.parametrize("name", BATCHES)
def test_every_request_and_head_by_itself(Hq, Hkv, d, name):
    """Heads and requests whose values lie 2^12 apart and more: each by its own measure."""
    cached, new, room = BATCHES[name]
    pb = pu.Problem(cached, new, Hq, Hkv, d, 16, seed=d + Hq, pad=3, extra_width=room)
    for r in range(len(cached)):
        n = -(-int(pb.kv_len[r]) // 16)
        for g in range(Hkv):
            pb.scale[pb.table[r, :n], pb.layer, 1, g] *= 2.0 ** (12 * ((r + g) % 4) - 20)
    check(pb, name)
