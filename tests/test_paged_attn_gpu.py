"""gist_attn_paged_fp8kv on the GPU against the definition in 64 bits.

The tolerance of each element counts the roundings: the output's one rounding to
bf16 (2^-9 of it, doubled for a neighbour) and, relative to the largest value
the request's heads hold, 2^-10 for the weights and scores (scores: q carried to
2^-11 or better and fp32 sums move a softmax weight by under 2^-11 of itself for
logits of a few units; weights: 11 bits or more)."""
from __future__ import annotations

import numpy as np
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


SENTINEL = -77.0


def run(pb, args=None, status=0, **kw):
    args = args or pb.args()
    out = torch.full_like(args[0], SENTINEL)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    dims = dict(pb.dims, **kw)
    binding.gist_attn_paged_fp8kv(*args, out, dims=dims, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == status
    return out.float().cpu().numpy().astype(np.float64)


def close(got, ref, what=""):
    written = ~np.isnan(ref)
    assert (got[~written] == SENTINEL).all(), f"{what}: padding rows were written"
    g, r = got[written], ref[written]
    assert np.isfinite(g).all(), what
    top = np.abs(r).max() if r.size else 0.0
    err, bound = np.abs(g - r), 2.0 ** -8 * np.abs(r) + 2.0 ** -10 * top
    worst = float((err / np.maximum(bound, 1e-30)).max()) if r.size else 0.0
    assert worst <= 1.0, f"{what}: worst error / bound {worst:.3f}"


HEADS = [(14, 2, 64), (32, 8, 128), (8, 8, 128), (4, 4, 64), (16, 1, 64), (16, 1, 128), (6, 2, 128)]


@pytest.mark.parametrize("Hq,Hkv,d", HEADS)
@pytest.mark.parametrize("bl", [16, 48, 128, 256])
def test_decode_lengths_around_the_tiles(Hq, Hkv, d, bl):
    lens = [0, 1, 15, 16, 62, 63, 64, 126, 127, 128, 129, 254, 255, 256, 257, 511, 700]
    pb = pu.Problem(lens, [1] * len(lens), Hq, Hkv, d, bl, seed=bl + d + Hq, pad=3)
    close(run(pb), pb.expected(), f"{Hq}/{Hkv}/{d} bl={bl}")


@pytest.mark.parametrize("Hq,Hkv,d", HEADS)
def test_several_new_tokens(Hq, Hkv, d):
    cached = [0, 0, 100, 255, 256, 30, 127, 511, 3]
    new = [1, 7, 2, 3, 4, 0, 2, 5, 6]
    pb = pu.Problem(cached, new, Hq, Hkv, d, 32, seed=d + Hq, pad=2)
    close(run(pb), pb.expected(), f"{Hq}/{Hkv}/{d}")


@pytest.mark.parametrize("Hq,Hkv,d", HEADS)
def test_chunks_and_decoding_requests_together(Hq, Hkv, d):
    cached = [0, 77, 400, 0, 130, 20]
    new = [130, 1, 65, 33, 1, 150]
    pb = pu.Problem(cached, new, Hq, Hkv, d, 16, seed=d, pad=5)
    close(run(pb), pb.expected(), f"{Hq}/{Hkv}/{d}")


@pytest.mark.parametrize("Hq,Hkv,d", HEADS)
@pytest.mark.parametrize("new", [1, 2, 5])
def test_few_tiles_of_requests_that_the_table_leaves_room_for(Hq, Hkv, d, new):
    """The same short sequences with room for long ones in the table: a sequence's
    tiles then go to several blocks of the grid and are joined."""
    lens = [0, 1, 126, 127, 128, 129, 255, 256, 383, 700]
    pb = pu.Problem(lens, [new] * len(lens), Hq, Hkv, d, 32, seed=d + Hq + new, pad=1, extra_width=300)
    close(run(pb), pb.expected(), f"{Hq}/{Hkv}/{d} new={new}")


@pytest.mark.parametrize("d", [64, 128])
def test_joined_parts_with_bad_blocks_and_nan(d):
    """A block outside the pool in one part of a sequence zeroes its rows; a NaN in one
    part reaches the element it stands in."""
    pb = pu.Problem([500, 700, 900], [2, 2, 2], 4, 2, d, 16, seed=3, extra_width=300)
    ref = pb.expected()
    args = list(pb.args())
    t = pb.table.copy()
    t[1, 30] = pb.dims["num_blocks"]
    args[3] = pb.i32(t)
    args[1][int(t[2, 40]), pb.layer, 1, 1, 5, 7] = 0x7F  # V, KV head 1, element 7
    got = run(pb, args, status=binding.STATUS_BAD_BLOCK)
    assert (got[2:4] == 0).all() and np.isnan(got[4:6, 2:, 7]).all()
    got[2:4] = ref[2:4]
    got[4:6, 2:, 7] = ref[4:6, 2:, 7]
    close(got, ref, "others")


def test_wide_groups():
    """Groups wider than 16 heads, up to 128."""
    for Hq, Hkv, d in ((40, 1, 64), (128, 1, 128), (66, 2, 128)):
        pb = pu.Problem([0, 90, 300], [1, 2, 5], Hq, Hkv, d, 32, seed=Hq)
        close(run(pb), pb.expected(), f"{Hq}/{Hkv}")


def test_one_long_sequence():
    for Hq, Hkv, d in ((14, 2, 64), (4, 1, 128)):
        pb = pu.Problem([20011], [1], Hq, Hkv, d, 64, seed=2)
        close(run(pb), pb.expected(), f"long {d}")


def test_many_short_sequences():
    rng = np.random.default_rng(0)
    cached = [int(x) for x in rng.integers(0, 40, 700)]
    pb = pu.Problem(cached, [int(x) for x in rng.integers(0, 3, 700)], 4, 2, 64, 16, seed=1)
    close(run(pb), pb.expected(), "many")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new", [1, 40])
def test_bytes_no_token_sees(d, new):
    """NaN codes behind the last key, and table entries behind the last block that
    name nothing, change nothing."""
    pb = pu.Problem([5, 60, 100, 254], [new] * 4, 8, 2, d, 64, seed=9, extra_width=3)
    ref = pb.expected()
    for r, C in enumerate(pb.kv_len):
        if C % 64:
            pb.codes[pb.table[r, C // 64], :, :, :, C % 64:] = 0x7F
    pb.codes[:, 0] = 0xFF  # the other layer
    close(run(pb), ref, "hidden NaN")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new", [1, 3, 40])
def test_nan_in_the_cache_reaches_the_tokens_that_see_it(d, new):
    pb = pu.Problem([200], [new], 4, 2, d, 16, seed=10)
    pos = 200 if new > 1 else 150  # seen by tokens 1.. of several, or by the only one
    blk = pb.table[0, pos // 16]
    pb.codes[blk, 1, 1, 0, pos % 16, 7] = 0x7F  # V of KV head 0, element 7
    args = pb.args()
    out = torch.full_like(args[0], SENTINEL)
    binding.gist_attn_paged_fp8kv(*args, out, dims=pb.dims)
    got = out.float().cpu().numpy()
    seen = np.array([200 + i >= pos for i in range(new)])
    nan = np.isnan(got)
    assert nan[seen][:, :2, 7].all() and not nan[~seen].any()
    assert not nan[:, 2:].any() and not nan[:, :2, :7].any() and not nan[:, :2, 8:].any()


@pytest.mark.parametrize("new", [1, 40])
def test_scales_far_apart(new):
    """Block scales spread over 2^12, and a softmax with a few large weights."""
    for d in (64, 128):
        pb = pu.Problem([300, 50], [new, new], 8, 2, d, 16, seed=11, spread=12)
        pb.q.mul_(3.0)
        close(run(pb), pb.expected(), f"spread d={d}")


def test_scales_that_are_no_powers_of_two():
    rng = np.random.default_rng(3)
    for new in (1, 33):
        pb = pu.Problem([300, 50], [new, 1], 8, 2, 128, 32, seed=12)
        pb.scale = (pb.scale * rng.uniform(0.5, 1.5, pb.scale.shape)).astype(np.float32).astype(np.float64)
        close(run(pb), pb.expected(), "scales")


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("magnitude", [1e-30, 1e4, 1e30])
def test_magnitudes_of_q(new, magnitude):
    """q far from 1, brought back by the softmax scale: no range of its own."""
    pb = pu.Problem([300], [new], 8, 2, 128, 32, seed=13)
    pb.q = (pb.q.double() * magnitude).to(torch.bfloat16)
    scale = float(np.float32(0.09 / magnitude))
    close(run(pb, softmax_scale=scale), pb.expected(softmax_scale=scale), "magnitude")


def test_prerotated_and_far_positions():
    for new in (1, 35):
        pb = pu.Problem([90, 300], [new, 2], 4, 2, 128, 16, seed=14)
        close(run(pb, flags=binding.FLAG_PREROTATED), pb.expected(rotated=True), "prerotated")


@pytest.mark.parametrize("new", [1, 30])
def test_tokens_that_see_no_key(new):
    """kv_len smaller than the new tokens (a request that was not served): zeros."""
    pb = pu.Problem([0, 40], [new, new], 4, 2, 64, 16, seed=15)
    pb.kv_len = np.array([0, 40 + new])
    got = run(pb)
    assert (got[:new] == 0).all()
    close(got, pb.expected(), "unserved")
    if new > 1:
        pb.kv_len = np.array([7, 40 + new])
        got = run(pb)
        assert (got[:new - 7] == 0).all()
        close(got, pb.expected(), "partly")


@pytest.mark.parametrize("new", [1, 30])
def test_bad_blocks_and_lengths(new):
    pb = pu.Problem([40, 50, 60], [new] * 3, 4, 2, 64, 16, seed=16)
    ref = pb.expected()
    for bad in (-1, pb.dims["num_blocks"]):
        t = pb.table.copy()
        t[1, 1] = bad
        args = list(pb.args())
        args[3] = pb.i32(t)
        got = run(pb, args, status=binding.STATUS_BAD_BLOCK)
        assert (got[new:2 * new] == 0).all()
        got[new:2 * new] = ref[new:2 * new]
        close(got, ref, "others")
    args = list(pb.args())
    lens = pb.kv_len.copy()
    lens[2] = pb.dims["max_blocks"] * 16 + 1
    args[5] = pb.i32(lens)
    got = run(pb, args, status=binding.STATUS_BAD_BLOCK)
    assert (got[2 * new:] == 0).all()
    for starts in ([0, new, 10 ** 6, 3 * new], [0, new, -4, 3 * new], [0, 2 * new, new, 3 * new]):
        args = list(pb.args())
        args[4] = pb.i32(starts)
        run(pb, args, status=binding.STATUS_BAD_BLOCK)


def test_same_answer_again_and_on_another_stream():
    pb = pu.Problem([1000, 30, 500], [1, 4, 60], 14, 2, 64, 16, seed=17)
    a = run(pb)
    assert np.array_equal(a, run(pb))
    args = pb.args()
    out = torch.full_like(args[0], SENTINEL)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    binding.gist_attn_paged_fp8kv(*args, out, dims=pb.dims, stream=s)
    s.synchronize()
    assert np.array_equal(a, out.float().cpu().numpy())
