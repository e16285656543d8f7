"""gist_kv_append_fp8 on the GPU against a block-by-block construction in 64 bits.

Scales and codes of values are exact (powers of two, one rounding).  A rotated
key is computed in fp32 before its one rounding to E4M3, so it may land on the
other side of a rounding border: then the code is the neighbour (codes of one
sign are ordered as their values)."""
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


def ordered(codes):
    """Codes as integers in the order of their values (both zeros 0)."""
    c = codes.astype(np.int64)
    return np.where(c & 128, -(c & 127), c & 127)


def check(pb, k, v, slot, position, rotated=False, status=0):
    dims = dict(pb.dims, flags=binding.FLAG_PREROTATED if rotated else 0, num_tokens=len(slot))
    pool, scale = pb.args()[1:3]
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    binding.gist_kv_append_fp8(k.to(DEV), v.to(DEV), pool, scale, pb.i32(slot),
                               None if rotated else pb.i32(position), dims=dims, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == status
    good = np.where(np.asarray(slot) < pb.dims["num_blocks"] * pb.bl, slot, -1)
    codes, scales = pu.append(k.double().numpy(), v.double().numpy(), pb.codes, pb.scale, good, np.asarray(position), pb.bl,
                              pb.layer, rotated)
    got = pool.cpu().numpy()
    np.testing.assert_array_equal(scale.cpu().numpy().astype(np.float64), scales)
    np.testing.assert_array_equal(got[:, :, 1], codes[:, :, 1])
    far = np.abs(ordered(got[:, :, 0]) - ordered(codes[:, :, 0]))
    if rotated:
        assert far.max() == 0
    else:
        # fp32 against 64 bits: |angle| <= pi to 2^-22 or so, a few roundings of
        # 2^-24: under 2^-20 of the pair; a border is met once in about
        # 2^-20 / 2^-4 / 2 of the codes: 2^-15; the neighbour, never further
        assert far.max() <= 1 and (far > 0).sum() <= max(3, far.size * 2.0 ** -13)
    return got, scale


def fresh(pb, seed, magnitude=1.0):
    rng = np.random.default_rng(seed)
    n = pb.dims
    x = rng.standard_normal((2, pb.T, n["num_kv_heads"], n["head_dim"])) * magnitude
    return tuple(torch.from_numpy(a).to(torch.bfloat16) for a in x)


def places(pb):
    slot, position = [], []
    for r, (c, n) in enumerate(zip(pb.cached, pb.new)):
        for p in range(c, c + n):
            slot.append(int(pb.table[r, p // pb.bl]) * pb.bl + p % pb.bl)
            position.append(p)
    return slot, position


@pytest.mark.parametrize("Hkv,d,bl,cached,new", [
    (2, 64, 16, [0, 5, 16, 31], [1, 1, 1, 1]),
    (8, 128, 256, [4000, 255, 256, 0, 70], [1, 1, 1, 1, 1]),
    (1, 128, 16, [3, 0, 40], [50, 16, 7]),
    (3, 64, 48, [47, 1], [100, 200]),
    (2, 128, 256, [100], [700]),          # more rows of a block than a thread holds
    (2, 64, 256, [0, 255], [513, 300]),
    (4, 64, 5, [3, 0, 11], [9, 5, 1]),
    (32, 128, 32, [10] * 40, [1] * 40),
])
@pytest.mark.parametrize("magnitude", [1.0, 1e-3, 300.0])
def test_every_code_and_scale(Hkv, d, bl, cached, new, magnitude):
    pb = pu.Problem(cached, new, Hkv, Hkv, d, bl, seed=bl + d)
    k, v = fresh(pb, 5, magnitude)
    check(pb, k, v, *places(pb))


def test_prerotated_keys_are_exact():
    pb = pu.Problem([7, 100], [20, 3], 4, 4, 128, 32, seed=3)
    k, v = fresh(pb, 6)
    check(pb, k, v, *places(pb), rotated=True)


def test_far_positions():
    pb = pu.Problem([3, 9], [9, 2], 2, 2, 64, 16, seed=4)
    k, v = fresh(pb, 7)
    slot, position = places(pb)
    check(pb, k, v, slot, [p + 2 ** 30 + 17 for p in position])


def test_special_values():
    """Zeros, infinities, NaN, subnormals and the largest bf16 values."""
    pb = pu.Problem([4, 0, 0, 0], [3, 2, 2, 2], 2, 2, 64, 16, seed=5)
    k, v = fresh(pb, 8)
    for x in (k, v):
        x[0, 0, 3], x[1, 0, 4], x[2, 1, 5] = float("inf"), float("-inf"), float("nan")
        x[3:5] = 0
        x[5:7] *= 1e-39
        x[7:9] = torch.where(x[7:9] > 0, 3.3e38, -3.3e38).to(torch.bfloat16)
    check(pb, k, v, *places(pb), rotated=True)


def test_skipped_and_bad_slots():
    pb = pu.Problem([4, 9], [6, 5], 2, 2, 64, 16, seed=6)
    k, v = fresh(pb, 9)
    slot, position = places(pb)
    slot[2], slot[8] = -1, -5
    check(pb, k, v, slot, position)
    slot[9] = pb.dims["num_blocks"] * 16
    check(pb, k, v, slot, position, status=binding.STATUS_BAD_BLOCK)


def test_token_by_token_equals_all_at_once():
    """Growing scales are powers of two: in the range of normal codes a block
    written a token at a time holds what one call writes."""
    pb = pu.Problem([0], [64], 2, 2, 64, 32, seed=7)
    rng = np.random.default_rng(1)
    x = torch.from_numpy(np.exp2(rng.uniform(-2, 6, (2, 64, 2, 64))) * rng.choice([-1, 1], (2, 64, 2, 64))).to(torch.bfloat16)
    slot, position = places(pb)
    pool, scale = pb.args()[1:3]
    pool2, scale2 = pool.clone(), scale.clone()
    dims = dict(pb.dims, flags=binding.FLAG_PREROTATED)
    binding.gist_kv_append_fp8(x[0].to(DEV), x[1].to(DEV), pool, scale, pb.i32(slot), dims=dims)
    for t in range(64):
        binding.gist_kv_append_fp8(x[0, t:t + 1].to(DEV), x[1, t:t + 1].to(DEV), pool2, scale2, pb.i32(slot[t:t + 1]),
                                   dims=dict(dims, num_tokens=1))
    torch.cuda.synchronize()
    assert torch.equal(scale, scale2) and torch.equal(pool, pool2)
