"""The ragged serving step without a GPU: the C entry points refuse bad arguments
on the host before anything reaches CUDA, the binding refuses tensors that are
not what it says, and the 64-bit definitions that the GPU tests compare with
hold against independent ones."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

import paged_utils as pu
from attention_cached_kv_gb300 import _build, binding

P16 = 0x10000  # a fake, aligned device address: never dereferenced by a call that fails on the host
BASE = dict(num_requests=3, num_tokens=5, max_new=4, num_q_heads=8, num_kv_heads=2, head_dim=64, block_len=16,
            max_blocks=4, num_blocks=9, num_layers=2, layer=1, rope_theta=1e4, softmax_scale=0.0)


@pytest.fixture(scope="module")
def lib():
    _build.build()
    lib = binding.load_library()
    if torch.cuda.is_available():
        pytest.skip("fake device addresses: host-only test")
    return lib


def ptr(x):
    return ctypes.c_void_p(x) if x else None


def dims(d):
    return None if d is None else ctypes.byref(binding.make_paged_dims(d))


PLAN = ["cached_len", "new_len", "block_table", "free_blocks", "num_free", "free_range", "q_start", "kv_len", "slot", "position",
        "free_range_out"]


def plan(lib, d=BASE, **kw):
    # distinct addresses: outputs that alias inputs are refused
    a = {n: P16 + 64 * i for i, n in enumerate(PLAN)} | {"num_free": 6} | kw
    return lib.gist_paged_plan(*[a[n] if n == "num_free" else ptr(a[n]) for n in PLAN], dims(d), None)


@pytest.mark.parametrize("kw,code", [
    (dict(d=None), binding.ERR_NULL), (dict(cached_len=0), binding.ERR_NULL), (dict(new_len=0), binding.ERR_NULL),
    (dict(block_table=0), binding.ERR_NULL), (dict(free_blocks=0), binding.ERR_NULL), (dict(free_range=0), binding.ERR_NULL),
    (dict(q_start=0), binding.ERR_NULL), (dict(kv_len=0), binding.ERR_NULL), (dict(slot=0), binding.ERR_NULL),
    (dict(position=0), binding.ERR_NULL), (dict(free_range_out=0), binding.ERR_NULL), (dict(num_free=-1), binding.ERR_DIMS),
    (dict(kv_len=P16), binding.ERR_DIMS),                 # kv_len == cached_len
    (dict(free_range_out=P16 + 64 * 5), binding.ERR_DIMS),
    (dict(slot=P16 + 2), binding.ERR_ALIGN), (dict(d=dict(BASE, num_requests=-1)), binding.ERR_DIMS),
    (dict(d=dict(BASE, num_tokens=-1)), binding.ERR_DIMS), (dict(d=dict(BASE, block_len=0)), binding.ERR_DIMS),
    (dict(d=dict(BASE, max_blocks=0)), binding.ERR_DIMS), (dict(d=dict(BASE, num_blocks=1 << 28)), binding.ERR_DIMS),
    (dict(d=dict(BASE, num_requests=16385)), binding.ERR_UNSUPPORTED),
])
def test_plan_refuses(lib, kw, code):
    assert plan(lib, **kw) == code


def append(lib, d=BASE, k=P16, v=P16, pool=P16, scale=P16, slot=P16, position=P16):
    return lib.gist_kv_append_fp8(*[ptr(x) for x in (k, v, pool, scale, slot, position)], dims(d), None)


@pytest.mark.parametrize("kw,code", [
    (dict(d=None), binding.ERR_NULL), (dict(k=0), binding.ERR_NULL), (dict(v=0), binding.ERR_NULL),
    (dict(pool=0), binding.ERR_NULL), (dict(scale=0), binding.ERR_NULL), (dict(slot=0), binding.ERR_NULL),
    (dict(position=0), binding.ERR_NULL), (dict(k=P16 + 8), binding.ERR_ALIGN), (dict(pool=P16 + 4), binding.ERR_ALIGN),
    (dict(scale=P16 + 2), binding.ERR_ALIGN), (dict(d=dict(BASE, head_dim=96)), binding.ERR_UNSUPPORTED),
    (dict(d=dict(BASE, layer=2)), binding.ERR_DIMS), (dict(d=dict(BASE, rope_theta=0.0)), binding.ERR_DIMS),
    (dict(d=dict(BASE, flags=8)), binding.ERR_DIMS), (dict(d=dict(BASE, flags=binding.FLAG_TEST_WITHHOLD)), binding.ERR_DIMS),
    (dict(d=dict(BASE, max_new=0)), binding.ERR_DIMS), (dict(d=dict(BASE, num_kv_heads=3)), binding.ERR_DIMS),
])
def test_append_refuses(lib, kw, code):
    assert append(lib, **kw) == code


def test_append_refuses_blocks_past_its_32_bit_counts(lib):
    """Refused before any work (no device here), the largest one allowed is not."""
    big = dict(BASE, num_blocks=1, max_blocks=1)
    assert append(lib, d=dict(big, block_len=(1 << 20) + 1)) == binding.ERR_UNSUPPORTED
    assert append(lib, d=dict(big, block_len=1 << 20, num_tokens=0)) == binding.OK


def test_append_of_nothing(lib):
    assert append(lib, d=dict(BASE, num_tokens=0), k=0, v=0, slot=0, position=0) == binding.OK


def attn(lib, d=BASE, q=P16, pool=P16, scale=P16, table=P16, q_start=P16, kv_len=P16, out=P16, ws=P16, ws_bytes=1 << 40):
    return lib.gist_attn_paged_fp8kv(*[ptr(x) for x in (q, pool, scale, table, q_start, kv_len, out, ws)], ws_bytes, dims(d), None)


@pytest.mark.parametrize("kw,code", [
    (dict(d=None), binding.ERR_NULL), (dict(q=0), binding.ERR_NULL), (dict(pool=0), binding.ERR_NULL),
    (dict(scale=0), binding.ERR_NULL), (dict(table=0), binding.ERR_NULL), (dict(q_start=0), binding.ERR_NULL),
    (dict(kv_len=0), binding.ERR_NULL), (dict(out=0), binding.ERR_NULL), (dict(q=P16 + 8), binding.ERR_ALIGN),
    (dict(out=P16 + 2), binding.ERR_ALIGN), (dict(pool=P16 + 8), binding.ERR_ALIGN), (dict(table=P16 + 1), binding.ERR_ALIGN),
    (dict(d=dict(BASE, block_len=24)), binding.ERR_UNSUPPORTED), (dict(d=dict(BASE, block_len=8)), binding.ERR_UNSUPPORTED),
    (dict(d=dict(BASE, num_q_heads=258)), binding.ERR_UNSUPPORTED),
    (dict(d=dict(BASE, max_blocks=1 << 26, block_len=16, num_blocks=9) | dict(max_blocks=(1 << 26) + 1)), binding.ERR_UNSUPPORTED),
    (dict(d=dict(BASE, softmax_scale=float("nan"))), binding.ERR_DIMS),
    (dict(d=dict(BASE, num_blocks=1 << 26, num_layers=64)), binding.ERR_DIMS),  # planes past 32 bits
])
def test_attention_refuses(lib, kw, code):
    assert attn(lib, **kw) == code


def test_attention_of_nothing(lib):
    assert attn(lib, d=dict(BASE, num_requests=0), q=0, out=0, ws=0) == binding.OK
    assert attn(lib, d=dict(BASE, num_tokens=0), q=0, out=0, ws=0) == binding.OK
    assert lib.gist_attn_paged_workspace_bytes(dims(dict(BASE, num_tokens=0))) == 0
    assert lib.gist_attn_paged_workspace_bytes(dims(dict(BASE, block_len=24))) == 0


def test_status_text(lib):
    assert "not served" in binding.status_string(binding.STATUS_NOT_SERVED)
    assert "scratch" in binding.status_string(binding.ERR_SCRATCH)


def test_binding_refuses_tensors_that_are_not_on_a_gpu():
    i = torch.zeros(8, dtype=torch.int32)
    with pytest.raises(TypeError, match="CUDA"):
        binding.gist_paged_plan(i, i, i, i, i, dims=BASE)
    with pytest.raises(TypeError, match="torch tensor"):
        binding.gist_kv_append_fp8(3, None, None, None, None, dims=BASE)
    with pytest.raises(TypeError, match="CUDA"):
        binding.gist_attn_paged_fp8kv(torch.zeros(8), None, None, None, None, None, dims=BASE)


# ------------------------------------------------ the 64-bit definitions themselves


def test_e4m3_codes_against_torch():
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(pu.E4M3, every)
    x = np.concatenate([np.random.default_rng(0).standard_normal(4000) * 50, pu.E4M3[:127], (pu.E4M3[:126] + pu.E4M3[1:127]) / 2])
    x = np.clip(x, -448, 448).astype(np.float32)
    got = pu.encode(x.astype(np.float64))
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(pu.E4M3[got], pu.E4M3[want])


def test_scale_is_the_smallest_power_of_two():
    rng = np.random.default_rng(1)
    for top in list(np.exp2(rng.uniform(-60, 60, 200))) + [448.0, 316.0, 3.5, 448.0 * 2 ** 7]:
        for limit in (448.0, 316.0):
            s = pu.pow2_scale(float(top), limit)
            assert np.log2(s) == round(np.log2(s)) and top <= limit * s and top > limit * s / 2
    assert pu.pow2_scale(0.0, 448.0) == 2.0 ** -100


def test_attention_definition_against_torch():
    pb = pu.Problem([5, 0], [3, 4], 4, 2, 64, 16, seed=1, device="cpu")
    got = pb.expected(rotated=True)
    for r in range(2):
        a, b, C = pb.q_start[r], pb.q_start[r + 1], pb.kv_len[r]
        ids = pb.table[r, :-(-C // 16)]
        kv = torch.from_numpy(pu.E4M3[pb.codes[ids, 1]] * pb.scale[ids, 1][..., None, None])
        k, v = kv.permute(1, 2, 0, 3, 4).reshape(2, 2, -1, 64)[:, :, :C].repeat_interleave(2, 1)
        mask = torch.ones(b - a, C, dtype=torch.bool).tril(C - (b - a))
        q = pb.q[a:b].double().transpose(0, 1)
        o = torch.nn.functional.scaled_dot_product_attention(q[None], k[None], v[None], attn_mask=mask)[0].transpose(0, 1)
        np.testing.assert_allclose(got[a:b], o.numpy(), atol=1e-12)
