"""The single-token step, the cache's blocks and the 4-bit projections without a GPU: the C entry
points refuse bad arguments on the host, the binding refuses tensors that are not what it says,
and the definitions that the GPU tests compare with hold against independent ones."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

import serving_utils as su
from attention_cached_kv_gb300 import _build, binding

P16 = 0x10000  # a fake, aligned device address: never dereferenced by a call that fails on the host
BASE = dict(num_requests=3, num_tokens=5, max_new=1, num_q_heads=8, num_kv_heads=2, head_dim=64, block_len=16, max_blocks=4,
            num_blocks=9, num_layers=2, layer=1, rope_theta=1e4, softmax_scale=0.0)
NULL, DIMS, UNSUPPORTED, ALIGN = binding.ERR_NULL, binding.ERR_DIMS, binding.ERR_UNSUPPORTED, binding.ERR_ALIGN


@pytest.fixture(scope="module")
def lib():
    _build.build()
    lib = binding.load_library()
    if torch.cuda.is_available():
        pytest.skip("fake device addresses: host-only test")
    return lib


def call(fn, names, numbers, d, kw):
    """fn(pointers and numbers by name, dims, no stream), every pointer another address."""
    a = {n: P16 + 256 * i for i, n in enumerate(names)} | numbers
    kw = dict(kw)
    d = kw.pop("d", d)
    a |= kw
    args = [a[n] if n in numbers else ctypes.c_void_p(a[n]) if a[n] else None for n in names]
    return fn(*args, None if d is None else ctypes.byref(binding.make_paged_dims(d)), None)


DECODE = ["q", "kv_pool", "block_table", "q_start", "kv_len", "out", "workspace", "workspace_bytes"]


def decode(lib, **kw):
    return call(lib.gist_attn_paged_decode, DECODE, {"workspace_bytes": 1 << 40}, BASE, kw)


@pytest.mark.parametrize("kw,code", [(dict(d=None), NULL)] + [({n: 0}, NULL) for n in ("q", "kv_pool", "block_table", "kv_len", "out")] + [
    (dict(q=P16 + 8), ALIGN), (dict(kv_pool=P16 + 2), ALIGN), (dict(out=P16 + 2), ALIGN), (dict(kv_len=P16 + 2), ALIGN),
    (dict(q_start=P16 + 1), ALIGN), (dict(d=dict(BASE, max_new=2)), UNSUPPORTED), (dict(d=dict(BASE, block_len=24)), UNSUPPORTED),
    (dict(d=dict(BASE, head_dim=96)), UNSUPPORTED), (dict(d=dict(BASE, num_q_heads=258)), UNSUPPORTED),
    (dict(d=dict(BASE, max_blocks=(1 << 26) + 1)), UNSUPPORTED), (dict(d=dict(BASE, num_requests=1 << 26, max_blocks=64)), UNSUPPORTED),
    (dict(d=dict(BASE, num_q_heads=(1 << 23) + 1, num_kv_heads=(1 << 23) + 1, num_layers=1, layer=0, max_blocks=1)), UNSUPPORTED),
    (dict(q_start=0, d=dict(BASE, num_tokens=2)), DIMS), (dict(d=dict(BASE, num_kv_heads=3)), DIMS),
    (dict(d=dict(BASE, layer=2)), DIMS), (dict(d=dict(BASE, flags=2)), DIMS), (dict(d=dict(BASE, softmax_scale=float("inf"))), DIMS),
    (dict(d=dict(BASE, num_requests=-1)), DIMS), (dict(d=dict(BASE, num_blocks=0)), DIMS),
])
def test_decode_refuses(lib, kw, code):
    assert decode(lib, **kw) == code


def test_decode_of_nothing(lib):
    nothing = dict(q=0, kv_pool=0, block_table=0, kv_len=0, out=0, workspace=0)
    assert decode(lib, d=dict(BASE, num_requests=0), **nothing) == binding.OK
    assert decode(lib, d=dict(BASE, num_tokens=0), **nothing) == binding.OK
    assert binding.paged_decode_workspace_bytes(dict(BASE, num_tokens=0)) == 0
    assert binding.paged_decode_workspace_bytes(dict(BASE, block_len=24)) == 0


def test_decode_refuses_more_tiles_than_it_counts(lib):
    """B Hkv (W block_len / 16 + 1) up to 2^31 - 2^25: the last run's end is counted in 31 bits too."""
    d = dict(BASE, max_blocks=64)  # 130 tiles a request
    most = ((1 << 31) - (1 << 25)) // 130
    assert decode(lib, d=dict(d, num_requests=most + 1)) == UNSUPPORTED
    assert decode(lib, d=dict(d, num_requests=most), q=0) == NULL  # counted, and refused for another reason
    assert binding.paged_decode_workspace_bytes(dict(d, num_requests=most + 1)) == 0


FREE = ["cached_len", "block_table", "ref_count", "free_blocks", "free_range"]
COMPACT = ["cached_len", "block_table", "block_table_out", "new_id", "copy_src", "copy_dst", "num_copies", "free_blocks", "free_range"]
FORK = ["cached_len", "parent", "block_table", "free_blocks", "num_free", "free_range", "cached_len_out", "copy_src", "copy_dst",
        "copy_rows", "num_copies", "free_range_out"]
COPY = ["kv_pool", "kv_scale", "elem_bytes", "copy_src", "copy_dst", "copy_rows", "num_copies", "max_copies"]
PAGES = {"free": (FREE, {}), "compact": (COMPACT, {}), "fork": (FORK, {"num_free": 6}), "copy": (COPY, {"elem_bytes": 2, "max_copies": 4})}


def pages(lib, which, **kw):
    return call(getattr(lib, "gist_pages_" + which), *PAGES[which], BASE, kw)


NEEDED = [(w, n) for w, (names, numbers) in PAGES.items() for n in names
          if n not in numbers and (w, n) not in (("copy", "kv_scale"), ("copy", "copy_rows"), ("copy", "num_copies"))]


@pytest.mark.parametrize("which,name", NEEDED)
def test_pages_refuse_null_and_unaligned(lib, which, name):
    assert pages(lib, which, **{name: 0}) == NULL
    assert pages(lib, which, **{name: P16 + 0x9001}) == ALIGN


@pytest.mark.parametrize("which,kw,code", [(w, dict(d=None), NULL) for w in PAGES] + [
    (w, dict(d=dict(BASE, **bad)), DIMS) for w in PAGES for bad in (dict(num_blocks=0), dict(block_len=0), dict(max_blocks=0))] + [
    (w, dict(d=dict(BASE, block_len=1, num_blocks=(1 << 30) + 1)), UNSUPPORTED) for w in PAGES] + [
    ("free", dict(d=dict(BASE, num_requests=1 << 24, max_blocks=1 << 13)), UNSUPPORTED),
    ("compact", dict(d=dict(BASE, num_requests=(1 << 30) + 1, max_blocks=1)), UNSUPPORTED),
    ("fork", dict(num_free=-1), DIMS), ("fork", dict(d=dict(BASE, num_requests=16385)), UNSUPPORTED),
    ("fork", dict(cached_len_out=P16), DIMS), ("fork", dict(free_range_out=P16 + 256 * 5), DIMS),
    ("copy", dict(elem_bytes=4), DIMS), ("copy", dict(max_copies=-1), DIMS), ("copy", dict(d=dict(BASE, head_dim=32)), UNSUPPORTED),
    ("copy", dict(d=dict(BASE, num_layers=0)), DIMS), ("copy", dict(d=dict(BASE, num_kv_heads=0)), DIMS),
    ("copy", dict(d=dict(BASE, num_layers=1 << 20, num_kv_heads=64)), UNSUPPORTED), ("copy", dict(kv_scale=P16 + 2), ALIGN),
    ("copy", dict(kv_pool=P16 + 8), ALIGN)])
def test_pages_refuse(lib, which, kw, code):
    assert pages(lib, which, **kw) == code


def test_copies_of_nothing(lib):
    assert pages(lib, "copy", max_copies=0, kv_pool=0, copy_src=0, copy_dst=0) == binding.OK


QKV = ["x", "w", "w_scale", "position", "q", "k_new", "v_new", "d_model", "group"]
OUT = ["attn_out", "w", "w_scale", "y", "d_model", "group"]


def qkv(lib, **kw):
    return call(lib.gist_qkv_rope_w4, QKV, {"d_model": 256, "group": 64}, BASE, kw)


def out_proj(lib, **kw):
    return call(lib.gist_out_proj_w4, OUT, {"d_model": 256, "group": 64}, BASE, kw)


@pytest.mark.parametrize("fn,names", [(qkv, QKV[:7]), (out_proj, OUT[:4])])
def test_projections_refuse(lib, fn, names):
    for n in names:
        assert fn(lib, **{n: 0}) == NULL
        assert fn(lib, **{n: P16 + 0x9001}) == ALIGN
    assert fn(lib, d=None) == NULL
    for g in (0, 16, 96, 256):
        assert fn(lib, group=g) == UNSUPPORTED
    assert fn(lib, d_model=0) == DIMS and fn(lib, d_model=-64) == DIMS
    assert fn(lib, d_model=65536 + 128) == UNSUPPORTED
    for bad, code in ((dict(head_dim=80), UNSUPPORTED), (dict(num_kv_heads=3), DIMS), (dict(num_tokens=-1), DIMS),
                      (dict(num_tokens=(1 << 20) + 1), UNSUPPORTED), (dict(num_q_heads=1 << 14), UNSUPPORTED)):
        assert fn(lib, d=dict(BASE, **bad)) == code
    assert fn(lib, d=dict(BASE, num_tokens=0), **{n: 0 for n in names}) == binding.OK


def test_projections_refuse_sizes_of_their_own(lib):
    assert qkv(lib, d_model=224) == UNSUPPORTED               # no multiple of the group
    assert qkv(lib, d=dict(BASE, rope_theta=0.0)) == DIMS
    assert out_proj(lib, d_model=264) == UNSUPPORTED          # rows in tiles of 16
    assert out_proj(lib, group=128, d=dict(BASE, num_q_heads=3, num_kv_heads=3)) == UNSUPPORTED


def test_binding_refuses_tensors_that_are_not_on_a_gpu():
    i, x = torch.zeros(64, dtype=torch.int32), torch.zeros((1, 64), dtype=torch.bfloat16)
    for f in (lambda: binding.gist_attn_paged_decode(x, x, i, i, dims=BASE), lambda: binding.gist_pages_free(i, i, dims=BASE),
              lambda: binding.gist_pages_compact(i, i, dims=BASE), lambda: binding.gist_pages_fork(i, i, i, i, i, dims=BASE),
              lambda: binding.gist_pages_copy(x, None, i, i, dims=BASE),
              lambda: binding.gist_qkv_rope_w4(x, i, x, i, group=64, dims=BASE),
              lambda: binding.gist_out_proj_w4(x, i, x, group=64, dims=BASE)):
        with pytest.raises(TypeError, match="CUDA"):
            f()
    with pytest.raises(TypeError, match="torch tensor"):
        binding.gist_pages_free(i, None, dims=BASE)


# ------------------------------------------------ the definitions themselves


def test_attention_definition_against_torch():
    pb = su.Decode([37, 0, 16], 4, 2, 64, 16, seed=1, device="cpu")
    got, tol = pb.expected(rotated=True)
    assert not got[1].any()
    for r in (0, 2):
        C = pb.lens[r]
        ids = pb.table[r, :-(-C // 16)]
        k, v = pb.pool[ids, 1].double().permute(1, 2, 0, 3, 4).reshape(2, 2, -1, 64)[:, :, :C].repeat_interleave(2, 1)
        o = torch.nn.functional.scaled_dot_product_attention(pb.q[r].double()[None, :, None], k[None], v[None])[0, :, 0]
        np.testing.assert_allclose(got[r], o.numpy(), atol=1e-12)
        assert (tol[r] < 0.05).all()


def test_page_definitions_by_hand():
    table = np.array([[4, 2, 9], [4, 2, 0], [7, 7, 7]])
    f = su.free([33, 17, 0], table, 16, 10)
    assert f["ref_count"].tolist() == [0, 0, 2, 0, 2, 0, 0, 0, 0, 1] and f["free_range"].tolist() == [0, 7]
    c = su.compact([33, 17, 0], table, 16, 10)
    assert c["block_table"].tolist() == [[0, 2, 1], [0, 2, 0], [7, 7, 7]]
    assert c["copy_src"].tolist() == [4, 9, -1, -1, -1] and c["copy_dst"].tolist() == [0, 1, -1, -1, -1]
    k = su.fork([33, 17, 0], [-1, -1, 0], table, [5, 6], [1, 2], 16, 10)
    assert k["block_table"].tolist() == [[4, 2, 9], [4, 2, 0], [4, 2, 6]] and k["cached_len"].tolist() == [33, 17, 33]
    assert (k["copy_src"][0], k["copy_dst"][0], k["copy_rows"][0], k["free_range"].tolist()) == (9, 6, 1, [2, 2])


def test_packed_weights_by_hand():
    assert su.pack(np.array([[1, 2, 15, 0]])).tolist() == [[0x21, 0x0F]]
    w = su.W4(4, 64, 32, seed=3)
    x = np.random.default_rng(0).standard_normal((2, 64))
    code = np.stack([w.w.numpy() & 15, w.w.numpy() >> 4], -1).reshape(4, 64).astype(float) - 8
    want = sum((x[:, 32 * g:32 * g + 32] @ code[:, 32 * g:32 * g + 32].T) * w.scale.double().numpy()[:, g] for g in range(2))
    np.testing.assert_allclose(w.times(x)[0], want, rtol=1e-12)


def test_out_proj_refuses_more_inputs_than_it_stages(lib):
    """K = Hq d up to 65536, for any number of tokens."""
    for T in (1, 8, 64):
        assert out_proj(lib, d=dict(BASE, num_tokens=T, num_q_heads=1026, num_kv_heads=2)) == UNSUPPORTED  # 1026 heads of 64
        assert out_proj(lib, d=dict(BASE, num_tokens=T, num_q_heads=1024, num_kv_heads=2), w=0) == NULL
