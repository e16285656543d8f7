"""Attention of single tokens over a bf16 paged cache is as exact as fp32 arithmetic is: how many of
its outputs are not the bf16 that the definition in 64 bits rounds to."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import serving_utils as su
from attention_cached_kv_gb300 import binding
from paged_utils import rotate

pytestmark = pytest.mark.gpu
DEV = "cuda"
LENS = [300, 4000, 9000, 2500, 1000, 77]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    binding.load_library()
    yield
    torch.cuda.empty_cache()


def exact(pb):
    """[B][Hq][d] in 64 bits."""
    d, out = pb.q.shape[-1], torch.zeros(pb.q.shape, dtype=torch.float64, device=DEV)
    for r, C in enumerate(pb.lens):
        q = torch.from_numpy(rotate(pb.q[r:r + 1].double().numpy(), np.array([C - 1])))[0].to(DEV)
        rows = pb.pool[torch.tensor(pb.table[r, :-(-C // pb.bl)]), pb.layer].double().to(DEV)
        for g in range(rows.shape[2]):
            k, v = (rows[:, i, g].reshape(-1, d)[:C] for i in (0, 1))
            h = slice(g * pb.G, (g + 1) * pb.G)
            out[r, h] = torch.softmax(q[h] @ k.T / math.sqrt(d), -1) @ v
    return out


# An output rounds the other way than the exact value where its error passes the value's distance from
# the next midpoint of two bf16, for a share of about (error / step) of outputs; a step is 2^-8 to
# 2^-7 of the value, 0.0055 of it on average, and outputs being sums of both signs the mean of their
# size over a value is about 4.  fp32 arithmetic leaves a weight off by 2^-24 of its score a rounding,
# of which a score (additions of the products, scale, difference from the maximum) has some three that count,
# and 2^-22 for the exponential: scores reach about 5 times the spread of q, so
#   spread 1:  3 x 5 x 2^-24 + 2^-22 = 1.1e-6, a share of 0.08 %;   spread 4:  3.8e-6, 0.28 %.
# The share of n elements is a count with its own scatter: about sqrt(n share) for events that
# do not depend on each other, of which three are allowed (5 of 6144 where 4.9 are expected says nothing).
# Operands of 17 bits are off by 2^-17 / sqrt(12) in each weight and by as much of each of q's products:
# 0.3 % and 0.5 %, which the sum over all layouts (119 k elements: 0.10 and 0.33 % allowed) tells apart.
LAYOUTS = [(8, 8, 128), (16, 8, 64), (24, 8, 128), (16, 4, 64), (14, 2, 64), (32, 4, 128), (32, 2, 64), (32, 2, 128), (40, 2, 64)]
SHARES = [(1.0, 0.0008), (4.0, 0.0028)]


def turned(Hq, Hkv, d, spread):
    """How many outputs are not the exact value's bf16, and of how many."""
    pb = su.Decode(LENS, Hq, Hkv, d, 64, seed=Hq + d, spread=spread)
    got = binding.gist_attn_paged_decode(*pb.args(), dims=pb.dims)
    ref, tol = (torch.from_numpy(x) for x in pb.expected())
    assert ((got.cpu().double() - ref).abs() <= tol).all()
    return int((got != exact(pb).to(torch.bfloat16)).sum()), got.numel()


@pytest.mark.parametrize("Hq,Hkv,d", LAYOUTS)
@pytest.mark.parametrize("spread,most", SHARES)
def test_outputs_that_round_the_other_way(Hq, Hkv, d, spread, most):
    count, n = turned(Hq, Hkv, d, spread)
    assert count <= n * most + 3 * math.sqrt(n * most)


@pytest.mark.parametrize("spread,most", SHARES)
def test_over_all_layouts(spread, most):
    counts = [turned(*h, spread) for h in LAYOUTS]
    count, n = sum(c for c, _ in counts), sum(m for _, m in counts)
    assert count <= n * most + 3 * math.sqrt(n * most)
