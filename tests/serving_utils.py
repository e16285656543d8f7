"""Definitions of the single-token step over a bf16 paged cache, of the cache's blocks and of
the 4-bit projections, in 64 bits on the CPU, with seeded problems for their tests."""
from __future__ import annotations

import math

import numpy as np
import torch

from paged_utils import THETA, rotate

BF16 = 2.0 ** -8  # half a step, relative


def bf16(x):
    return torch.from_numpy(np.asarray(x)).to(torch.bfloat16)


class Decode:
    """A seeded bf16 cache with requests of the given lengths in it (the new token among them)."""

    def __init__(self, lens, Hq, Hkv, d, bl, seed=0, layers=2, layer=1, extra_width=0, spread=1.0, device="cuda"):
        rng = np.random.default_rng(seed)
        self.lens, self.bl, self.G, self.layer, self.device = list(lens), bl, Hq // Hkv, layer, device
        n = [-(-max(t, 0) // bl) for t in lens]
        W, nb = max([1] + n) + extra_width, sum(n) + 3
        perm, at = rng.permutation(nb), 0
        self.table = np.full((len(lens), W), -7, np.int64)  # entries past a request's blocks name nothing
        for r, k in enumerate(n):
            self.table[r, :k] = perm[at:at + k]
            at += k
        g = torch.Generator().manual_seed(seed)
        self.pool = torch.randn((nb, layers, 2, Hkv, bl, d), generator=g).to(torch.bfloat16)
        for r, t in enumerate(lens):  # rows past the length: never seen
            if t > 0 and t % bl:
                self.pool[self.table[r, t // bl], :, :, :, t % bl:] = math.nan
        self.q = (torch.randn((len(lens), Hq, d), generator=g) * spread).to(torch.bfloat16)
        self.dims = dict(num_requests=len(lens), num_tokens=len(lens), max_new=1, num_q_heads=Hq, num_kv_heads=Hkv, head_dim=d,
                         block_len=bl, max_blocks=W, num_blocks=nb, num_layers=layers, layer=layer, rope_theta=THETA,
                         softmax_scale=0.0)

    def i32(self, x):
        return torch.tensor(np.asarray(x), dtype=torch.int32, device=self.device)

    def args(self):
        """q, pool, table, kv_len on the device."""
        return self.q.to(self.device), self.pool.to(self.device), self.i32(self.table), self.i32(self.lens)

    def expected(self, rotated=False):
        return attend(self.q.double().numpy(), self.pool[:, self.layer].double().numpy(), self.table, self.lens, self.bl,
                      self.G, rotated, self.dims["softmax_scale"] or None)


def attend(q, pool, table, lens, bl, G, rotated=False, scale=None):
    """out [B][Hq][d] and how far it may be off.  Of a head's scores each is off by 2^-17 of
    sum |q_i k_i| (q kept to 17 bits), as much again for the 128 fp32 additions; its weight by
    that and 2^-15 (exponential, 16 bits of P, the sums); the result is rounded once."""
    B, Hq, d = q.shape
    out, tol = np.zeros(q.shape), np.zeros(q.shape)
    sc = scale or 1 / math.sqrt(d)
    for r, C in enumerate(lens):
        if C <= 0:
            continue
        ids = table[r, :-(-C // bl)]
        x = q[r:r + 1] if rotated else rotate(q[r:r + 1], np.array([C - 1]))
        for h in range(Hq):
            k = pool[ids, 0, h // G].reshape(-1, d)[:C]
            v = pool[ids, 1, h // G].reshape(-1, d)[:C]
            s = k @ x[0, h] * sc
            w = np.exp(s - s.max())
            w /= w.sum()
            out[r, h] = w @ v
            off = 2.0 ** -16 * sc * (np.abs(k) @ np.abs(x[0, h])).max()
            tol[r, h] = (2 * off + 2.0 ** -15) * (w @ np.abs(v)) + BF16 * np.abs(out[r, h]) * 1.01
    return out, tol


def near(got, ref, tol, what=""):
    got = got.float().cpu().numpy().astype(np.float64)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.abs(got - ref)[bad].max():.3e}"


# --------------------------------------------------------------- the blocks


def blocks(length, bl, W):
    """Live entries of a row."""
    return min(W, -(-length // bl)) if length > 0 else 0


def free(cached, table, bl, nb):
    """ref_count, free_blocks, free_range, status."""
    ref, status = np.zeros(nb, np.int64), 0
    W = table.shape[1]
    for r, c in enumerate(cached):
        if c > W * bl:
            status |= 1
        for j in range(blocks(c, bl, W)):
            b = table[r, j]
            if 0 <= b < nb:
                ref[b] += 1
            else:
                status |= 1
    ids = np.flatnonzero(ref == 0)
    return dict(ref_count=ref, free_blocks=padded(ids, nb), free_range=np.array([0, len(ids)]), status=status)


def padded(x, n):
    return np.concatenate([np.asarray(x, np.int64), np.full(n - len(x), -1, np.int64)])


def compact(cached, table, bl, nb):
    f = free(cached, table, bl, nb)
    used = np.flatnonzero(f["ref_count"])
    n, W = len(used), table.shape[1]
    src, dst = [b for b in used if b >= n], sorted(set(range(n)) - set(used.tolist()))
    name = {int(b): int(b) for b in used} | dict(zip([int(b) for b in src], dst))
    out = table.copy()
    for r, c in enumerate(cached):
        for j in range(blocks(c, bl, W)):
            out[r, j] = name.get(int(table[r, j]), table[r, j])
    return dict(block_table=out, new_id=np.array([name.get(b, -1) for b in range(nb)]), copy_src=padded(src, nb // 2),
                copy_dst=padded(dst, nb // 2), num_copies=np.array([len(src)]), free_blocks=padded(np.arange(n, nb), nb),
                free_range=np.array([0, nb - n]), status=f["status"])


def fork(cached, parent, table, free_blocks, free_range, bl, nb):
    B, W = table.shape
    table, length, status = table.copy(), np.array(cached), 0
    begin, end = max(free_range[0], 0), max(min(free_range[1], len(free_blocks)), 0)
    asked, src, dst, rows = 0, [], [], []
    forks = [p >= 0 and p != r for r, p in enumerate(parent)]
    for r, p in enumerate(parent):
        if not forks[r]:
            continue
        length[r] = 0
        if p >= B or forks[p] or not 0 <= cached[p] <= W * bl:
            status |= 8
            continue
        full, part = divmod(int(cached[p]), bl)
        if part:
            asked += 1
            if asked > end - begin:
                status |= 8
                continue
            a, b = int(table[p, full]), int(free_blocks[begin + asked - 1])
            if not (0 <= a < nb and 0 <= b < nb):
                status |= 1
                src.append(-1), dst.append(-1), rows.append(-1)
                continue
            src.append(a), dst.append(b), rows.append(part)
            table[r, full] = b
        table[r, :full] = table[p, :full]
        length[r] = cached[p]
    return dict(block_table=table, cached_len=length, copy_src=padded(src, B), copy_dst=padded(dst, B), copy_rows=padded(rows, B),
                num_copies=np.array([len(src)]), free_range=np.array([max(free_range[0], 0) + len(src), free_range[1]]), status=status)


def same(got: dict, want: dict):
    for k, v in want.items():
        if k != "status":
            assert np.array_equal(got[k].cpu().numpy().reshape(-1), np.asarray(v).reshape(-1)), k


# --------------------------------------------------------------- 4-bit projections


def pack(code):
    """Codes 0..15 [N][K] as bytes [N][K / 2], the even input in the low four bits."""
    return torch.from_numpy((code[:, 0::2] | code[:, 1::2] << 4).astype(np.uint8))


class W4:
    """Seeded weights [N][K]: packed codes, bf16 scales, and their values."""

    def __init__(self, N, K, group, seed=0):
        rng = np.random.default_rng(seed)
        code = rng.integers(0, 16, (N, K))
        self.w = pack(code)
        self.scale = bf16(rng.uniform(0.5, 1.5, (N, K // group)) / math.sqrt(K) / 4)
        self.value = (code - 8) * np.repeat(self.scale.double().numpy(), group, axis=1)

    def times(self, x):
        """x [T][K] w^T and how far fp32 sums may be off: a value goes through at most 128 additions
        in its group's MMAs, K / 32 of the groups' sums and 64 of the parts', each off by a
        step (2^-23: tensor cores may cut off) of the sum of magnitudes at most."""
        K = x.shape[1]
        return x @ self.value.T, (192 + K / 32) * 2.0 ** -23 * (np.abs(x) @ np.abs(self.value).T)


def rotated(y, off, position):
    """y [T][heads][d] turned, and the turned bound: each result has both values of its pair."""
    half = y.shape[-1] // 2
    both = np.abs(y) * 2.0 ** -22 + off  # sine and cosine to fp32
    pair = np.concatenate([both[..., half:], both[..., :half]], -1)
    return rotate(y, position), both + pair
