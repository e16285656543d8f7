"""The ragged serving step's definitions in 64 bits on the CPU (numpy loops over
requests, tokens and blocks), and seeded problems for its tests."""
from __future__ import annotations

import math

import numpy as np
import torch

THETA = 1e4


def e4m3_values() -> np.ndarray:
    """The value of each of the 256 E4M3 codes, from the format's definition."""
    out = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        out[c] = math.nan if (c & 127) == 127 else -v if c >> 7 else v
    return out


E4M3 = e4m3_values()


def encode(x: np.ndarray) -> np.ndarray:
    """Nearest E4M3 codes of |x| <= 448 (ties to the even code); non-finite to NaN."""
    grid = E4M3[:127]
    a = np.abs(np.where(np.isfinite(x), x, 0.0))
    hi = np.minimum(np.searchsorted(grid, a), 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - grid[lo], grid[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi).astype(np.uint8)
    return np.where(np.isfinite(x), code | np.where(np.signbit(x), 128, 0).astype(np.uint8), 127).astype(np.uint8)


def rotate(x: np.ndarray, position: np.ndarray, theta: float = THETA) -> np.ndarray:
    """x [n][heads][d] turned at its positions: pairs (j, j + d/2), theta^(-2j/d)."""
    half = x.shape[-1] // 2
    ang = np.asarray(position, dtype=np.float64)[:, None] * theta ** (-np.arange(half) / half)
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
    a, b = x[..., :half], x[..., half:]
    return np.concatenate([a * c - b * s, b * c + a * s], -1)


def plan(cached, new, table, free, free_range, T, bl, num_blocks):
    """The plan's outputs, request by request; status bits as the last."""
    table = table.copy()
    W = table.shape[1]
    slot, position = np.full(T, -1, np.int64), np.full(T, -1, np.int64)
    begin, end = max(free_range[0], 0), min(free_range[1], len(free))
    avail, asked, taken, row, status = max(end - begin, 0), 0, 0, 0, 0
    q_start, kv_len = [], []
    for r, (c, n) in enumerate(zip(cached, new)):
        q_start.append(min(row, T))
        valid = c >= 0 and n >= 0 and c + n <= W * bl
        have, want = (-(-c // bl), -(-(c + n) // bl)) if valid else (0, 0)
        asked += want - have
        m = max(n, 0)
        ok = valid and row + m <= T and (want == have or asked <= avail)
        if ok:
            for b in range(have, want):
                table[r, b] = free[begin + taken]
                taken += 1
            for i in range(n):
                pos = c + i
                blk = table[r, pos // bl]
                position[row + i] = pos
                if 0 <= blk < num_blocks:
                    slot[row + i] = blk * bl + pos % bl
                else:
                    status |= 1
        else:
            status |= 8
        kv_len.append(c + n if ok else 0)
        row += m
    q_start.append(min(row, T))
    return dict(block_table=table, q_start=np.array(q_start), kv_len=np.array(kv_len), slot=slot, position=position,
                free_range=np.array([max(free_range[0], 0) + taken, free_range[1]]), status=status)


def pow2_scale(top: float, limit: float) -> float:
    if top == 0:
        return 2.0 ** -100
    e = math.ceil(math.log2(top / limit))
    while top > limit * 2.0 ** e:
        e += 1
    while top <= limit * 2.0 ** (e - 1):
        e -= 1
    return 2.0 ** min(max(e, -100), 119)


def append(k, v, codes, scale, slot, position, bl, layer, rotated=False):
    """New codes and scales of pool codes [nb][L][2][Hkv][bl][d] after the write."""
    codes, scale = codes.copy(), scale.astype(np.float64).copy()
    slot = np.asarray(slot)
    t = 0
    while t < len(slot):
        if slot[t] < 0:
            t += 1
            continue
        blk, off = divmod(int(slot[t]), bl)
        n, last = 1, 1  # entries of the block: skipped ones (< 0) keep their place
        while t + n < len(slot) and off + n < bl and (slot[t + n] < 0 or slot[t + n] == slot[t] + n):
            n += 1
            last = n if slot[t + n - 1] >= 0 else last
        n = last
        live = slot[t:t + n] >= 0
        rest = np.concatenate([np.arange(off), off + np.flatnonzero(~live)])
        for kv, x in enumerate((k, v)):
            turn = kv == 0 and not rotated
            for g in range(k.shape[1]):
                rows = x[t:t + n, g][live]
                fin = np.abs(rows[np.isfinite(rows)])
                need = pow2_scale(float(fin.max()) if fin.size else 0.0, 316.0 if turn else 448.0)
                old = scale[blk, layer, kv, g]
                s = need if off == 0 else max(old, need)
                if off and s > old:
                    codes[blk, layer, kv, g, rest] = encode(E4M3[codes[blk, layer, kv, g, rest]] * (old / s))
                scale[blk, layer, kv, g] = s
                with np.errstate(invalid="ignore"):
                    y = rotate(rows[:, None] / s, position[t:t + n][live])[:, 0] if turn else rows / s
                new = encode(np.where(np.isfinite(y), np.clip(y, -448, 448), y))
                codes[blk, layer, kv, g, off + np.flatnonzero(live)] = new
        t += n
    return codes, scale


def attend(q, codes, scale, table, q_start, kv_len, bl, layer, G, rotated=False, softmax_scale=None):
    """Attention over the cache in 64 bits; NaN rows where nothing is written."""
    out = np.full(q.shape, np.nan)
    d = q.shape[-1]
    sc = softmax_scale or 1 / math.sqrt(d)
    for r in range(len(kv_len)):
        a, b, C = q_start[r], q_start[r + 1], kv_len[r]
        if a == b:
            continue
        nb = -(-C // bl)
        ids = table[r, :nb]
        pos = C - (b - a) + np.arange(b - a)
        x = q[a:b] if rotated else rotate(q[a:b], pos)
        for h in range(q.shape[1]):
            g = h // G
            kk = (E4M3[codes[ids, layer, 0, g]] * scale[ids, layer, 0, g][:, None, None]).reshape(-1, d)[:C]
            vv = (E4M3[codes[ids, layer, 1, g]] * scale[ids, layer, 1, g][:, None, None]).reshape(-1, d)[:C]
            for i, p in enumerate(pos):
                if p < 0:
                    out[a + i, h] = 0.0
                    continue
                s = kk[:p + 1] @ x[i, h] * sc
                w = np.exp(s - s.max())
                out[a + i, h] = (w / w.sum()) @ vv[:p + 1]
    return out


class Problem:
    """A seeded cache with requests in it (device tensors), all tokens already written."""

    def __init__(self, cached, new, Hq, Hkv, d, bl, seed=0, device="cuda", pad=0, layers=2, layer=1, spread=2,
                 extra_width=0):
        rng = np.random.default_rng(seed)
        B = len(cached)
        total = [c + n for c, n in zip(cached, new)]
        self.cached, self.new, self.bl, self.G, self.layer = cached, new, bl, Hq // Hkv, layer
        self.T = sum(new) + pad
        W = max([1] + [-(-t // bl) for t in total]) + extra_width
        nb = sum(-(-t // bl) for t in total) + 3
        perm = rng.permutation(nb)
        self.table = np.full((B, W), -7, np.int64)  # entries past a request's blocks name nothing
        at = 0
        for r, t in enumerate(total):
            n = -(-t // bl)
            self.table[r, :n] = perm[at:at + n]
            at += n
        self.codes = encode(np.clip(rng.standard_normal((nb, layers, 2, Hkv, bl, d)) * 100, -448, 448))
        self.scale = 2.0 ** -rng.integers(6, 7 + spread, (nb, layers, 2, Hkv)).astype(np.float64)
        self.q_start = np.concatenate([[0], np.cumsum(new)])
        self.kv_len = np.array(total)
        self.q = torch.from_numpy(rng.standard_normal((self.T, Hq, d))).to(torch.bfloat16)
        self.dims = dict(num_requests=B, num_tokens=self.T, max_new=max(list(new) + [1]), num_q_heads=Hq, num_kv_heads=Hkv,
                         head_dim=d, block_len=bl, max_blocks=W, num_blocks=nb, num_layers=layers, layer=layer,
                         rope_theta=THETA, softmax_scale=0.0)
        self.device = device

    def i32(self, x):
        return torch.tensor(np.asarray(x), dtype=torch.int32, device=self.device)

    def args(self):
        """q, pool, scale, table, q_start, kv_len on the device."""
        return (self.q.to(self.device), torch.from_numpy(self.codes).to(self.device),
                torch.from_numpy(self.scale).float().to(self.device), self.i32(self.table), self.i32(self.q_start),
                self.i32(self.kv_len))

    def expected(self, rotated=False, softmax_scale=None):
        return attend(self.q.double().numpy(), self.codes, self.scale.astype(np.float32).astype(np.float64), self.table,
                      self.q_start, self.kv_len, self.bl, self.layer, self.G, rotated, softmax_scale)
