"""Cases of the ragged serving step over an E4M3 paged cache.

Three operators, used one after another in every decoding or chunked-prefill
step of a server whose requests have lengths of their own:

  plan    from the requests' cached lengths and new-token counts, on the device:
          blocks for the new tokens out of a free list, the block table, the
          slot and the position of every token
  append  the new tokens' keys (rotated) and values into the E4M3 pool at their
          slots, with the scale of each block and KV head kept large enough
  attn    causal attention of each request's new tokens over its cached
          sequence, read through the block table

``run`` computes a case in its plain form (elementary torch operations) or, with
``own`` set, through the framework's entry points.  ``exact`` gives the same
outputs from the definitions in 64 bits.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DEV = "cuda"
THETA = 1e4
LAYERS, LAYER = 2, 1  # the pool holds two layers; the calls work on the second


def _plan(name, batch, cached, new, block_len):
    return {"name": name, "op": "plan", "batch": batch, "cached": cached, "new_lo": new[0],
            "new_hi": new[1], "block_len": block_len}


def _append(name, batch, cached, new, heads, dim, block_len):
    return {"name": name, "op": "append", "batch": batch, "cached": cached, "new_lo": new[0],
            "new_hi": new[1], "kv_heads": heads, "dim": dim, "block_len": block_len}


def _attn(name, batch, cached, new, heads, dim, block_len):
    return {"name": name, "op": "attn", "batch": batch, "cached_lo": cached[0], "cached_hi": cached[1],
            "new_lo": new[0], "new_hi": new[1], "q_heads": heads[0], "kv_heads": heads[1], "dim": dim,
            "block_len": block_len}


def listed():
    return [
        # one decoding step of a small batch: pure latency
        _plan("plan decode 32", 32, 4096, (1, 1), 256),
        # a step that mixes decoding requests with prompt chunks, small blocks
        _plan("plan mixed 500", 500, 2000, (0, 257), 16),
        # a large batch of prompts, as an offline pass over many documents makes it
        _plan("plan prompts 2048", 2048, 300, (1, 255), 32),
        # the decoding step's write: one token for each of 64 requests
        _append("append decode 64", 64, 4000, (1, 1), 8, 128, 256),
        # prompt chunks of the small model (2 KV heads of 64), blocks of 16
        _append("append chunks d64", 24, 500, (100, 500), 2, 64, 16),
        # a long prompt chunk for each of 8 requests, 8 KV heads of 128
        _append("append prompts d128", 8, 4096, (1500, 2048), 8, 128, 64),
        # four short conversations on the small model: latency
        _attn("attn decode short", 4, (17, 200), (1, 1), (14, 2), 64, 16),
        # the paged decode with grouped heads, lengths spread around 4096
        _attn("attn decode gqa 32", 32, (2500, 5600), (1, 1), (32, 8), 128, 256),
        # the same with a KV head for every query head
        _attn("attn decode mha 32", 32, (2500, 5600), (1, 1), (32, 32), 128, 256),
        # one long document: few rows, a long axis
        _attn("attn decode one long", 1, (131000, 131000), (1, 1), (14, 2), 64, 64),
        # drafted tokens checked for 16 requests at once
        _attn("attn verify 16", 16, (500, 3000), (2, 5), (32, 8), 128, 32),
        # prompt chunks behind a cached context, with the last chunk ragged
        _attn("attn chunks 4", 4, (1000, 6000), (700, 1024), (32, 8), 128, 64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "append", "attn", "attn"])
    block_len = rng.choice([16, 32, 64, 128, 256])
    if op == "plan":
        lo = rng.randint(0, 1)
        c = _plan("", _log(rng, 1, 2048), _log(rng, 16, 8000), (lo, max(lo, _log(rng, 1, 250))), block_len)
    elif op == "append":
        heads, dim = rng.choice([(2, 64), (8, 128), (4, 64), (32, 128)])
        batch = _log(rng, 1, 128)
        hi = _log(rng, 1, max(1, min(2000, 80000 // (batch * heads))))
        c = _append("", batch, _log(rng, 8, 4000), (max(1, hi // 2), hi), heads, dim, block_len)
    else:
        q_heads, kv_heads, dim = rng.choice([(14, 2, 64), (32, 8, 128), (32, 32, 128), (16, 4, 64)])
        kind = rng.choice(["decode", "decode", "verify", "chunks"])
        if kind == "chunks":
            batch, hi = _log(rng, 1, 4), _log(rng, 20, 1000)
            new, cached = (hi // 2, hi), _log(rng, 16, 5000)
        else:
            batch = _log(rng, 1, 64)
            new = (1, 1) if kind == "decode" else (1, rng.randint(2, 6))
            cached = _log(rng, 16, 260000 // (batch * kv_heads))
        c = _attn("", batch, (cached // 2, cached), new, (q_heads, kv_heads), dim, block_len)
    del c["name"]
    return c


def _lengths(case):
    """Cached and new tokens of each request: the same for every seed, so that the work is."""
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    B, op = case["batch"], case["op"]
    lo, hi = (case["cached_lo"], case["cached_hi"]) if op == "attn" else (0, case["cached"])
    cached = [rng.randint(lo, hi) for _ in range(B)]
    new = [rng.randint(case["new_lo"], case["new_hi"]) for _ in range(B)]
    if op == "plan" and B > 2:
        cached[1] = 0  # a request that starts
    return cached, new


def _generator(seed, stream):
    return torch.Generator(device=DEV).manual_seed(16 * int(seed) + stream)


def _e4m3(shape, seed, stream):
    """E4M3 values of normal deviates filling the type's range, as a scaled cache holds them."""
    out = torch.empty(shape, dtype=torch.float8_e4m3fn, device=DEV)
    flat, g, step = out.view(-1), _generator(seed, stream), 1 << 28
    for a in range(0, flat.numel(), step):
        n = min(step, flat.numel() - a)
        flat[a:a + n] = (torch.randn(n, generator=g, device=DEV) * 100.0).clamp_(-448, 448).to(torch.float8_e4m3fn)
    return out


def prepare(case, seed):
    case = dict(case)
    cached, new = _lengths(case)
    B, bl = case["batch"], case["block_len"]
    total = [c + n for c, n in zip(cached, new)]
    T = sum(new)
    width = max(1, -(-max(total) // bl)) + 1
    used = torch.tensor([-(-(c if case["op"] == "plan" else t) // bl) for c, t in zip(cached, total)], device=DEV)
    num_blocks = sum(-(-t // bl) for t in total) + 7
    i32 = dict(dtype=torch.int32, device=DEV)
    perm = torch.randperm(num_blocks, generator=_generator(seed, 0), device=DEV).to(torch.int32)
    ahead = torch.cumsum(used, 0) - used
    col = torch.arange(width, device=DEV)
    table = torch.where(col < used[:, None], perm[(ahead[:, None] + col).clamp(max=num_blocks - 1)], -1).to(torch.int32)
    s = {"case": case, "B": B, "T": T, "bl": bl, "num_blocks": num_blocks, "width": width,
         "cached_len": torch.tensor(cached, **i32), "new_len": torch.tensor(new, **i32), "block_table": table.contiguous()}
    s["dims"] = dict(num_requests=B, num_tokens=T, max_new=max(new), num_q_heads=case.get("q_heads", case.get("kv_heads", 1)),
                     num_kv_heads=case.get("kv_heads", 1), head_dim=case.get("dim", 64), block_len=bl, max_blocks=width,
                     num_blocks=num_blocks, num_layers=LAYERS, layer=LAYER, rope_theta=THETA, softmax_scale=0.0)
    s["q_start"] = torch.cat([torch.zeros(1, **i32), torch.cumsum(s["new_len"], 0).to(torch.int32)])
    s["kv_len"] = s["cached_len"] + s["new_len"]
    if case["op"] == "plan":
        n_used = int(used.sum())
        s["free_blocks"] = perm.clone()
        s["free_range"] = torch.tensor([n_used, num_blocks], **i32)
        s["plan"] = [torch.empty(n, **i32) for n in (B + 1, B, T, T, 2)]  # a server's own buffers
        return s
    Hkv, d = case["kv_heads"], case["dim"]
    s["pool"] = _e4m3((num_blocks, LAYERS, 2, Hkv, bl, d), seed, 1)
    s["scale"] = torch.exp2(torch.randint(-8, -5, (num_blocks, LAYERS, 2, Hkv), generator=_generator(seed, 2), device=DEV).float())
    request = torch.repeat_interleave(torch.arange(B, device=DEV), s["new_len"].long())
    position = torch.arange(T, device=DEV) - s["q_start"].long()[request] + s["cached_len"].long()[request]
    s["position"] = position.to(torch.int32)
    s["slot"] = (table.long()[request, position // bl] * bl + position % bl).to(torch.int32)
    if case["op"] == "append":
        s["k"] = torch.randn((T, Hkv, d), generator=_generator(seed, 3), device=DEV).to(torch.bfloat16)
        s["v"] = torch.randn((T, Hkv, d), generator=_generator(seed, 4), device=DEV).to(torch.bfloat16)
    else:
        s["q"] = torch.randn((T, case["q_heads"], d), generator=_generator(seed, 5), device=DEV).to(torch.bfloat16)
        s["out"] = torch.empty_like(s["q"])
        s["workspace"] = torch.empty(64 << 20, dtype=torch.uint8, device=DEV)
    return s


# ------------------------------------------------------------- the plain forms


def _plain_plan(s):
    bl, T, W = s["bl"], s["T"], s["width"]
    cached, new = s["cached_len"].long(), s["new_len"].long()
    begin, end = s["free_range"].long()
    have = (cached + bl - 1) // bl
    need = (cached + new + bl - 1) // bl - have
    before = torch.cumsum(need, 0) - need
    served = (need == 0) | (before + need <= end - begin)
    kv_len = torch.where(served, cached + new, 0)
    q_start = torch.cat([torch.zeros(1, dtype=torch.long, device=DEV), torch.cumsum(new, 0)])
    col = torch.arange(W, device=DEV)
    fresh = served[:, None] & (col >= have[:, None]) & (col < (have + need)[:, None])
    take = (begin + before[:, None] + col - have[:, None]).clamp(0, s["num_blocks"] - 1)
    s["block_table"].copy_(torch.where(fresh, s["free_blocks"][take], s["block_table"]))
    t = torch.arange(T, device=DEV)
    r = torch.searchsorted(q_start[1:].contiguous(), t, right=True).clamp(max=s["B"] - 1)
    position = cached[r] + t - q_start[r]
    block = s["block_table"].long()[r, (position // bl).clamp(max=W - 1)]
    ok = served[r]
    slot = torch.where(ok, block * bl + position % bl, -1)
    taken = torch.where(served, need, 0).sum()
    return {"block_table": s["block_table"], "q_start": q_start.int(), "kv_len": kv_len.int(), "slot": slot.int(),
            "position": torch.where(ok, position, -1).int(), "free_range": torch.stack([begin + taken, end]).int()}


def _rotate(x, position, dtype):
    """Rotate-half pairs (j, j + d/2) at theta^(-2j/d), the angles in 64 bits."""
    half = x.shape[-1] // 2
    freq = THETA ** (-torch.arange(half, device=x.device, dtype=torch.float64) / half)
    angle = position.double()[:, None] * freq
    cos, sin = torch.cos(angle)[:, None].to(dtype), torch.sin(angle)[:, None].to(dtype)
    x = x.to(dtype)
    a, b = x[..., :half], x[..., half:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _pow2_scale(amax, most):
    """The smallest power of two s with amax <= most * s (most: 448 = 0.875 * 2^9, or 316)."""
    m, e = torch.frexp(amax)
    e = torch.where(m <= most / 512.0, e - 9, e - 8)
    return torch.where(amax > 0, torch.exp2(e.clamp(-100, 119).float()), torch.exp2(torch.full_like(amax, -100.0)))


def _plain_append(s):
    bl, n = s["bl"], s["num_blocks"]
    pool, scale, slot = s["pool"], s["scale"], s["slot"].long()
    blk, off = slot // bl, slot % bl
    Hkv = pool.shape[3]
    amax = torch.stack([s["k"].float().abs().amax(-1), s["v"].float().abs().amax(-1)], 1)  # [T][2][Hkv]
    top = torch.zeros((n, 2, Hkv), device=DEV).index_reduce(0, blk, amax, "amax")
    first = torch.full((n,), bl, device=DEV).index_reduce(0, blk, off, "amin")
    need = torch.stack([_pow2_scale(top[:, 0], 316.0), _pow2_scale(top[:, 1], 448.0)], 1)
    old = scale[:, LAYER].clone()
    now = torch.where((first == 0)[:, None, None], need, torch.maximum(old, need))
    now = torch.where((first < bl)[:, None, None], now, old)
    # the block that each request's first new token shares with its cached ones
    head = blk[s["q_start"][:-1].long()]
    rows = pool[head, LAYER].float()
    keep = rows * (old[head] / now[head])[..., None, None]
    before = torch.arange(bl, device=DEV) < first[head][:, None]
    rows = torch.where(before[:, None, None, :, None], keep, rows).to(torch.float8_e4m3fn)
    raw = pool.view(torch.uint8)
    raw[head, LAYER] = rows.view(torch.uint8)
    k = _rotate(s["k"], s["position"], torch.float32) / now[blk, 0][..., None]
    v = s["v"].float() / now[blk, 1][..., None]
    new = torch.stack([k, v], 1).to(torch.float8_e4m3fn).view(torch.uint8)  # [T][2][Hkv][d]
    raw[blk, LAYER, :, :, off] = new
    scale[:, LAYER] = now
    return {"pool": pool, "scale": scale}


def _plain_attn(s):
    case = s["case"]
    B, T, bl, W = s["B"], s["T"], s["bl"], s["width"]
    Hq, Hkv, d = case["q_heads"], case["kv_heads"], case["dim"]
    G, N = Hq // Hkv, case["new_hi"]
    table = s["block_table"].clamp(min=0).long()
    kv = s["pool"].view(torch.uint8)[:, LAYER][table].view(torch.float8_e4m3fn).float()  # [B][W][2][Hkv][bl][d]
    kv = kv * s["scale"][:, LAYER][table][..., None, None]
    k, v = kv.permute(2, 0, 3, 1, 4, 5).reshape(2, B, Hkv, W * bl, d)
    start, new, length = s["q_start"][:-1].long(), s["new_len"].long(), s["kv_len"].long()
    i = torch.arange(N, device=DEV)
    live = i < new[:, None]
    row = torch.where(live, start[:, None] + i, 0)
    pos = (length - new)[:, None] + i  # [B][N]
    q = _rotate(s["q"], s["position"], torch.float32)[row].view(B, N, Hkv, G, d)
    q = q.permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * N, d)
    score = torch.matmul(q, k.transpose(2, 3)) * (1.0 / math.sqrt(d))
    seen = torch.arange(W * bl, device=DEV) <= pos[..., None]  # [B][N][keys]
    score = score.view(B, Hkv, G, N, W * bl).masked_fill(~seen[:, None, None], -math.inf)
    p = torch.exp(score - score.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, Hkv, G * N, W * bl), v).view(B, Hkv, G, N, d)
    o = o.permute(0, 3, 1, 2, 4).reshape(B * N, Hq, d).to(torch.bfloat16)
    s["out"][row.view(-1)[live.view(-1)]] = o[live.view(-1)]
    return s["out"]


def run(s):
    op = s["case"]["op"]
    if own:
        from attention_cached_kv_gb300 import binding
        if op == "plan":
            p = binding.gist_paged_plan(s["cached_len"], s["new_len"], s["block_table"], s["free_blocks"], s["free_range"],
                                        s["plan"], dims=s["dims"])
            return {"block_table": s["block_table"], "q_start": p.q_start, "kv_len": p.kv_len, "slot": p.slot,
                    "position": p.position, "free_range": p.free_range}
        if op == "append":
            binding.gist_kv_append_fp8(s["k"], s["v"], s["pool"], s["scale"], s["slot"], s["position"], dims=s["dims"])
            return {"pool": s["pool"], "scale": s["scale"]}
        return binding.gist_attn_paged_fp8kv(s["q"], s["pool"], s["scale"], s["block_table"], s["q_start"], s["kv_len"],
                                             s["out"], s["workspace"], dims=s["dims"])
    return {"plan": _plain_plan, "append": _plain_append, "attn": _plain_attn}[op](s)


def work(case):
    cached, new = _lengths(case)
    B, T, bl = case["batch"], sum(new), case["block_len"]
    taken = sum(-(-(c + n) // bl) - -(-c // bl) for c, n in zip(cached, new))
    if case["op"] == "plan":
        # lengths in; starts, lengths, slots and positions out; the taken blocks' ids read and written
        return {"bytes": 4 * (2 * B + (B + 1) + B + 2 * T + 2 * taken + 4), "flops": 0}
    d, Hkv = case["dim"], case["kv_heads"]
    if case["op"] == "append":
        blocks = sum(-(-(c + n) // bl) - c // bl for c, n in zip(cached, new))
        # bf16 keys and values in, E4M3 out; slot and position; the touched blocks' scales read and written
        return {"bytes": T * 2 * Hkv * d * 3 + 8 * T + blocks * 2 * Hkv * 8, "flops": 6 * T * Hkv * d}
    Hq = case["q_heads"]
    keys = sum(c + n for c, n in zip(cached, new))
    blocks = sum(-(-(c + n) // bl) for c, n in zip(cached, new))
    pairs = sum(n * c + n * (n + 1) // 2 for c, n in zip(cached, new))
    return {"bytes": keys * 2 * Hkv * d + blocks * (8 * Hkv + 4) + 2 * T * Hq * d * 2, "flops": 4 * pairs * Hq * d}


# ------------------------------------------- the definitions, in 64 bits


def _exact_plan(s):
    bl = s["bl"]
    cached, new = s["cached_len"].tolist(), s["new_len"].tolist()
    free, (begin, end) = s["free_blocks"].tolist(), s["free_range"].tolist()
    table = s["block_table"].tolist()
    q_start, kv_len, slot, position, asked, taken = [0], [], [], [], 0, 0
    for r, (c, n) in enumerate(zip(cached, new)):
        have, want = -(-c // bl), -(-(c + n) // bl)
        asked += want - have
        ok = want == have or asked <= end - begin
        if ok:
            for b in range(have, want):
                table[r][b] = free[begin + taken]
                taken += 1
        for pos in range(c, c + n):
            slot.append(table[r][pos // bl] * bl + pos % bl if ok else -1)
            position.append(pos if ok else -1)
        q_start.append(q_start[-1] + n)
        kv_len.append(c + n if ok else 0)
    named = dict(block_table=table, q_start=q_start, kv_len=kv_len, slot=slot, position=position, free_range=[begin + taken, end])
    return {k: torch.tensor(v, dtype=torch.int32) for k, v in named.items()}


def _spin(x, position):
    """x (64 bits, [n][heads][d]) turned by e^(i position theta_j), the pairs as complex numbers."""
    half = x.shape[-1] // 2
    j = torch.arange(half, device=x.device, dtype=torch.float64)
    turn = torch.polar(torch.ones((), device=x.device, dtype=torch.float64), position.double()[:, None] * torch.exp(-math.log(THETA) * j / half))
    z = torch.complex(x[..., :half].contiguous(), x[..., half:].contiguous()) * turn[:, None]
    return torch.cat([z.real, z.imag], -1)


def _exact_append(s):
    bl = s["bl"]
    pool, scale = s["pool"].double()[:, LAYER], s["scale"].double()[:, LAYER]
    slot, starts = s["slot"].tolist(), s["q_start"].tolist()
    planes = [(_spin(s["k"].double(), s["position"]), 316.0, s["k"]), (s["v"].double(), 448.0, s["v"])]
    for r in range(s["B"]):
        a = starts[r]
        while a < starts[r + 1]:
            blk, off = divmod(slot[a], bl)
            b = min(starts[r + 1], a + bl - off)
            for kv, (x, most, given) in enumerate(planes):
                top = given[a:b].double().abs().amax((0, 2))  # [Hkv]
                s_new = torch.exp2(torch.ceil(torch.log2((top / most).clamp(min=2.0 ** -100))))
                if off:
                    s_new = torch.maximum(s_new, scale[blk, kv])
                    old = pool[blk, kv, :, :off] * (scale[blk, kv] / s_new)[:, None, None]
                    pool[blk, kv, :, :off] = old.float().to(torch.float8_e4m3fn).double()
                scale[blk, kv] = s_new
                codes = (x[a:b] / s_new[None, :, None]).float().to(torch.float8_e4m3fn).double()
                pool[blk, kv, :, off:off + b - a] = codes.transpose(0, 1)
            a = b
    whole, scales = s["pool"].double(), s["scale"].double()
    whole[:, LAYER], scales[:, LAYER] = pool, scale
    return {"pool": whole, "scale": scales}


def _exact_attn(s):
    case, bl = s["case"], s["bl"]
    G, d = case["q_heads"] // case["kv_heads"], case["dim"]
    q = _spin(s["q"].double(), s["position"])
    out = torch.empty_like(q)
    starts, lengths = s["q_start"].tolist(), s["kv_len"].tolist()
    for r, C in enumerate(lengths):
        a, b = starts[r], starts[r + 1]
        ids = s["block_table"][r, :-(-C // bl)].long()
        rows = s["pool"][ids, LAYER].double() * s["scale"][ids, LAYER].double()[..., None, None]  # [nb][2][Hkv][bl][d]
        for g in range(case["kv_heads"]):
            k, v = rows[:, 0, g].reshape(-1, d)[:C], rows[:, 1, g].reshape(-1, d)[:C]
            x = q[a:b, g * G:(g + 1) * G].transpose(0, 1)  # [G][n][d]
            w = x @ k.T / math.sqrt(d)
            seen = torch.ones((b - a, C), dtype=torch.bool, device=w.device).tril(C - (b - a))
            w = torch.softmax(w.masked_fill(~seen, -math.inf), -1)
            out[a:b, g * G:(g + 1) * G] = (w @ v).transpose(0, 1)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"plan": _exact_plan, "append": _exact_append, "attn": _exact_attn}[case["op"]](s)
