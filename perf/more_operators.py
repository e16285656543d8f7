"""Cases of the single-token serving step over a bf16 paged cache, and of the cache's pages.

  attn     attention of one new token a request over a bf16 paged cache, each request
           with a length of its own
  fork     requests that go on from others (beams, samples of one prompt): full blocks
           shared, the last one copied as far as it is filled
  compact  the blocks in use brought to the front of the pool, tables renamed
  free     reference counts and the free list, from the tables of the requests alive
  copy     whole blocks copied within the pool
  qkv, out the projections before and after the attention of a few tokens, with 4-bit
           weights and a scale per group of inputs

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


def _attn(name, batch, keys, heads, dim, block_len):
    return {"name": name, "op": "attn", "batch": batch, "lo": keys[0], "hi": keys[1], "q_heads": heads[0],
            "kv_heads": heads[1], "dim": dim, "block_len": block_len}


def _pages(name, op, batch, keys, heads, dim, block_len, layers, fp8, **more):
    return {"name": name, "op": op, "batch": batch, "lo": keys[0], "hi": keys[1], "kv_heads": heads, "dim": dim,
            "block_len": block_len, "layers": layers, "fp8": fp8, **more}


def _proj(name, op, tokens, heads, dim, d_model, group):
    return {"name": name, "op": op, "tokens": tokens, "q_heads": heads[0], "kv_heads": heads[1], "dim": dim,
            "d_model": d_model, "group": group}


def listed():
    return [
        # a handful of short conversations on the small model: latency
        _attn("attn short 6", 6, (9, 300), (14, 2), 64, 16),
        # a full decoding batch with grouped heads, from fresh requests to long ones
        _attn("attn gqa 48", 48, (200, 9000), (32, 8), 128, 64),
        # a KV head for every query head
        _attn("attn mha 12", 12, (1000, 8000), (32, 32), 128, 256),
        # one long document: few rows, a long axis
        _attn("attn one long", 1, (180001, 180001), (14, 2), 64, 64),
        # three more samples of each of 16 prompts
        _pages("fork samples", "fork", 16, (30, 4000), 8, 128, 256, 4, False, children=3),
        # a fragmented E4M3 pool before it is saved or shrunk
        _pages("compact e4m3", "compact", 32, (500, 4000), 8, 128, 64, 4, True, slack=2.0),
        # the free list of a large server, a third of whose requests have ended
        _pages("free 2048", "free", 2048, (0, 2000), 2, 64, 16, 1, False, slack=1.5),
        # a few small pages: latency
        _pages("copy 3", "copy", 3, (16, 16), 2, 64, 16, 24, False),
        # the next token of one conversation, wide model
        _proj("qkv one token", "qkv", 1, (32, 8), 128, 4096, 128),
        # five conversations on the small model: latency
        _proj("qkv small 5", "qkv", 5, (14, 2), 64, 896, 32),
        # a decoding batch's output projection
        _proj("out 32", "out", 32, (32, 8), 128, 4096, 64),
        # a wide layer, as many tokens as the path is meant for
        _proj("out large 64", "out", 64, (64, 8), 128, 8192, 128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "fork", "compact", "free", "copy", "qkv", "qkv", "out", "out"])
    block_len = rng.choice([16, 32, 64, 128, 256])
    if op == "attn":
        q_heads, kv_heads, dim = rng.choice([(14, 2, 64), (32, 8, 128), (32, 32, 128), (16, 4, 64), (16, 1, 128), (12, 4, 128)])
        batch = _log(rng, 1, 96)
        hi = _log(rng, 16, min(250_000, 700_000_000 // (batch * kv_heads * dim * 4)))
        c = _attn("", batch, (max(1, int(hi * rng.uniform(0.02, 1))), hi), (q_heads, kv_heads), dim, block_len)
    elif op in ("qkv", "out"):
        q_heads, kv_heads, dim = rng.choice([(14, 2, 64), (32, 8, 128), (32, 32, 128), (16, 4, 64), (64, 8, 128)])
        group = rng.choice([32, 64, 128])
        c = _proj("", op, _log(rng, 1, 64), (q_heads, kv_heads), dim, 128 * _log(rng, 4, 64), group)
    elif op == "free":
        c = _pages("", "free", _log(rng, 1, 4000), (0, _log(rng, 20, 3000)), 2, 64, block_len, 1, False,
                   slack=rng.uniform(1.1, 3.0))
    else:
        kv_heads, dim = rng.choice([(2, 64), (8, 128), (4, 64)])
        layers, fp8 = rng.randint(1, 6), rng.random() < 0.5
        page = 2 * kv_heads * dim * block_len * layers * (1 if fp8 else 2)
        if op == "copy":
            c = _pages("", "copy", _log(rng, 1, max(1, min(500, 250_000_000 // page))), (block_len, block_len), kv_heads, dim,
                       block_len, layers, fp8)
        else:
            batch = _log(rng, 1, 32)
            most = max(2 * block_len, min(6000, 300_000_000 // page * block_len // batch))
            hi = _log(rng, block_len, most)
            more = {"children": rng.randint(1, 4)} if op == "fork" else {"slack": rng.uniform(1.2, 2.5)}
            c = _pages("", op, batch, (max(1, hi // 8), hi), kv_heads, dim, block_len, layers, fp8, **more)
    del c["name"]
    return c


def _lengths(case):
    """Cached tokens of each request: the same for every seed, so that the work is."""
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    out = [rng.randint(case["lo"], case["hi"]) for _ in range(case["batch"])]
    if case["op"] == "free":
        out = [0 if rng.random() < 0.33 else n for n in out]
    return out


def _shape(case):
    """Of a page case: blocks of each request, how many of them it shares with the one before,
    blocks in use, blocks in all, and blocks in use past the first so many."""
    bl, n = case["block_len"], [-(-t // case["block_len"]) for t in _lengths(case)]
    if case["op"] == "copy":
        return n, [0] * len(n), len(n), 2 * len(n) + 3, 0
    shared = [min(n[r - 1], n[r]) // 2 if r % 2 and case["op"] != "fork" else 0 for r in range(len(n))]
    live = sum(n) - sum(shared)
    if case["op"] == "fork":
        return n, shared, live, live + len(n) * case["children"] + 5, 0
    total = max(int(live * case["slack"]), live + 1, 2)
    return n, shared, live, total, min(live, total - live) // 2


def _copies(case):
    """Rows that a fork copies for each child, in the children's order (parents in turn)."""
    return [t % case["block_len"] for t in _lengths(case) * case["children"] if t % case["block_len"]]


def _generator(seed, stream, device=DEV):
    return torch.Generator(device=device).manual_seed(16 * int(seed) + stream)


def _normal(shape, seed, stream, dtype, spread=1.0):
    """Normal deviates, in pieces."""
    out = torch.empty(shape, dtype=dtype, device=DEV)
    flat, g, step = out.view(-1), _generator(seed, stream), 1 << 28
    for a in range(0, flat.numel(), step):
        n = min(step, flat.numel() - a)
        x = torch.randn(n, generator=g, device=DEV) * spread
        flat[a:a + n] = (x.clamp_(-448, 448) if dtype == torch.float8_e4m3fn else x).to(dtype)
    return out


def _dims(case, requests, tokens, width, num_blocks, layers, layer):
    return dict(num_requests=requests, num_tokens=tokens, max_new=1, num_q_heads=case.get("q_heads", case["kv_heads"]),
                num_kv_heads=case["kv_heads"], head_dim=case["dim"], block_len=case.get("block_len", 16), max_blocks=width,
                num_blocks=num_blocks, num_layers=layers, layer=layer, rope_theta=THETA, softmax_scale=0.0)


def prepare(case, seed):
    case = dict(case)
    return {"attn": _prepare_attn, "qkv": _prepare_proj, "out": _prepare_proj}.get(case["op"], _prepare_pages)(case, seed)


def _prepare_attn(case, seed):
    lens, bl, B = _lengths(case), case["block_len"], case["batch"]
    n = torch.tensor([-(-t // bl) for t in lens])
    width, num_blocks, layers = int(n.max()) + 1, int(n.sum()) + 7, 2
    perm = torch.randperm(num_blocks, generator=_generator(seed, 0, "cpu"))
    col = torch.arange(width)
    ahead = torch.cumsum(n, 0) - n
    table = torch.where(col < n[:, None], perm[(ahead[:, None] + col).clamp(max=num_blocks - 1)], -1)
    i32 = dict(dtype=torch.int32, device=DEV)
    s = {"case": case, "table": table.to(torch.int32).to(DEV), "kv_len": torch.tensor(lens, **i32),
         "dims": _dims(case, B, B, width, num_blocks, layers, 1)}
    s["pool"] = _normal((num_blocks, layers, 2, case["kv_heads"], bl, case["dim"]), seed, 1, torch.bfloat16)
    s["q"] = _normal((B, case["q_heads"], case["dim"]), seed, 2, torch.bfloat16)
    s["out"] = torch.empty_like(s["q"])
    s["workspace"] = torch.empty(64 << 20, dtype=torch.uint8, device=DEV)
    return s


def _prepare_pages(case, seed):
    op, bl, lens = case["op"], case["block_len"], _lengths(case)
    n, shared, live, num_blocks, above = _shape(case)
    g = _generator(seed, 0, "cpu")
    # the ids in use: all but `above` of them among the first `live`
    low, high = torch.randperm(live, generator=g), live + torch.randperm(num_blocks - live, generator=g)
    used = torch.cat([low[:live - above], high[:above]])
    used = used[torch.randperm(live, generator=g)]
    unused = torch.cat([low[live - above:], high[above:]])
    unused = unused[torch.randperm(num_blocks - live, generator=g)]
    n_t, shared_t = torch.tensor(n), torch.tensor(shared)
    first = torch.cumsum(n_t - shared_t, 0) - (n_t - shared_t)
    width = max(1, max(n)) + 1
    col = torch.arange(width)
    at = torch.where(col < shared_t[:, None], first.roll(1)[:, None] + col, (first - shared_t)[:, None] + col)
    table = torch.where(col < n_t[:, None], used[at.clamp(0, max(live - 1, 0))] if live else torch.zeros_like(at), -1)
    i32 = dict(dtype=torch.int32, device=DEV)
    s = {"case": case, "n_blocks": num_blocks}
    if op == "fork":
        kids = case["children"]
        B = len(n) * (1 + kids)
        table = torch.cat([table, torch.full((len(n) * kids, width), -1)])
        s["parent"] = torch.tensor([-1] * len(n) + list(range(len(n))) * kids, **i32)
        s["cached_len"] = torch.tensor(lens + [0] * (len(n) * kids), **i32)
        s["free_blocks"] = unused.to(torch.int32).to(DEV)
        s["free_range"] = torch.tensor([0, len(unused)], **i32)
        s["out"] = [torch.empty(k, **i32) for k in (B, B, B, B, 1, 2)]
        s["count"] = len(_copies(case))
    else:
        B = len(n)
        s["cached_len"] = torch.tensor(lens, **i32)
        if op == "compact":
            s["out"] = [torch.empty((B, width), **i32)] + [torch.empty(k, **i32) for k in
                                                           (num_blocks, num_blocks // 2, num_blocks // 2, 1, num_blocks, 2)]
            s["count"] = above
        elif op == "free":
            s["out"] = [torch.empty(k, **i32) for k in (num_blocks, num_blocks, 2)]
        else:
            s["src"], s["dst"], s["count"] = used.to(torch.int32).to(DEV), unused[:live].to(torch.int32).to(DEV), live
    s["table"] = table.to(torch.int32).contiguous().to(DEV)
    s["dims"] = _dims(case, B, B, width, num_blocks, case["layers"], 0)
    if op != "free":
        shape = (num_blocks, case["layers"], 2, case["kv_heads"], bl, case["dim"])
        s["pool"] = _normal(shape, seed, 1, torch.float8_e4m3fn if case["fp8"] else torch.bfloat16, 100.0 if case["fp8"] else 1.0)
        s["scale"] = torch.exp2(torch.randint(-8, -5, shape[:4], generator=_generator(seed, 2), device=DEV).float()) if case["fp8"] else None
    return s


def _sizes(case):
    """Outputs and inputs of a projection."""
    if case["op"] == "qkv":
        return (case["q_heads"] + 2 * case["kv_heads"]) * case["dim"], case["d_model"]
    return case["d_model"], case["q_heads"] * case["dim"]


def _prepare_proj(case, seed):
    T, (N, K) = case["tokens"], _sizes(case)
    s = {"case": case, "dims": _dims(case, T, T, 1, 1, 1, 0)}
    s["x"] = _normal((T, K), seed, 1, torch.bfloat16)
    # codes of a bell-shaped weight, two to a byte, and scales that make outputs of about one
    code = (torch.randn((N, K), generator=_generator(seed, 2), device=DEV) * 3 + 8).round_().clamp_(0, 15).to(torch.uint8)
    s["w"] = code[:, 0::2] | (code[:, 1::2] << 4)
    spread = torch.rand((N, K // case["group"]), generator=_generator(seed, 3), device=DEV) + 0.5
    s["w_scale"] = (spread / (3 * math.sqrt(K))).to(torch.bfloat16)
    s["position"] = torch.randint(0, 8192, (T,), generator=_generator(seed, 4), device=DEV).to(torch.int32)
    d, bf = case["dim"], dict(dtype=torch.bfloat16, device=DEV)
    if case["op"] == "qkv":
        s["out"] = [torch.empty((T, h, d), **bf) for h in (case["q_heads"], case["kv_heads"], case["kv_heads"])]
    else:
        s["x"] = s["x"].view(T, case["q_heads"], d)
        s["out"] = torch.empty((T, N), **bf)
    return s


# ------------------------------------------------------------- the plain forms


def _rotate(x, position):
    """Rotate-half pairs (j, j + d/2) at theta^(-2j/d), the angles in 64 bits."""
    half = x.shape[-1] // 2
    freq = THETA ** (-torch.arange(half, device=x.device, dtype=torch.float64) / half)
    angle = position.double()[:, None] * freq
    cos, sin = torch.cos(angle)[:, None].float(), torch.sin(angle)[:, None].float()
    a, b = x[..., :half], x[..., half:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _plain_attn(s):
    case, d = s["case"], s["dims"]
    B, W, bl, Hkv, dim = case["batch"], d["max_blocks"], case["block_len"], case["kv_heads"], case["dim"]
    G = case["q_heads"] // Hkv
    table, length = s["table"].clamp(min=0).long(), s["kv_len"].long()
    kv = s["pool"][:, d["layer"]][table].float()  # [B][W][2][Hkv][bl][d]
    k, v = kv.permute(2, 0, 3, 1, 4, 5).reshape(2, B, Hkv, W * bl, dim)
    q = _rotate(s["q"].float(), length - 1).view(B, Hkv, G, dim)
    score = torch.matmul(q, k.transpose(2, 3)) * (1.0 / math.sqrt(dim))
    seen = torch.arange(W * bl, device=DEV) < length[:, None]
    score = score.masked_fill(~seen[:, None, None], -math.inf)
    p = torch.exp(score - score.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    s["out"].copy_(torch.matmul(p, v).reshape(B, Hkv * G, dim))
    return s["out"]


def _plain_copy(s, src, dst, rows=None):
    src, dst = src.long(), dst.long()
    pool = s["pool"].view(torch.uint8) if s["case"]["fp8"] else s["pool"]
    blocks = pool[src]
    if rows is not None:
        keep = torch.arange(s["case"]["block_len"], device=DEV) < rows[:, None]
        blocks = torch.where(keep[:, None, None, None, :, None], blocks, pool[dst])
    pool[dst] = blocks
    if s["scale"] is not None:
        s["scale"][dst] = s["scale"][src]
    return {"pool": s["pool"]} | ({} if s["scale"] is None else {"scale": s["scale"]})


def _dense(keep, values, size):
    """The values where `keep`, in order, then -1: [size]."""
    at = torch.where(keep, torch.cumsum(keep, 0) - 1, size)
    return torch.full((size + 1,), -1, dtype=torch.int32, device=DEV).scatter_(0, at, values.int())[:size]


def _plain_fork(s):
    bl, table, parent = s["case"]["block_len"], s["table"], s["parent"].long()
    B, W = table.shape
    forked = parent >= 0
    p = parent.clamp(min=0)
    c = s["cached_len"].long()[p]
    part = forked & (c % bl != 0)
    before = torch.cumsum(part, 0) - part.long()
    begin, end = s["free_range"].long()
    served = ~part | (before < end - begin)
    taken = s["free_blocks"].long()[(begin + before).clamp(0, s["free_blocks"].numel() - 1)]
    col = torch.arange(W, device=DEV)
    rows = torch.where((part & served)[:, None] & (col == (c // bl)[:, None]), taken[:, None], table.long()[p])
    mine = (forked & served)[:, None] & (col < ((c + bl - 1) // bl)[:, None])
    moved = part & served
    last = table.long()[p, (c // bl).clamp(max=W - 1)]
    src, dst, n = _dense(moved, last, B), _dense(moved, taken, B), _dense(moved, c % bl, B)
    table.copy_(torch.where(mine, rows, table.long()))
    out = _plain_copy(s, src[:s["count"]], dst[:s["count"]], n[:s["count"]])
    length = torch.where(forked, torch.where(served, c, 0), s["cached_len"].long())
    return out | {"block_table": table, "cached_len": length.int(), "src": src, "dst": dst, "rows": n,
                  "count": moved.sum().int().view(1), "free_range": torch.stack([begin + moved.sum(), end]).int()}


def _references(s):
    bl, table = s["case"]["block_len"], s["table"].long()
    n = (s["cached_len"].long() + bl - 1) // bl
    live = torch.arange(table.shape[1], device=DEV) < n[:, None]
    ref = torch.zeros(s["n_blocks"] + 1, dtype=torch.int32, device=DEV)
    ref.index_add_(0, torch.where(live, table, s["n_blocks"]).view(-1), torch.ones(table.numel(), dtype=torch.int32, device=DEV))
    return ref[:-1], live


def _plain_free(s):
    ref, _ = _references(s)
    ids = torch.arange(s["n_blocks"], device=DEV)
    count = (ref == 0).sum()
    return {"ref": ref, "free": _dense(ref == 0, ids, s["n_blocks"]), "range": torch.stack([torch.zeros_like(count), count]).int()}


def _plain_compact(s):
    nb = s["n_blocks"]
    ref, live = _references(s)
    used = ref > 0
    n = used.sum()
    ids = torch.arange(nb, device=DEV)
    src, dst = _dense(used & (ids >= n), ids, nb // 2), _dense(~used & (ids < n), ids, nb // 2)
    new = torch.where(used & (ids < n), ids, -1)
    a, b = src[:s["count"]].long(), dst[:s["count"]].long()
    new[a] = b
    table = torch.where(live, new[s["table"].clamp(min=0).long()], s["table"].long()).int()
    rest = torch.where(ids < nb - n, n + ids, -1).int()
    return _plain_copy(s, a, b) | {"block_table": table, "new_id": new.int(), "src": src, "dst": dst,
                                   "count": torch.full((1,), s["count"], dtype=torch.int32, device=DEV), "free": rest,
                                   "range": torch.stack([n * 0, nb - n]).int()}


def _plain_proj(s):
    case, x = s["case"], s["x"]
    T, (N, K) = case["tokens"], _sizes(case)
    code = torch.stack([s["w"] & 15, s["w"] >> 4], -1).view(N, K).float() - 8
    w = code.view(N, -1, case["group"]) * s["w_scale"].float()[..., None]
    y = torch.matmul(x.reshape(T, K).float(), w.view(N, K).t())
    if case["op"] == "out":
        s["out"].copy_(y)
        return s["out"]
    q, k, v = y.view(T, -1, case["dim"]).split([case["q_heads"], case["kv_heads"], case["kv_heads"]], 1)
    s["out"][0].copy_(_rotate(q, s["position"]))
    s["out"][1].copy_(_rotate(k, s["position"]))
    s["out"][2].copy_(v)
    return {"q": s["out"][0], "k": s["out"][1], "v": s["out"][2]}


def run(s):
    op = s["case"]["op"]
    if own:
        return _own(s, op)
    if op == "copy":
        return _plain_copy(s, s["src"], s["dst"])
    return {"attn": _plain_attn, "fork": _plain_fork, "compact": _plain_compact, "free": _plain_free}.get(op, _plain_proj)(s)


def _own(s, op):
    from attention_cached_kv_gb300 import binding
    case, dims = s["case"], s["dims"]
    if op == "attn":
        return binding.gist_attn_paged_decode(s["q"], s["pool"], s["table"], s["kv_len"], None, s["out"], s["workspace"], dims=dims)
    if op == "qkv":
        q, k, v = binding.gist_qkv_rope_w4(s["x"], s["w"], s["w_scale"], s["position"], *s["out"], group=case["group"], dims=dims)
        return {"q": q, "k": k, "v": v}
    if op == "out":
        return binding.gist_out_proj_w4(s["x"], s["w"], s["w_scale"], s["out"], group=case["group"], dims=dims)
    if op == "free":
        f = binding.gist_pages_free(s["cached_len"], s["table"], s["out"], dims=dims)
        return {"ref": f.ref_count, "free": f.free_blocks, "range": f.free_range}
    if op == "copy":
        binding.gist_pages_copy(s["pool"], s["scale"], s["src"], s["dst"], dims=dims)
        return {"pool": s["pool"]} | ({} if s["scale"] is None else {"scale": s["scale"]})
    if op == "fork":
        f = binding.gist_pages_fork(s["cached_len"], s["parent"], s["table"], s["free_blocks"], s["free_range"], s["out"], dims=dims)
        binding.gist_pages_copy(s["pool"], s["scale"], f.copy_src, f.copy_dst, f.copy_rows, f.num_copies, dims=dims)
        more = {"block_table": s["table"], "cached_len": f.cached_len, "src": f.copy_src, "dst": f.copy_dst, "rows": f.copy_rows,
                "count": f.num_copies, "free_range": f.free_range}
    else:
        f = binding.gist_pages_compact(s["cached_len"], s["table"], s["out"], dims=dims)
        binding.gist_pages_copy(s["pool"], s["scale"], f.copy_src, f.copy_dst, None, f.num_copies, dims=dims)
        more = {"block_table": f.block_table, "new_id": f.new_id, "src": f.copy_src, "dst": f.copy_dst, "count": f.num_copies,
                "free": f.free_blocks, "range": f.free_range}
    return {"pool": s["pool"]} | ({} if s["scale"] is None else {"scale": s["scale"]}) | more


def work(case):
    op = case["op"]
    if op == "attn":
        lens, Hkv, d = _lengths(case), case["kv_heads"], case["dim"]
        blocks = sum(-(-t // case["block_len"]) for t in lens)
        return {"bytes": sum(lens) * 4 * Hkv * d + 4 * blocks + len(lens) * (4 + 4 * case["q_heads"] * d),
                "flops": 4 * sum(lens) * case["q_heads"] * d}
    if op in ("qkv", "out"):
        T, (N, K) = case["tokens"], _sizes(case)
        return {"bytes": N * K // 2 + 2 * N * (K // case["group"]) + 2 * T * (N + K) + (4 * T if op == "qkv" else 0),
                "flops": 2 * T * N * K}
    n, shared, live, nb, above = _shape(case)
    row = 2 * case["kv_heads"] * case["dim"] * case["layers"] * (1 if case["fp8"] else 2)
    scales = 8 * case["kv_heads"] * case["layers"] if case["fp8"] else 0
    if op == "copy":
        return {"bytes": live * (2 * (row * case["block_len"] + scales) + 8), "flops": 0}
    if op == "fork":
        rows, B = _copies(case), len(n) * (1 + case["children"])
        entries = sum(n) * (1 + case["children"])  # the parents' read, the children's written
        return {"bytes": 2 * (row * sum(rows) + scales * len(rows)) + 4 * (entries + len(rows) + 6 * B + 5), "flops": 0}
    if op == "free":
        return {"bytes": 4 * (len(n) + sum(n) + 2 * nb + 2), "flops": 0}
    width = max(1, max(n)) + 1
    return {"bytes": above * 2 * (row * case["block_len"] + scales) + 4 * (len(n) + 2 * len(n) * width + 2 * nb + 2 * (nb // 2) + 3),
            "flops": 0}


# ------------------------------------------- the definitions, in 64 bits


def _spin(x, position):
    """x (64 bits, [n][heads][d]) turned by e^(i position theta_j), the pairs as complex numbers."""
    half = x.shape[-1] // 2
    j = torch.arange(half, device=x.device, dtype=torch.float64)
    one = torch.ones((), device=x.device, dtype=torch.float64)
    turn = torch.polar(one, position.double()[:, None] * torch.exp(-math.log(THETA) * j / half))
    z = torch.complex(x[..., :half].contiguous(), x[..., half:].contiguous()) * turn[:, None]
    return torch.cat([z.real, z.imag], -1)


def _exact_attn(s):
    case, bl, layer = s["case"], s["case"]["block_len"], s["dims"]["layer"]
    G, d = case["q_heads"] // case["kv_heads"], case["dim"]
    q = _spin(s["q"].double(), s["kv_len"] - 1)
    out = torch.empty_like(q)
    for r, C in enumerate(s["kv_len"].tolist()):
        ids = s["table"][r, :-(-C // bl)].long()
        rows = s["pool"][ids, layer].double()  # [nb][2][Hkv][bl][d]
        for g in range(case["kv_heads"]):
            k, v = rows[:, 0, g].reshape(-1, d)[:C], rows[:, 1, g].reshape(-1, d)[:C]
            w = torch.softmax(q[r, g * G:(g + 1) * G] @ k.T / math.sqrt(d), -1)
            out[r, g * G:(g + 1) * G] = w @ v
    return out


def _exact_moved(s, moves):
    """The pool's values and scales after block `a` went to `b` as far as `rows`, for each of the moves."""
    pool = s["pool"].double()
    scale = None if s["scale"] is None else s["scale"].double()
    for a, b, rows in moves:
        pool[b, :, :, :, :rows] = pool[a, :, :, :, :rows].clone()
        if scale is not None:
            scale[b] = scale[a]
    return {"pool": pool} | ({} if scale is None else {"scale": scale})


def _padded(values, size):
    return torch.tensor(values + [-1] * (size - len(values)), dtype=torch.int32)


def _exact_fork(s):
    bl = s["case"]["block_len"]
    cached, table, free = s["cached_len"].tolist(), s["table"].tolist(), s["free_blocks"].tolist()
    begin, end = s["free_range"].tolist()
    moves, length = [], list(cached)
    for r, p in enumerate(s["parent"].tolist()):
        if p < 0:
            continue
        c = cached[p]
        full, rows = divmod(c, bl)
        if rows and len(moves) == end - begin:
            length[r] = 0
            continue
        length[r] = c
        table[r][:full] = table[p][:full]
        if rows:
            table[r][full] = free[begin + len(moves)]
            moves.append((table[p][full], table[r][full], rows))
    B = len(cached)
    named = {"src": 0, "dst": 1, "rows": 2}
    return _exact_moved(s, moves) | {k: _padded([m[i] for m in moves], B) for k, i in named.items()} | {
        "block_table": torch.tensor(table, dtype=torch.int32), "cached_len": torch.tensor(length, dtype=torch.int32),
        "count": torch.tensor([len(moves)], dtype=torch.int32), "free_range": torch.tensor([begin + len(moves), end], dtype=torch.int32)}


def _counts(s):
    bl, ref = s["case"]["block_len"], [0] * s["n_blocks"]
    for length, row in zip(s["cached_len"].tolist(), s["table"].tolist()):
        for b in row[:-(-length // bl)]:
            ref[b] += 1
    return ref


def _exact_free(s):
    ref = _counts(s)
    free = [b for b, n in enumerate(ref) if n == 0]
    return {"ref": torch.tensor(ref, dtype=torch.int32), "free": _padded(free, len(ref)),
            "range": torch.tensor([0, len(free)], dtype=torch.int32)}


def _exact_compact(s):
    bl, ref = s["case"]["block_len"], _counts(s)
    used = [b for b, n in enumerate(ref) if n]
    n = len(used)
    src, dst = [b for b in used if b >= n], sorted(set(range(n)) - set(used))
    name = {b: b for b in used} | dict(zip(src, dst))
    table = [[name[b] if j < -(-length // bl) else b for j, b in enumerate(row)]
             for length, row in zip(s["cached_len"].tolist(), s["table"].tolist())]
    nb = s["n_blocks"]
    return _exact_moved(s, [(a, b, bl) for a, b in zip(src, dst)]) | {
        "block_table": torch.tensor(table, dtype=torch.int32), "new_id": torch.tensor([name.get(b, -1) for b in range(nb)], dtype=torch.int32),
        "src": _padded(src, nb // 2), "dst": _padded(dst, nb // 2), "count": torch.tensor([len(src)], dtype=torch.int32),
        "free": _padded(list(range(n, nb)), nb), "range": torch.tensor([0, nb - n], dtype=torch.int32)}


def _exact_proj(s):
    case, T = s["case"], s["case"]["tokens"]
    N, K = _sizes(case)
    value = torch.arange(-8, 8, device=DEV, dtype=torch.float64)
    raw = s["w"].long()
    w = torch.empty((N, K), dtype=torch.float64, device=DEV)
    w[:, 0::2], w[:, 1::2] = value[raw % 16], value[raw // 16]
    x = s["x"].reshape(T, K).double()
    y = torch.zeros((T, N), dtype=torch.float64, device=DEV)
    for i in range(K // case["group"]):
        at = slice(i * case["group"], (i + 1) * case["group"])
        y += (x[:, at] @ w[:, at].T) * s["w_scale"][:, i].double()
    if case["op"] == "out":
        return y
    y, Hq, Hkv = y.view(T, -1, case["dim"]), case["q_heads"], case["kv_heads"]
    return {"q": _spin(y[:, :Hq], s["position"]), "k": _spin(y[:, Hq:Hq + Hkv], s["position"]), "v": y[:, Hq + Hkv:]}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "copy":
        return _exact_moved(s, [(a, b, case["block_len"]) for a, b in zip(s["src"].tolist(), s["dst"].tolist())])
    return {"attn": _exact_attn, "fork": _exact_fork, "compact": _exact_compact, "free": _exact_free}.get(case["op"], _exact_proj)(s)
