"""What is measured of the serving operators around the compressed cache: rotary positions, decode
attention of a batch that shares a long prefix, decode attention that also gathers every tile's
attention mass, and the eviction of tiles by that mass.

Each case names one operator and its sizes. ``prepare`` makes the inputs from the seed, ``run`` one
pass: the plain form (elementary torch operations in 32 bits, angles in 64) or, where ``own`` is
true, the library's calls. ``exact`` computes the same outputs in 64 bits from the quantities the
pages were packed from, without unpacking a page.

The caches are K4V2 pages with fp32 scales (16-token pages of one KV head, tiles of 64 or 128
tokens), packed here in the documented format from drawn codes and scales.
"""
import math

import torch

own = False

DEV = "cuda"
DT = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
P = 16  # tokens of a page


# ------------------------------------------------------------------ the cases
def listed():
    def rope(name, seqs, tokens, q_heads, kv_heads, dim, rope_dim, dtype, interleaved=False, heads_first=False,
             inverse=False, far=131072, factor=1.0, scale=1.0):
        return dict(name=name, op="rope", seqs=seqs, tokens=tokens, q_heads=q_heads, kv_heads=kv_heads, dim=dim,
                    rope_dim=rope_dim, dtype=dtype, interleaved=interleaved, heads_first=heads_first,
                    inverse=inverse, far=far, factor=factor, scale=scale)

    def shared(name, seqs, queries, q_heads, kv_heads, dim, tile, prefix, suffix_min, suffix_max, dtype="fp16"):
        return dict(name=name, op="shared", seqs=seqs, queries=queries, q_heads=q_heads, kv_heads=kv_heads, dim=dim,
                    tile=tile, prefix=prefix, suffix_min=suffix_min, suffix_max=suffix_max, dtype=dtype)

    def mass(name, seqs, q_heads, kv_heads, dim, tile, len_min, len_max, decay, dtype="fp16"):
        return dict(name=name, op="mass", seqs=seqs, q_heads=q_heads, kv_heads=kv_heads, dim=dim, tile=tile,
                    len_min=len_min, len_max=len_max, decay=decay, dtype=dtype)

    def evict(name, seqs, tile, len_min, len_max, keep, sink, recent):
        return dict(name=name, op="evict", seqs=seqs, tile=tile, len_min=len_min, len_max=len_max, keep=keep,
                    sink=sink, recent=recent)

    return [
        # one decode step of 32 sequences: the new token's 64 query and 8 key heads, each at its own position
        rope("rope_step", 32, 1, 64, 8, 128, 128, "fp16"),
        # a prompt chunk of four sequences before it is encoded
        rope("rope_prompt", 4, 4096, 64, 8, 128, 128, "fp16", heads_first=True),
        # part of a wide head, interleaved, scaled for long contexts, an odd chunk
        rope("rope_partial", 8, 1021, 24, 4, 256, 64, "bf16", interleaved=True, far=1 << 20, factor=8.0, scale=1.2),
        # the gradient of a training step's queries and keys, kept in fp32
        rope("rope_grad", 2, 2048, 24, 4, 128, 128, "fp32", inverse=True),
        # a few requests on one system prompt, one KV head: latency
        shared("shared_small", 4, 1, 4, 1, 128, 128, 1024, 1, 200),
        # 32 requests on one long document
        shared("shared_batch", 32, 1, 64, 8, 128, 128, 16384, 1, 1024),
        # speculative verification of three tokens over a shared prefix, 64-token tiles, odd batch
        shared("shared_verify", 21, 3, 32, 8, 128, 64, 8192, 70, 515),
        # wide heads in bf16
        shared("shared_wide", 8, 1, 24, 4, 256, 128, 16384, 33, 700, "bf16"),
        # a long-context batch that watches its tiles
        mass("mass_batch", 16, 64, 8, 128, 128, 16384, 16384, 1.0),
        # ragged lengths, 64-token tiles, fading mass
        mass("mass_ragged", 7, 32, 8, 128, 64, 1, 9000, 0.95),
        # a batch cut back to half of its tiles
        evict("evict_batch", 32, 128, 12000, 16384, 64, 1, 8),
        # very long sequences of small tiles
        evict("evict_long", 8, 64, 1, 1 << 20, 4096, 2, 16),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "rope", "shared", "shared", "mass", "evict"])
    if op == "rope":
        dim = rng.choice([64, 96, 128, 256])
        heads = rng.choice([(4, 1), (16, 2), (24, 4), (64, 8), (32, 32), (7, 7)])
        dtype = rng.choice(["fp16", "bf16", "fp32"])
        per_token = (heads[0] + heads[1]) * dim * (4 if dtype == "fp32" else 2)
        seqs = _log(rng, 1, 64)
        tokens = _log(rng, 1, max(1, min(16384, 4 * 4096 * 72 * 256 // (per_token * seqs))))
        return dict(op=op, seqs=seqs, tokens=tokens, q_heads=heads[0], kv_heads=heads[1], dim=dim,
                    rope_dim=rng.choice([dim, dim, dim // 2, 32]), dtype=dtype, interleaved=rng.random() < 0.5,
                    heads_first=rng.random() < 0.5, inverse=rng.random() < 0.3, far=_log(rng, 1000, 1 << 20),
                    factor=rng.choice([1.0, 4.0, 32.0]), scale=rng.choice([1.0, 1.35]))
    if op == "shared":
        dim, tile = rng.choice([(128, 128), (128, 64), (128, 128), (256, 128)])
        heads = rng.choice([(4, 1), (8, 8), (24, 4), (32, 8), (64, 8)])
        queries = rng.choice([1, 1, 1, 2, 4])
        seqs = _log(rng, 2, 48)
        most = 32 * 64 * 16384 * 128 // (heads[0] * queries * seqs * dim)
        prefix = max(1, min(_log(rng, tile, 32768), most // 2) // tile) * tile
        top = max(queries, min(_log(rng, 8, 1200), 32 * 8 * 1024 * 128 // (seqs * heads[1] * dim)))
        return dict(op=op, seqs=seqs, queries=queries, q_heads=heads[0], kv_heads=heads[1], dim=dim, tile=tile,
                    prefix=prefix, suffix_min=rng.randint(queries, top), suffix_max=top,
                    dtype=rng.choice(["fp16", "bf16"]))
    if op == "mass":
        dim, tile = rng.choice([(128, 128), (128, 64), (256, 128)])
        heads = rng.choice([(4, 1), (8, 8), (24, 4), (32, 8), (64, 8)])
        seqs = _log(rng, 1, 32)
        top = _log(rng, 300, max(301, min(32768, 16 * 64 * 16384 * 128 // (seqs * heads[0] * dim))))
        return dict(op=op, seqs=seqs, q_heads=heads[0], kv_heads=heads[1], dim=dim, tile=tile,
                    len_min=rng.randint(1, top), len_max=top, decay=rng.choice([1.0, 0.9, 0.0]),
                    dtype=rng.choice(["fp16", "bf16"]))
    tile = rng.choice([64, 128])
    top = _log(rng, 1000, 1 << 19)
    tiles = max(4, top // tile)
    keep = _log(rng, 2, tiles)
    sink = rng.randint(0, min(4, keep - 1))
    return dict(op=op, seqs=_log(rng, 1, max(1, min(32, (8 << 20) // top))), tile=tile, len_min=rng.randint(0, top), len_max=top, keep=keep, sink=sink,
                recent=rng.randint(0, min(16, keep - sink)))


# ----------------------------------------------------------------- the inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _lengths(lo, hi, n, g):
    """n lengths over [lo, hi], the last one hi."""
    x = torch.randint(lo, hi + 1, (n,), generator=g, device=DEV)
    x[-1] = hi
    return x


def _side(bits, shape, dim, tile, g):
    """Codes, row scales and column scales of `shape` tiles as an encoder leaves them: codes gathered
    around the middle of their range, steps that differ by token, channel scales that differ by channel,
    a few channels far larger."""
    mid = (2 ** bits - 1) / 2
    codes = torch.randn((*shape, tile, dim), generator=g, device=DEV)
    codes = codes.mul_((2 ** bits - 1) / 5).add_(mid).round_().clamp_(0, 2 ** bits - 1).to(torch.uint8)
    # a unit-variance row: step about 5 / (2^bits - 1) standard deviations
    a = 5.0 / (2 ** bits - 1) * torch.exp(0.2 * torch.randn((*shape, tile), generator=g, device=DEV))
    b = -a * (mid + 0.1 * torch.randn((*shape, tile), generator=g, device=DEV))
    c = torch.exp(0.3 * torch.randn((*shape, dim), generator=g, device=DEV))
    big = torch.rand((*shape[:-1], 1, dim), generator=g, device=DEV) < 0.02
    c = torch.where(big, c * 2.0, c)
    return codes, a, b, c


def _scales_of_pages(a, b, c, dim, tile):
    """fp32 scale bytes of every page of the tiles: a[16], b[16] and the page's slice of c."""
    n = tile // P
    parts = torch.cat([a.unflatten(-1, (n, P)), b.unflatten(-1, (n, P)), c.unflatten(-1, (n, dim // n))], -1)
    return parts.contiguous().view(torch.uint8)


def _pack(k, v, dim, tile):
    """Page bytes [..., pages, bytes] of tiles given as (codes, a, b, c) of the keys and of the values."""
    n = tile // P
    x = k[0].reshape(*k[0].shape[:-2], n, 2, 8, dim // 64, 4, 2, 4, 2)  # page, token 8 hi + g, channel 64 q + 16 r + 8 h + 2 t + e
    d = x.dim() - 7
    x = x.movedim((d, d + 1, d + 2, d + 5, d + 3, d + 4, d + 6), (d, d + 2, d + 1, d + 3, d + 4, d + 5, d + 6))
    kc = (x.select(d, 0) | (x.select(d, 1) << 4)).flatten(d)
    y = v[0].reshape(*v[0].shape[:-2], n, 2, 4, 2, dim // 64, 2, 4, 8)  # page, token 8 h + 2 t + e, channel 64 q + 32 w + 8 c + g
    d = y.dim() - 7
    y = y.movedim((d, d + 2, d + 3, d + 6, d + 1, d + 4, d + 5), (d, d + 1, d + 2, d + 3, d + 4, d + 5, d + 6))
    vc = (y.select(d, 0).select(d, 0) | (y.select(d, 1).select(d, 0) << 2) | (y.select(d, 0).select(d, 1) << 4)
          | (y.select(d, 1).select(d, 1) << 6)).flatten(d)
    return torch.cat([kc, _scales_of_pages(*k[1:], dim, tile), vc, _scales_of_pages(*v[1:], dim, tile)], -1)


def _cache(case, units, seed):
    """A cache of `units` tiles per KV head under a random placement: (cache bytes, page ids [units, pages], the quantities)."""
    g = _gen(seed)
    dim, tile, heads = case["dim"], case["tile"], case["kv_heads"]
    k, v = _side(4, (units, heads), dim, tile, g), _side(2, (units, heads), dim, tile, g)
    pages = _pack(k, v, dim, tile)  # [units, heads, pages, bytes]
    ids = torch.randperm(units * (tile // P), generator=g, device=DEV)
    cache = torch.empty((ids.numel(), heads, pages.shape[-1]), dtype=torch.uint8, device=DEV)
    cache[ids] = pages.transpose(1, 2).flatten(0, 1)
    return cache, ids.to(torch.int32).view(units, tile // P), (k, v)


def _sizes(case, seed):
    """Lengths of the sequences and the tiles each has in the pages (past the prefix, where there is one)."""
    g = _gen(seed + 17)
    if case["op"] == "shared":
        lens = case["prefix"] + _lengths(case["suffix_min"], case["suffix_max"], case["seqs"], g)
        done = (lens - case["queries"] + 1) // case["tile"] - case["prefix"] // case["tile"]
    else:
        lens = _lengths(case["len_min"], case["len_max"], case["seqs"], g)
        done = lens // case["tile"]
    return lens, done.clamp(min=0)


def _attention_inputs(case, seed):
    g = _gen(seed)
    lens, done = _sizes(case, seed)
    tile, B = case["tile"], case["seqs"]
    first = case.get("prefix", 0) // tile
    per = done.tolist()
    units = first + sum(per)
    cache, ids, sides = _cache(case, max(1, units), seed + 5)
    # tile t >= first of sequence b is unit index[b, t - first]; -1 past the committed tiles
    most = max(1, max(per))
    index = torch.arange(most, device=DEV)[None, :] + (first + done.cumsum(0) - done)[:, None]
    index = torch.where(torch.arange(most, device=DEV)[None, :] < done[:, None], index, -1)
    table = torch.where(index[..., None] >= 0, ids[index.clamp(min=0)], -1).flatten(1)
    table = torch.cat([torch.full((B, first * (tile // P)), -1, dtype=torch.int32, device=DEV), table], 1)
    Q = case.get("queries", 1)
    shape = (B, Q, case["q_heads"], case["dim"])
    q = 2.0 * torch.randn(shape, generator=g, device=DEV)
    cap = tile + Q - 2 if case["op"] == "shared" else tile
    tails = torch.randn((2, B, case["kv_heads"], max(1, cap), case["dim"]), generator=g, device=DEV)
    dt = DT[case["dtype"]]
    return dict(lens=lens, done=done, index=index, sides=sides, cache=cache, table=table.to(torch.int32).contiguous(),
                prefix_table=ids[:first].flatten().contiguous(), q=q.to(dt), tail_k=tails[0].to(dt), tail_v=tails[1].to(dt))


def _mass_before(case, seed):
    g = _gen(seed + 29)
    return torch.rand((case["seqs"], max(1, case["len_max"] // case["tile"])), generator=g, device=DEV).square() * 4


def _rope_inputs(case, seed):
    g = _gen(seed)
    dt, B, S = DT[case["dtype"]], case["seqs"], case["tokens"]
    xs = []
    for h in (case["q_heads"], case["kv_heads"]):
        shape = (B, h, S, case["dim"]) if case["heads_first"] else (B, S, h, case["dim"])
        x = torch.randn(shape, generator=g, device=DEV).to(dt)
        xs.append(x.transpose(1, 2) if case["heads_first"] else x)  # [B, S, heads, dim]
    start = torch.randint(0, case["far"], (B, 1), generator=g, device=DEV)
    pos = (start + torch.arange(S, device=DEV)).to(torch.int32)
    i = torch.arange(case["rope_dim"] // 2, device=DEV, dtype=torch.float64)
    inv_freq = 10000.0 ** (-2.0 * i / case["rope_dim"]) / case["factor"]
    return xs, pos, inv_freq


def _evict_inputs(case, seed):
    g = _gen(seed)
    tile, B, n = case["tile"], case["seqs"], case["tile"] // P
    lens = _lengths(case["len_min"], case["len_max"], B, g)
    tiles = max(1, case["len_max"] // tile)
    # masses of a long-tailed kind, some of them equal (tiles never looked at)
    mass = torch.randn((B, tiles), generator=g, device=DEV).exp()
    mass = torch.where(torch.rand((B, tiles), generator=g, device=DEV) < 0.2, torch.zeros_like(mass), mass)
    table = torch.randperm(B * tiles * n, generator=g, device=DEV).to(torch.int32).view(B, tiles * n)
    done = (lens // tile)[:, None]
    mass = torch.where(torch.arange(tiles, device=DEV) < done, mass, 0.0)
    table = torch.where(torch.arange(tiles * n, device=DEV) < done * n, table, -1)
    return lens.to(torch.int32), mass, table.to(torch.int32)


def prepare(case, seed):
    op = case["op"]
    if op == "rope":
        xs, pos, inv_freq = _rope_inputs(case, seed)
        return dict(case=case, xs=xs, outs=[torch.empty_like(x) for x in xs], pos=pos, inv_freq=inv_freq)
    if op == "evict":
        lens, mass, table = _evict_inputs(case, seed)
        return dict(case=case, lens=lens, mass=mass, table=table, mass_out=torch.empty_like(mass),
                    table_out=torch.empty_like(table), lens_out=torch.empty_like(lens),
                    freed=torch.empty_like(table), freed_count=torch.empty_like(lens),
                    err=torch.zeros(1, dtype=torch.int32, device=DEV))
    s = _attention_inputs(case, seed)
    s.pop("sides")
    s.update(case=case, err=torch.zeros(1, dtype=torch.int32, device=DEV))
    s["lens32"], s["max_len"] = s["lens"].to(torch.int32), int(s["lens"].max())
    s["scale"] = 1.0 / math.sqrt(case["dim"])
    if op == "mass":
        s["q"] = s["q"][:, 0].contiguous()
        s["mass"] = _mass_before(case, seed)
        s["mass_out"] = torch.empty_like(s["mass"])
    s["out"] = torch.empty(s["q"].shape, dtype=torch.float32, device=DEV)
    s["lse"] = torch.empty(s["q"].shape[:-1], dtype=torch.float32, device=DEV)
    return s


# ------------------------------------------------------------- the plain forms
def _rope_plain(case, xs, pos, inv_freq):
    angle = pos.to(torch.float64)[..., None] * inv_freq  # [B, S, pairs]
    if case["inverse"]:
        angle = -angle
    cos, sin = (f(angle).float()[:, :, None] * case["scale"] for f in (torch.cos, torch.sin))
    r = case["rope_dim"]
    outs = []
    for x in xs:
        f = x.float()
        a, b = (f[..., 0:r:2], f[..., 1:r:2]) if case["interleaved"] else (f[..., :r // 2], f[..., r // 2:r])
        u, w = a * cos - b * sin, a * sin + b * cos
        turned = torch.stack([u, w], -1).flatten(-2) if case["interleaved"] else torch.cat([u, w], -1)
        outs.append(torch.cat([turned, f[..., r:]], -1).to(x.dtype))
    return outs


def _hadamard(n, dtype):
    h = torch.ones((1, 1), dtype=dtype, device=DEV)
    while h.shape[0] < n:
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
    return h / math.sqrt(n)


def _dequantised(pages, dim, tile):
    """Rotated keys and values [..., pages * 16, dim] of page bytes [..., pages, bytes], whole tiles."""
    n, cols = tile // P, dim * P // tile
    kb, vb = 8 * dim, 4 * dim
    kp = kb + 8 * P + 4 * cols

    def scales(at):
        f = pages[..., at:at + 8 * P + 4 * cols].contiguous().view(torch.float32)
        c = f[..., 2 * P:].unflatten(-2, (-1, n)).flatten(-2)  # [..., tiles, dim]
        return f[..., :P, None], f[..., P:2 * P, None], c.repeat_interleave(n, -2)[..., None, :]

    x = pages[..., :kb].unflatten(-1, (dim // 64, 8, 4, 4, 2, 2))  # q, g, t, r, h, e
    x = torch.stack([x & 15, x >> 4], -7)  # hi
    d = x.dim() - 7
    x = x.movedim((d, d + 2, d + 1, d + 4, d + 5, d + 3, d + 6), (d, d + 1, d + 2, d + 3, d + 4, d + 5, d + 6))
    y = pages[..., kp:kp + vb].unflatten(-1, (dim // 64, 8, 4, 2, 4))  # q, g, t, w, c
    y = torch.stack([torch.stack([(y >> (2 * h + 4 * e)) & 3 for e in (0, 1)], -6) for h in (0, 1)], -7)
    d = y.dim() - 7
    y = y.movedim((d, d + 4, d + 1, d + 2, d + 5, d + 6, d + 3), (d, d + 1, d + 2, d + 3, d + 4, d + 5, d + 6))
    out = []
    for codes, at in ((x, kb), (y, kp + vb)):
        a, b, c = scales(at)
        codes = codes.reshape(*pages.shape[:-1], P, dim).float()
        out.append((c * (a * codes + b)).flatten(-3, -2))
    return out


def _attend(case, s, k, v, where, q):
    """Softmax attention of q [B, Q, Hkv, G, D] over k, v [B, Hkv, L, D] whose entry i is token where[b, i] (-1: none) of its sequence,
    and, for a shared prefix, over the prefix's keys and values first. Returns the scores' weights, their sum and largest score."""
    Q = q.shape[1]
    seen = s["lens"][:, None] - Q + 1 + torch.arange(Q, device=DEV)  # tokens query j sees
    ok = (where[:, None] >= 0) & (where[:, None] < seen[..., None])  # [B, Q, L]
    t = torch.einsum("bqhgd,bhld->bqhgl", q, k) * s["scale"]
    return torch.where(ok[:, :, None, None], t, -math.inf)


def _own_tokens(case, s, H):
    """Rotated keys and values of each sequence's own tokens (tiles in its pages, then raw tail rows) and their positions."""
    dim, tile = case["dim"], case["tile"]
    first = case.get("prefix", 0)
    table = s["table"][:, first // P:]
    k, v = _dequantised(s["cache"][table.clamp(min=0).long()].transpose(1, 2), dim, tile)
    end = first + s["done"] * tile  # tokens below are in pages
    at = first + torch.arange(k.shape[2], device=DEV)
    rows = torch.arange(s["tail_k"].shape[2], device=DEV)
    where = torch.cat([torch.where(at < end[:, None], at, -1), end[:, None] + rows], 1)
    where = torch.where(where < s["lens"][:, None], where, -1)
    return (torch.cat([k, s["tail_k"].float() @ H], 2), torch.cat([v, s["tail_v"].float() @ H], 2), where)


def _shared_plain(case, s):
    H = _hadamard(case["dim"], torch.float32)
    B, Q, Hkv = case["seqs"], case["queries"], case["kv_heads"]
    q = (s["q"].float() @ H).unflatten(2, (Hkv, -1))
    pages = s["cache"][s["prefix_table"].long()].transpose(0, 1)
    pk, pv = _dequantised(pages, case["dim"], case["tile"])  # [Hkv, prefix, D]
    k, v, where = _own_tokens(case, s, H)
    t0 = torch.einsum("bqhgd,hld->bqhgl", q, pk) * s["scale"]
    t1 = _attend(case, s, k, v, where, q)
    m = torch.maximum(t0.amax(-1), t1.amax(-1))[..., None]
    p0, p1 = torch.exp(t0 - m), torch.exp(t1 - m)
    l = p0.sum(-1) + p1.sum(-1)
    o = torch.einsum("bqhgl,hld->bqhgd", p0, pv) + torch.einsum("bqhgl,bhld->bqhgd", p1, v)
    out = (o / l[..., None]) @ H
    return out.reshape(s["q"].shape), (m[..., 0] + torch.log(l)).reshape(B, Q, -1)


def _mass_plain(case, s):
    H = _hadamard(case["dim"], torch.float32)
    B, Hkv, tile = case["seqs"], case["kv_heads"], case["tile"]
    q = (s["q"].float() @ H).view(B, 1, Hkv, -1, case["dim"])
    k, v, where = _own_tokens(case, s, H)
    t = _attend(case, s, k, v, where, q)
    m = t.amax(-1, keepdim=True)
    p = torch.exp(t - m)
    l = p.sum(-1, keepdim=True)
    p = p / l
    out = torch.einsum("bqhgl,bhld->bqhgd", p, v) @ H
    tiles = s["mass"].shape[1]
    got = p[..., :s["table"].shape[1] * P].unflatten(-1, (-1, tile)).sum(-1).sum((1, 2, 3))  # [B, tiles]
    got = torch.cat([got, got.new_zeros(B, max(0, tiles - got.shape[1]))], 1)[:, :tiles]
    new = case["decay"] * s["mass"] + got
    new = torch.where(torch.arange(tiles, device=DEV) < s["done"][:, None], new, 0.0)
    return out.reshape(s["q"].shape), (m + torch.log(l)).reshape(B, -1), new


def _evict_plain(case, lens, mass, table):
    tile, n = case["tile"], case["tile"] // P
    B, T = mass.shape
    tiles = torch.arange(T, device=DEV)
    done = (lens // tile)[:, None]
    cut = done > case["keep"]
    safe = (tiles < case["sink"]) | (tiles >= done - case["recent"])
    key = torch.where(safe, math.inf, mass)
    key = torch.where(tiles < done, key, -math.inf)
    order = torch.sort(key, dim=1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(1, order, tiles.expand(B, T))
    keep = (tiles < done) & (~cut | (rank < case["keep"]))
    drop = (tiles < done) & ~keep
    pages = table[:, :T * n].unflatten(1, (T, n))

    def compact(which, what, fill):
        at = torch.where(which, which.cumsum(1) - 1, T)
        at = at.view(B, T, *[1] * (what.dim() - 2)).expand(what.shape)
        out = torch.full((B, T + 1, *what.shape[2:]), fill, dtype=what.dtype, device=DEV)
        return out.scatter_(1, at, what)[:, :T]

    return (compact(keep, mass, 0.0), compact(keep, pages, -1).flatten(1), (lens - drop.sum(1) * tile).to(torch.int32),
            compact(drop, pages, -1).flatten(1), (drop.sum(1) * n).to(torch.int32))


# ------------------------------------------------------------------ the passes
def _layout(kv, case, s):
    return kv.dense_layout(case["dim"], case["tile"], case["kv_heads"], s["cache"].shape[0],
                           kv.BF16 if case["dtype"] == "bf16" else kv.FP16)


def run(state):
    case, s = state["case"], state
    op = case["op"]
    if own:
        import quantized_kv_cache_kvarn_gb300 as kv

        if op == "rope":
            turn = kv.rope_backward if case["inverse"] else kv.rope
            turn(s["xs"], s["outs"], s["pos"], s["inv_freq"], interleaved=case["interleaved"], scale=case["scale"])
            return s["outs"]
        if op == "evict":
            if "layout" not in s:
                s["layout"] = kv.dense_layout(128, case["tile"], 1, s["table"].numel())
            kv.evict_tiles(s["mass"], s["table"], s["lens"], s["layout"], case["len_max"], case["keep"], s["mass_out"],
                           s["table_out"], s["lens_out"], s["freed"], s["freed_count"], s["err"],
                           sink_tiles=case["sink"], recent_tiles=case["recent"])
            return s["mass_out"], s["table_out"], s["lens_out"], s["freed"], s["freed_count"]
        if "layout" not in s:  # kept by a serving program from step to step
            s["layout"] = _layout(kv, case, s)
            n = (kv.decode_shared_workspace_bytes(s["layout"], case["seqs"], case["q_heads"], case["queries"], s["max_len"],
                                                  case["prefix"]) if op == "shared" else
                 kv.decode_mass_workspace_bytes(s["layout"], case["seqs"], case["q_heads"], s["max_len"]))
            s["ws"] = torch.empty(n, dtype=torch.uint8, device=DEV)
        if op == "shared":
            kv.decode_shared(s["q"], s["layout"], s["cache"], s["prefix_table"], case["prefix"], s["table"], s["lens32"],
                             s["max_len"], s["out"], s["ws"], s["err"], s["scale"], s["tail_k"], s["tail_v"], s["lse"])
            return s["out"], s["lse"]
        kv.decode_mass(s["q"], s["layout"], s["cache"], s["table"], s["lens32"], s["max_len"], s["out"], s["mass"],
                       s["mass_out"], s["ws"], s["err"], s["scale"], s["tail_k"], s["tail_v"], s["lse"],
                       decay=case["decay"])
        return s["out"], s["lse"], s["mass_out"]
    if op == "rope":
        return _rope_plain(case, s["xs"], s["pos"], s["inv_freq"])
    if op == "evict":
        return _evict_plain(case, s["lens"], s["mass"], s["table"])
    return _shared_plain(case, s) if op == "shared" else _mass_plain(case, s)


# -------------------------------------------------------------------- the work
def work(case):
    op, B = case["op"], case["seqs"]
    if op == "rope":
        n = B * case["tokens"] * (case["q_heads"] + case["kv_heads"])
        size = 4 if case["dtype"] == "fp32" else 2
        return {"bytes": 2 * n * case["dim"] * size + 4 * B * case["tokens"], "flops": 3 * n * case["rope_dim"]}
    if op == "evict":
        tiles = (case["len_min"] + case["len_max"]) / 2 / case["tile"]
        one = 4 + 4 * (case["tile"] // P)  # a tile's mass and page ids
        return {"bytes": int(2 * B * tiles * one), "flops": int(2 * B * tiles)}
    dim, tile, Hkv, Hq, Q = case["dim"], case["tile"], case["kv_heads"], case["q_heads"], case.get("queries", 1)
    page_row = (12 * dim + 256 + 8 * dim * P // tile) / P  # bytes of a token of one KV head
    if op == "shared":
        first, own_len = case["prefix"], (case["suffix_min"] + case["suffix_max"]) / 2
    else:
        first, own_len = 0, (case["len_min"] + case["len_max"]) / 2
    raw = min(own_len, tile / 2 if own_len > tile else own_len)
    bytes_ = Hkv * (first * page_row + B * ((own_len - raw) * page_row + raw * 4 * dim)) + B * Q * Hq * dim * 6
    if op == "mass":
        bytes_ += 8 * B * own_len / tile
    return {"bytes": int(bytes_), "flops": int(4 * dim * B * Q * Hq * (first + own_len))}


# -------------------------------------------------------- the outputs in 64 bits
def _whole(sides, H):
    """Keys and values [units, heads, tile, dim] in the original basis, in 64 bits, from codes and scales."""
    return [(((a.double()[..., None] * codes.double() + b.double()[..., None]) * c.double()[..., None, :]) @ H)
            for codes, a, b, c in sides]


def _evicted(case, lens, mass, table):
    """The eviction sequence by sequence: among the unprotected tiles the lightest leave, of equal ones the last."""
    n = case["tile"] // P
    new_mass, new_table = torch.zeros_like(mass, dtype=torch.float64), torch.full_like(table, -1)
    freed, count, new_lens = torch.full_like(table, -1), torch.zeros_like(lens), lens.clone()
    for b, L in enumerate(lens.tolist()):
        done = L // case["tile"]
        gone = []
        if done > case["keep"]:
            m = mass[b].tolist()
            free = range(case["sink"], done - case["recent"])
            gone = sorted(sorted(free, key=lambda t: (m[t], -t))[:done - case["keep"]])
        left = sorted(set(range(done)) - set(gone))
        pages = table[b].unflatten(0, (-1, n))
        new_mass[b, :len(left)] = mass[b, left].double()
        new_table[b, :len(left) * n] = pages[left].flatten()
        freed[b, :len(gone) * n] = pages[gone].flatten()
        count[b] = len(gone) * n
        new_lens[b] = L - len(gone) * case["tile"]
    return new_mass, new_table, new_lens, freed, count


def exact(case, seed):
    op = case["op"]
    if op == "rope":
        xs, pos, inv_freq = _rope_inputs(case, seed)
        z = torch.polar(torch.full((), case["scale"], dtype=torch.float64, device=DEV),
                        (-1 if case["inverse"] else 1) * pos.double()[:, :, None, None] * inv_freq)
        r, outs = case["rope_dim"], []
        for x in xs:
            f = x.double()
            pair = f[..., :r].unflatten(-1, (-1, 2)) if case["interleaved"] else f[..., :r].unflatten(-1, (2, -1)).mT
            w = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * z)
            outs.append(torch.cat([w.flatten(-2) if case["interleaved"] else w.mT.flatten(-2), f[..., r:]], -1))
        return outs
    if op == "evict":
        return _evicted(case, *_evict_inputs(case, seed))
    s = _attention_inputs(case, seed)
    H = _hadamard(case["dim"], torch.float64)
    k, v = _whole(s["sides"], H)
    B, Hkv, tile, D = case["seqs"], case["kv_heads"], case["tile"], case["dim"]
    Q, G, first = case.get("queries", 1), case["q_heads"] // Hkv, case.get("prefix", 0) // tile
    outs, lses, tiles = [], [], []
    for b in range(B):
        n, L = int(s["done"][b]), int(s["lens"][b])
        at = torch.cat([torch.arange(first, device=DEV), s["index"][b, :n]])
        raw = L - (first + n) * tile

        def tokens(x, tail):
            x = x[at].transpose(0, 1).reshape(Hkv, -1, D)
            return torch.cat([x, tail[b, :, :raw].double()], 1)

        kb, vb = tokens(k, s["tail_k"]), tokens(v, s["tail_v"])
        q = s["q"][b].double().view(Q, Hkv, G, D).permute(1, 0, 2, 3)  # [Hkv, Q, G, D]
        t = torch.einsum("hqgd,hld->hqgl", q, kb) / math.sqrt(D)
        hidden = torch.arange(L, device=DEV) >= L - Q + 1 + torch.arange(Q, device=DEV)[:, None]
        t = t.masked_fill(hidden[None, :, None], -math.inf)
        lse = torch.logsumexp(t, -1)
        p = torch.exp(t - lse[..., None])
        outs.append(torch.einsum("hqgl,hld->qhgd", p, vb).reshape(Q, -1, D))
        lses.append(lse.transpose(0, 1).reshape(Q, -1))
        if op == "mass":
            tiles.append(p[..., :n * tile].unflatten(-1, (n, tile)).sum((0, 1, 2, 4)) if n else p.new_zeros(0))
    out, lse = torch.stack(outs), torch.stack(lses)
    if op == "shared":
        return out, lse
    before = _mass_before(case, seed).double()
    new = torch.zeros_like(before)
    for b, w in enumerate(tiles):
        new[b, :w.numel()] = case["decay"] * before[b, :w.numel()] + w
    return out[:, 0], lse[:, 0], new
