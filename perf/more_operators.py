"""What is measured of the operators around an 8-bit cache: norms of queries and keys with their rotation
in one pass (and their gradient), a cache of 8-bit codes with one scale per block of tokens and head
(written, read back, appended to, attended over with a sliding window and sinks), and the pages of a cache
whose sequences fork, end and leave their windows.

Each case names one operator and its sizes. ``prepare`` makes the inputs from the seed, ``run`` one pass:
the plain form (elementary torch operations in 32 bits, angles and long sums in 64) or, where ``own`` is
true, the library's calls. ``exact`` computes the same outputs in 64 bits.

The 8-bit pages hold 16 tokens of one KV head: key codes by token, value codes in the order of the decode's
operands, the two fp32 scales behind them; they are packed here in the documented format.
"""
import math

import torch

own = False

DEV = "cuda"
DT = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
P = 16  # tokens of a page, and of a block of the 8-bit cache
TOP = {"e4m3": 448.0, "int8": 127.0}
TINY = 2.0 ** -100  # the smallest magnitude that a block's scale stands for


# ------------------------------------------------------------------ the cases
def listed():
    def norm(name, seqs, tokens, q_heads, kv_heads, dim, rope_dim, dtype, interleaved=False, heads_first=False,
             grad=False, wide_weights=False, offset=0.0, far=131072, scale=1.0):
        return dict(name=name, op="norm", seqs=seqs, tokens=tokens, q_heads=q_heads, kv_heads=kv_heads, dim=dim,
                    rope_dim=rope_dim, dtype=dtype, interleaved=interleaved, heads_first=heads_first, grad=grad,
                    wide_weights=wide_weights, offset=offset, far=far, scale=scale)

    def store(name, seqs, kv_heads, dim, tokens, dtype, code, heads_first):
        return dict(name=name, op="store", seqs=seqs, kv_heads=kv_heads, dim=dim, tokens=tokens, dtype=dtype, code=code,
                    heads_first=heads_first)

    def decode(name, seqs, queries, q_heads, kv_heads, dim, len_min, len_max, window, sinks, dtype, code, append=False):
        return dict(name=name, op="decode", seqs=seqs, queries=queries, q_heads=q_heads, kv_heads=kv_heads, dim=dim,
                    len_min=len_min, len_max=len_max, window=window, sinks=sinks, dtype=dtype, code=code, append=append)

    def fork(name, seqs, beams, kv_heads, dim, tile, len_min, len_max, window=0, sinks=0, dtype="fp16"):
        return dict(name=name, op="fork", seqs=seqs, beams=beams, kv_heads=kv_heads, dim=dim, tile=tile, len_min=len_min,
                    len_max=len_max, window=window, sinks=sinks, dtype=dtype)

    def compact(name, pages, page_bytes, live, seqs, columns):
        return dict(name=name, op="compact", pages=pages, page_bytes=page_bytes, live=live, seqs=seqs, columns=columns)

    return [
        # one decode step of 32 sequences: the new token's 64 query and 8 key heads, each at its own position
        norm("norm_step", 32, 1, 64, 8, 128, 128, "fp16"),
        # a prompt chunk of four sequences before its keys are encoded
        norm("norm_prompt", 4, 4096, 64, 8, 128, 128, "bf16"),
        # the gradient of a training step's queries and keys, wide heads partly turned, an odd length
        norm("norm_grad", 2, 4093, 24, 4, 256, 64, "bf16", grad=True, wide_weights=True, offset=1.0),
        # a prompt chunk written to the cache and read back for the attention of the prompt's next chunk
        store("store_prompt", 4, 8, 128, 4096, "bf16", "e4m3", False),
        # wide heads, heads first, an odd number of sequences
        store("store_wide", 7, 4, 256, 2032, "fp16", "int8", True),
        # a few requests with a short window: append the newest token, then attend; latency counts
        decode("window_step", 4, 1, 4, 1, 128, 900, 1040, 512, 4, "fp16", "e4m3", append=True),
        # a batch of 16K contexts
        decode("decode_batch", 32, 1, 64, 8, 128, 16384, 16384, 0, 0, "fp16", "e4m3"),
        # long ragged contexts behind a window of 4096 tokens with four sinks, three tokens under verification
        decode("window_verify", 32, 3, 24, 4, 256, 2000, 65536, 4096, 4, "bf16", "int8"),
        # one step of beam search, 8 requests of 4 beams over compressed tiles
        fork("fork_beams", 32, 4, 8, 128, 128, 2000, 16384),
        # many sequences of an 8-bit cache that move on: some end, some fork, pages leave the window
        fork("fork_window", 512, 1, 8, 128, 16, 1, 32768, window=4096, sinks=4, dtype="bf16"),
        # a cache half of whose pages are free after evictions
        compact("compact_half", 32768, 15360, 0.5, 32, 512),
        # a small cache with few holes
        compact("compact_few", 1531, 8256, 0.9, 7, 200),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "store", "decode", "decode", "decode", "fork", "compact"])
    if op == "norm":
        dim = rng.choice([64, 96, 128, 256])
        heads = rng.choice([(4, 1), (16, 2), (24, 4), (64, 8), (32, 32), (7, 7)])
        dtype, grad = rng.choice(["fp16", "bf16", "fp32"]), rng.random() < 0.4
        per_token = (heads[0] + heads[1]) * dim * (4 if dtype == "fp32" else 2)
        seqs = _log(rng, 1, 64)
        return dict(op=op, seqs=seqs, tokens=_log(rng, 1, max(1, min(16384, 2 * 4096 * 72 * 256 // (per_token * seqs)))),
                    q_heads=heads[0], kv_heads=heads[1], dim=dim, rope_dim=rng.choice([dim, dim, dim // 2, 32]), dtype=dtype,
                    interleaved=rng.random() < 0.4, heads_first=rng.random() < 0.4, grad=grad,
                    wide_weights=rng.random() < 0.5, offset=rng.choice([0.0, 1.0]), far=_log(rng, 1000, 1 << 20),
                    scale=rng.choice([1.0, 1.35]))
    if op == "store":
        dim, heads, seqs = rng.choice([128, 256]), rng.choice([1, 2, 4, 8, 5]), _log(rng, 1, 64)
        return dict(op=op, seqs=seqs, kv_heads=heads, dim=dim,
                    tokens=P * _log(rng, 1, max(1, 4 * 4096 * 8 * 128 // (P * seqs * heads * dim))),
                    dtype=rng.choice(["fp16", "bf16"]), code=rng.choice(["e4m3", "int8"]), heads_first=rng.random() < 0.5)
    if op == "decode":
        dim = rng.choice([128, 128, 256])
        heads = rng.choice([(4, 1), (8, 8), (24, 4), (32, 8), (64, 8)])
        append = rng.random() < 0.4
        queries = 1 if append else rng.choice([1, 1, 2, 4, 8])
        seqs = _log(rng, 1, 48)
        window = rng.choice([0, 0, _log(rng, 1, 8192), _log(rng, 64, 8192)])
        most = 32 * 16384 * 8 * 128 // (seqs * heads[1] * dim * queries)
        top = max(20, _log(rng, 30, max(31, min(65536, most))))
        return dict(op=op, seqs=seqs, queries=queries, q_heads=heads[0], kv_heads=heads[1], dim=dim,
                    len_min=rng.randint(queries, top), len_max=top, window=window,
                    sinks=rng.choice([0, 1, 4, 37, 128]) if window else 0, dtype=rng.choice(["fp16", "bf16"]),
                    code=rng.choice(["e4m3", "int8"]), append=append)
    if op == "fork":
        tile = rng.choice([16, 64, 128])
        beams = rng.choice([1, 2, 4, 5])
        seqs = beams * _log(rng, 1, 256 // beams)
        top = _log(rng, 100, max(101, min(65536, 512 * 32768 // seqs)))
        window = rng.choice([0, _log(rng, 16, 8192)])
        return dict(op=op, seqs=seqs, beams=beams, kv_heads=rng.choice([1, 4, 8]), dim=rng.choice([128, 256]), tile=tile,
                    len_min=rng.randint(0, top), len_max=top, window=window, sinks=rng.choice([0, 4, 130]) if window else 0,
                    dtype=rng.choice(["fp16", "bf16"]))
    pages = _log(rng, 50, 32768)
    seqs = _log(rng, 1, 64)
    return dict(op=op, pages=pages, page_bytes=rng.choice([1920, 2304, 6528, 8256, 15360]), live=rng.choice([0.1, 0.5, 0.9, 0.99]),
                seqs=seqs, columns=max(1, min(pages // seqs, _log(rng, 4, 2048))))


# ----------------------------------------------------------------- the inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _lengths(lo, hi, n, g):
    """n lengths over [lo, hi], the last one hi."""
    x = torch.randint(lo, hi + 1, (n,), generator=g, device=DEV)
    x[-1] = hi
    return x


def _norm_inputs(case, seed):
    g = _gen(seed)
    dt, B, S, D = DT[case["dtype"]], case["seqs"], case["tokens"], case["dim"]
    wt = torch.float32 if case["wide_weights"] else dt
    xs, ws, dys = [], [], []
    for h in (case["q_heads"], case["kv_heads"]):
        shape = (B, h, S, D) if case["heads_first"] else (B, S, h, D)
        # activations of a projection: rows of different size, some channels larger
        big = 1 + 4 * (torch.rand(D, generator=g, device=DEV) < 0.03)
        for made in (xs, dys):
            x = torch.randn(shape, generator=g, device=DEV)
            if made is xs:
                x = x * big * torch.exp(0.7 * torch.randn((*shape[:-1], 1), generator=g, device=DEV))
            elif not case["grad"]:
                continue
            x = x.to(dt)
            made.append(x.transpose(1, 2) if case["heads_first"] else x)  # [B, S, heads, D]
        ws.append((1 - case["offset"] + 0.3 * torch.randn(D, generator=g, device=DEV)).to(wt))
    start = torch.randint(0, case["far"], (B, 1), generator=g, device=DEV)
    pos = (start + torch.arange(S, device=DEV)).to(torch.int32)
    i = torch.arange(case["rope_dim"] // 2, device=DEV, dtype=torch.float64)
    return xs, dys, ws, pos, 10000.0 ** (-2.0 * i / case["rope_dim"])


def _to_codes(x, code):
    """Blocks [..., 16, D] in fp32 -> (the values of their codes, the scale that each block's are in)."""
    top = x.abs().amax((-2, -1)).clamp(min=TINY)
    y = x * (TOP[code] / top)[..., None, None]
    y = y.to(torch.float8_e4m3fn).float() if code == "e4m3" else y.round()
    return y, top / TOP[code]


def _kv_like(shape, g):
    """Keys or values [..., tokens, D] as a model makes them: channels of different size, a few much larger."""
    c = torch.exp(0.5 * torch.randn((*shape[:-2], 1, shape[-1]), generator=g, device=DEV))
    c = torch.where(torch.rand(c.shape, generator=g, device=DEV) < 0.02, 3 * c, c)
    return torch.randn(shape, generator=g, device=DEV).mul_(c)


def _bytes_of(y, code):
    return y.to(torch.float8_e4m3fn).view(torch.uint8) if code == "e4m3" else (y + 128).to(torch.uint8)


def _pack(k, v, code):
    """Page bytes [..., bytes] of blocks given as (code values [..., 16, D], scales [...])."""
    D = k[0].shape[-1]
    kb = _bytes_of(k[0], code).unflatten(-1, (D // 128, 2, 4, 16))  # 16-byte units 8 a + 4 b + c
    odd = kb[..., 1::2, :, :, :, :].flip(-3)  # the two halves of 64 bytes swapped in odd tokens
    kb = torch.stack([kb[..., 0::2, :, :, :, :], odd], -5).flatten(-6)
    vb = _bytes_of(v[0], code).unflatten(-1, (D // 32, 4, 8)).unflatten(-4, (2, 4, 2))  # h, t, j, w, c, g
    d = vb.dim() - 6
    vb = vb.movedim((d, d + 1, d + 2, d + 3, d + 4, d + 5), (d + 4, d + 2, d + 5, d, d + 3, d + 1)).flatten(d)  # w, g, t, c, h, j
    scales = torch.stack([k[1], v[1]], -1).contiguous().view(torch.uint8)
    pad = torch.zeros((*scales.shape[:-1], 24), dtype=torch.uint8, device=DEV)
    return torch.cat([kb, vb, scales, pad], -1)


def _store_inputs(case, seed):
    g = _gen(seed)
    B, H, C, D, dt = case["seqs"], case["kv_heads"], case["tokens"], case["dim"], DT[case["dtype"]]
    k, v = (_kv_like((B, H, C, D), g).to(dt) for _ in range(2))
    if not case["heads_first"]:
        k, v = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (k, v))
    start = torch.randint(0, 64, (B,), generator=g, device=DEV).to(torch.int32)
    table = torch.randperm(B * (64 + C // P), generator=g, device=DEV).to(torch.int32).view(B, -1)
    return k, v, start, table


def _decode_inputs(case, seed, with_pages=True):
    g = _gen(seed)
    B, H, D, Q, dt = case["seqs"], case["kv_heads"], case["dim"], case["queries"], DT[case["dtype"]]
    W, S = case["window"], case["sinks"]
    lens = _lengths(case["len_min"], case["len_max"], B, g)
    done = (lens - Q + 1).clamp(min=0) // P  # blocks in pages
    T = max(1, (case["len_max"] - Q + 1) // P)
    at = torch.arange(T, device=DEV)
    seen = at < done[:, None]
    if W:  # blocks that no query sees have left the cache
        seen &= (at * P < S) | ((at + 1) * P > (lens - Q + 1 - W)[:, None])
    n = max(1, int(seen.sum()))
    unit = torch.where(seen, seen.flatten().cumsum(0).view(B, T) - 1, -1)
    ids = torch.randperm(n, generator=g, device=DEV)
    out = dict(lens=lens, done=done, unit=unit, table=torch.where(seen, ids[unit.clamp(min=0)], -1).to(torch.int32))
    out["q"] = (1.5 * torch.randn((B, Q, case["q_heads"], D), generator=g, device=DEV)).to(dt)
    tails = _kv_like((2, B, H, P + Q - 1, D), g).to(dt)
    out["tail_k"], out["tail_v"] = tails[0].contiguous(), tails[1].contiguous()
    if case["append"]:
        new = _kv_like((2, B, H, 1, D), g).to(dt)[..., 0, :]
        out["k"], out["v"] = new[0].contiguous(), new[1].contiguous()
    out["sides"] = k, v = [_to_codes(_kv_like((n, H, P, D), g).to(dt).float(), case["code"]) for _ in range(2)]
    if with_pages:
        pages = _pack(k, v, case["code"])
        out["cache"] = torch.empty_like(pages)
        out["cache"][ids] = pages
    return out


def _fork_inputs(case, seed):
    """Requests of `beams` sequences that share the first half of their tiles; new rows take beams of their
    own request (of any, where a request has one), a few end."""
    g = _gen(seed)
    B, n, N, k = case["seqs"], case["tile"] // P, case["tile"], case["beams"]
    lens = _lengths(case["len_min"], case["len_max"], B // k, g).repeat_interleave(k)
    T = max(1, case["len_max"] // N)
    done, at = (lens // N)[:, None], torch.arange(T, device=DEV)
    ids = torch.randperm((B * T * n * 5) // 4 + 8, generator=g, device=DEV).to(torch.int32)
    own_pages = ids[:B * T * n].view(B, T, n)
    first = own_pages.view(B // k, k, T, n)[:, :1].expand(-1, k, -1, -1).reshape(B, T, n)
    table = torch.where((at < done // 2)[..., None], first, own_pages)
    table = torch.where((at < done)[..., None], table, -1)
    if case["window"]:  # rows whose window has moved on before, and rows whose pages are still there
        left = ((at + 1) * N <= (lens[:, None] - 300 - case["window"])) & (at * N >= case["sinks"])
        table = torch.where(left[..., None], -1, table)
    table = table.flatten(1)
    refs = torch.zeros(ids.numel() + 1, dtype=torch.int32, device=DEV)
    refs.index_add_(0, table.flatten().long() % refs.numel(), torch.ones_like(table).flatten())
    refs = refs[:-1].contiguous()  # -1 counted in the entry behind the last
    held = torch.rand(refs.shape, generator=g, device=DEV) < 0.05
    refs += (held & (refs > 0)).to(torch.int32)  # some pages a prefix cache holds as well
    row = torch.arange(B, device=DEV)
    if k > 1:
        parents = row // k * k + torch.randint(0, k, (B,), generator=g, device=DEV)
    else:
        parents = torch.where(torch.rand(B, generator=g, device=DEV) < 0.05, torch.randint(0, B, (B,), generator=g, device=DEV), row)
        parents = torch.where(torch.rand(B, generator=g, device=DEV) < 0.03, -1, parents)
    tails = torch.randn((2, B, case["kv_heads"], N, case["dim"]), generator=g, device=DEV).to(DT[case["dtype"]])
    return dict(parents=parents.to(torch.int32), lens=lens.to(torch.int32), table=table.contiguous(), refs=refs,
                tail_k=tails[0].contiguous(), tail_v=tails[1].contiguous())


def _compact_inputs(case, seed, with_cache=True):
    g = _gen(seed)
    n = case["pages"]
    live = torch.rand(n, generator=g, device=DEV) < case["live"]
    refs = torch.where(live, torch.randint(1, 4, (n,), generator=g, device=DEV), 0).to(torch.int32)
    # rows name live pages (some of them twice) and have empty entries
    order = torch.argsort(live.to(torch.int8), descending=True, stable=True)
    pick = torch.randint(0, n, (case["seqs"], case["columns"]), generator=g, device=DEV) % live.sum().clamp(min=1)
    table = torch.where(live.any() & (torch.rand(pick.shape, generator=g, device=DEV) < 0.9), order[pick], -1).to(torch.int32)
    out = dict(refs=refs, table=table)
    if with_cache:
        out["cache"] = torch.randint(-2 ** 62, 2 ** 62, (n, case["page_bytes"] // 8), generator=g, device=DEV).view(torch.uint8)
    return out


def _word():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    op = case["op"]
    if op == "norm":
        xs, dys, ws, pos, inv_freq = _norm_inputs(case, seed)
        return dict(case=case, xs=xs, dys=dys, ws=ws, pos=pos, inv_freq=inv_freq, outs=[torch.empty_like(x) for x in xs],
                    dws=[torch.empty(case["dim"], dtype=torch.float32, device=DEV) for _ in xs])
    if op == "store":
        k, v, start, table = _store_inputs(case, seed)
        n = 32 * case["dim"] + 32
        return dict(case=case, k=k, v=v, start=start, table=table, err=_word(), outs=[torch.empty_like(k), torch.empty_like(v)],
                    cache=torch.zeros((table.numel(), case["kv_heads"], n), dtype=torch.uint8, device=DEV))
    if op == "decode":
        s = _decode_inputs(case, seed)
        s.pop("sides")
        s.update(case=case, err=_word(), lens32=s["lens"].to(torch.int32), scale=1.0 / math.sqrt(case["dim"]),
                 out=torch.empty(s["q"].shape, dtype=torch.float32, device=DEV),
                 lse=torch.empty(s["q"].shape[:-1], dtype=torch.float32, device=DEV))
        return s
    if op == "fork":
        s = _fork_inputs(case, seed)
        s.update(case=case, err=_word(), lens_out=torch.empty_like(s["lens"]), table_out=torch.empty_like(s["table"]),
                 refs_out=torch.empty_like(s["refs"]), freed=torch.empty_like(s["refs"]), freed_count=_word(),
                 tail_k_out=torch.zeros_like(s["tail_k"]), tail_v_out=torch.zeros_like(s["tail_v"]))
        return s
    s = _compact_inputs(case, seed)
    s.update(case=case, err=_word(), refs_out=torch.empty_like(s["refs"]), table_out=torch.empty_like(s["table"]),
             remap=torch.empty_like(s["refs"]), live=_word())
    return s


# ------------------------------------------------------------- the plain forms
def _turn(case, x, cos, sin):
    r = case["rope_dim"]
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if case["interleaved"] else (x[..., :r // 2], x[..., r // 2:r])
    u, w = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack([u, w], -1).flatten(-2) if case["interleaved"] else torch.cat([u, w], -1)
    return torch.cat([turned, x[..., r:]], -1)


def _norm_plain(case, xs, dys, ws, pos, inv_freq):
    angle = pos.to(torch.float64)[..., None] * inv_freq  # [B, S, pairs]
    cos, sin = (f(angle).float()[:, :, None] * case["scale"] for f in (torch.cos, torch.sin))

    def forward(x, w):
        f = x.float()
        z = f * torch.rsqrt(f.square().mean(-1, keepdim=True) + 1e-6) * (w.float() + case["offset"])
        return _turn(case, z, cos, sin).to(x.dtype)

    def backward(x, dy, w):
        f = x.float()
        r = torch.rsqrt(f.square().mean(-1, keepdim=True) + 1e-6)
        h = f * r
        g = _turn(case, dy.float(), cos, -sin)
        dh = g * (w.float() + case["offset"])
        dx = r * (dh - h * (dh * h).mean(-1, keepdim=True))
        return dx.to(x.dtype), (g * h).sum((0, 1, 2), dtype=torch.float64).float()

    if case["grad"]:
        return [backward(*t) for t in zip(xs, dys, ws)]
    return [forward(*t) for t in zip(xs, ws)]


def _store_plain(case, k, v):
    def back(x):
        y, scale = _to_codes(x.float().unflatten(2, (-1, P)), case["code"])
        return (y * scale[..., None, None]).flatten(2, 3).to(x.dtype)

    return back(k), back(v)


def _values_of_pages(pages, code, D):
    """Keys and values [..., 16, D] of page bytes [..., bytes]."""
    def values(b):
        return b.view(torch.float8_e4m3fn).float() if code == "e4m3" else b.float() - 128

    k = pages[..., :P * D].unflatten(-1, (8, 2, D // 128, 2, 4, 16))
    k = torch.stack([k.select(-5, 0), k.select(-5, 1).flip(-3)], -5).flatten(-4).flatten(-3, -2)
    v = pages[..., P * D:2 * P * D].unflatten(-1, (D // 32, 8, 4, 4, 2, 2))  # w, g, t, c, h, j
    d = v.dim() - 6
    v = v.movedim((d, d + 1, d + 2, d + 3, d + 4, d + 5), (d + 3, d + 5, d + 1, d + 4, d, d + 2)).flatten(d + 3).flatten(d, d + 2)
    scales = pages[..., 2 * P * D:2 * P * D + 8].contiguous().view(torch.float32)
    return values(k.contiguous()) * scales[..., :1, None], values(v.contiguous()) * scales[..., 1:, None]


def _decode_plain(case, s):
    B, Q, D, W, S = case["seqs"], case["queries"], case["dim"], case["window"], case["sinks"]
    L, done, T = s["lens"][:, None], s["done"][:, None], s["table"].shape[1]
    # the pages that queries can see: those of the sinks, and those from the window's start on
    first = min(T, -(-S // P)) if W else 0
    count = min(T, (W + Q - 1) // P + 2) if W else T
    start = torch.clamp((L - Q + 1 - W) // P, min=first) if W else torch.zeros_like(L)
    page = torch.cat([torch.arange(first, device=DEV).expand(B, first), start + torch.arange(count, device=DEV)], 1)
    ids = s["table"].gather(1, page.clamp(max=T - 1))
    k, v = _values_of_pages(s["cache"][ids.clamp(min=0).long()].transpose(1, 2), case["code"], D)  # [B, H, pages, 16, D]
    where = page[..., None] * P + torch.arange(P, device=DEV)
    tail_k, tail_v, whole = s["tail_k"], s["tail_v"], done
    if case["append"]:  # the newest token in its row of the tail, or the block that it completes
        whole = (L - 1) // P
        full = (L % P == 0)[..., None, None]
        row = (torch.arange(P, device=DEV) == (L - 1) % P)[:, None, :, None]
        raw = [torch.where(row, s[n][:, :, None], s["tail_" + n][:, :, :P]) for n in "kv"]
        block = [torch.where(full, (lambda y, a: y * a[..., None, None])(*_to_codes(x.float(), case["code"])), x.float()) for x in raw]
        kept = [torch.where(full, s["tail_" + n], torch.cat([x, s["tail_" + n][:, :, P:]], 2)) for n, x in zip("kv", raw)]
        tail_k, tail_v = block
    where = torch.where(page[..., None] < whole[..., None], where, -1).flatten(1)
    rest = whole * P + torch.arange(tail_k.shape[2], device=DEV)
    where = torch.cat([where, torch.where(rest < L, rest, -1)], 1)
    k, v = torch.cat([k.flatten(2, 3), tail_k.float()], 2), torch.cat([v.flatten(2, 3), tail_v.float()], 2)
    at = (L - Q + torch.arange(Q, device=DEV))[..., None]  # positions of the queries
    i = where[:, None]
    ok = (i >= 0) & (i <= at)
    if W:
        ok &= (i < S) | (i > at - W)
    q = s["q"].float().unflatten(2, (case["kv_heads"], -1))
    t = torch.einsum("bqhgd,bhld->bqhgl", q, k) * s["scale"]
    t = torch.where(ok[:, :, None, None], t, -math.inf)
    m = t.amax(-1, keepdim=True)
    p = torch.exp(t - m)
    l = p.sum(-1, keepdim=True)
    out = (torch.einsum("bqhgl,bhld->bqhgd", p, v) / l).reshape(s["q"].shape)
    lse = (m + torch.log(l)).reshape(s["q"].shape[:-1])
    return (out, lse, *kept) if case["append"] else (out, lse)


def _in_order(which, what, size, fill=-1):
    """The entries of `what` that `which` marks, in their order, then `fill`."""
    at = torch.where(which, which.cumsum(0) - 1, size)
    return torch.full((size + 1,), fill, dtype=what.dtype, device=DEV).scatter_(0, at, what)[:size]


def _fork_plain(case, s):
    N, n = case["tile"], case["tile"] // P
    p, alive = s["parents"].clamp(min=0).long(), s["parents"] >= 0
    lens = torch.where(alive, s["lens"][p], 0)
    T = s["table"].shape[1] // n
    at = torch.arange(T, device=DEV).repeat_interleave(n)
    before = at < s["lens"][:, None] // N  # entries that the old rows hold
    keep = before
    if case["window"]:  # what the next token's window and the sinks still see
        keep = before & ((at * N < case["sinks"]) | ((at + 1) * N > s["lens"][:, None] + 1 - case["window"]))
    kept = torch.where(keep, s["table"], -1)
    table = torch.where(alive[:, None], kept[p], -1)
    pages = s["refs"].numel()

    def counted(t):
        c = torch.zeros(pages + 1, dtype=torch.int32, device=DEV)
        return c.index_add_(0, torch.where(t >= 0, t, pages).flatten().long(), torch.ones_like(t).flatten())[:pages]

    refs = s["refs"] + counted(table) - counted(torch.where(before, s["table"], -1))
    gone = (s["refs"] > 0) & (refs <= 0)
    freed = _in_order(gone, torch.arange(pages, device=DEV, dtype=torch.int32), pages)
    live = torch.arange(N, device=DEV) < (lens % N)[:, None]

    def rows(x):
        return torch.where(live[:, None, :, None], x[p], torch.zeros((), dtype=x.dtype, device=DEV))

    return lens, table, refs, freed, gone.sum(dtype=torch.int32).view(1), rows(s["tail_k"]), rows(s["tail_v"])


def _compact_plain(case, s):
    live = s["refs"] > 0
    n, at = live.sum(), torch.arange(live.numel(), device=DEV)
    hole, mover = ~live & (at < n), live & (at >= n)
    size = live.numel()
    holes, movers = _in_order(hole, at, size), _in_order(mover, at, size)
    remap = torch.where(live, at, -1)
    remap = torch.cat([remap, remap[:1]]).scatter_(0, torch.where(movers >= 0, movers, size), holes)[:size]
    source = torch.cat([at, at[:1]]).scatter_(0, torch.where(holes >= 0, holes, size), movers)[:size]
    refs = torch.where(at < n, s["refs"][source], 0)
    table = torch.where(s["table"] >= 0, remap[s["table"].clamp(min=0).long()].to(torch.int32), -1)
    return s["cache"][source], refs, table, remap.to(torch.int32), n.to(torch.int32).view(1)


# ------------------------------------------------------------------ the passes
def run(state):
    case, s = state["case"], state
    op = case["op"]
    if own:
        import quantized_kv_cache_kvarn_gb300 as kv

        if op == "norm":
            more = dict(eps=1e-6, weight_offset=case["offset"], interleaved=case["interleaved"], scale=case["scale"])
            if not case["grad"]:
                kv.norm_rope(s["xs"], s["outs"], s["ws"], s["pos"], s["inv_freq"], **more)
                return s["outs"]
            if "ws_bytes" not in s:  # kept by a program from step to step
                s["ws_bytes"] = kv.norm_rope_backward_workspace_bytes(s["xs"])
                s["space"] = torch.empty(s["ws_bytes"], dtype=torch.uint8, device=DEV)
            kv.norm_rope_backward(s["xs"], s["dys"], s["outs"], s["ws"], s["dws"], s["pos"], s["inv_freq"], s["space"], **more)
            return [(dx, dw) for dx, dw in zip(s["outs"], s["dws"])]
        if op == "compact":
            if "space" not in s:
                s["space"] = torch.empty(kv.compact_pages_workspace_bytes(case["pages"]), dtype=torch.uint8, device=DEV)
            kv.compact_pages(s["cache"], s["refs"], s["table"], s["refs_out"], s["table_out"], s["remap"], s["live"],
                             s["space"], s["err"])
            return s["cache"], s["refs_out"], s["table_out"], s["remap"], s["live"]
        if "layout" not in s:
            kind = kv.BF16 if case["dtype"] == "bf16" else kv.FP16
            pages = s["refs"].numel() if op == "fork" else s["cache"].shape[0]
            if op == "fork" and case["tile"] != P:
                s["layout"] = kv.dense_layout(case["dim"], case["tile"], case["kv_heads"], pages, kind)
            else:
                s["layout"] = kv.q8_layout(case["dim"], case["kv_heads"], pages, kind)
            s["code"] = kv.Q8_INT8 if case.get("code") == "int8" else kv.Q8_E4M3
        if op == "store":
            kv.q8_encode_blocks(s["k"], s["v"], s["layout"], s["code"], s["start"], s["table"], s["cache"], s["err"])
            kv.q8_read_blocks(s["outs"][0], s["outs"][1], s["layout"], s["code"], s["start"], s["table"], s["cache"], s["err"])
            return s["outs"]
        if op == "fork":
            kv.fork_sequences(s["parents"], s["lens"], s["table"], s["refs"], s["layout"], case["len_max"], s["lens_out"],
                              s["table_out"], s["refs_out"], s["freed"], s["freed_count"], s["err"],
                              tails=((s["tail_k"], s["tail_k_out"]), (s["tail_v"], s["tail_v_out"])),
                              window=case["window"], sink_tokens=case["sinks"])
            return (s["lens_out"], s["table_out"], s["refs_out"], s["freed"], s["freed_count"], s["tail_k_out"],
                    s["tail_v_out"])
        if "space" not in s:
            n = kv.q8_decode_workspace_bytes(s["layout"], case["seqs"], case["q_heads"], case["queries"], case["len_max"],
                                             case["window"], case["sinks"])
            s["space"] = torch.empty(n, dtype=torch.uint8, device=DEV)
        if case["append"]:
            kv.q8_append(s["k"], s["v"], s["layout"], s["code"], s["lens32"], case["len_max"], s["tail_k"], s["tail_v"],
                         s["table"], s["cache"], s["err"])
        kv.q8_decode(s["q"], s["layout"], s["code"], s["cache"], s["table"], s["lens32"], case["len_max"], s["out"],
                     s["space"], s["err"], s["scale"], s["tail_k"], s["tail_v"], s["lse"], window=case["window"],
                     sink_tokens=case["sinks"])
        return (s["out"], s["lse"], s["tail_k"], s["tail_v"]) if case["append"] else (s["out"], s["lse"])
    if op == "norm":
        return _norm_plain(case, s["xs"], s["dys"], s["ws"], s["pos"], s["inv_freq"])
    if op == "store":
        return _store_plain(case, s["k"], s["v"])
    if op == "decode":
        return _decode_plain(case, s)
    return _fork_plain(case, s) if op == "fork" else _compact_plain(case, s)


# -------------------------------------------------------------------- the work
def work(case):
    op = case["op"]
    if op == "norm":
        n = case["seqs"] * case["tokens"] * (case["q_heads"] + case["kv_heads"]) * case["dim"]
        size = 4 if case["dtype"] == "fp32" else 2
        return {"bytes": (3 if case["grad"] else 2) * n * size + 4 * case["seqs"] * case["tokens"],
                "flops": (16 if case["grad"] else 8) * n}
    if op == "store":
        n = 2 * case["seqs"] * case["kv_heads"] * case["tokens"] * case["dim"]  # read and written, codes written and read
        return {"bytes": 6 * n, "flops": 4 * n}
    if op == "decode":
        B, Q, D, W, S = case["seqs"], case["queries"], case["dim"], case["window"], case["sinks"]
        length = (case["len_min"] + case["len_max"]) / 2
        seen = min(length, W + S + Q - 1) if W else length
        raw = min(seen, 8 + Q)
        rows = B * Q * case["q_heads"]
        return {"bytes": int(B * case["kv_heads"] * ((seen - raw) * (2 * D + 0.5) + raw * 4 * D) + rows * (6 * D + 4)),
                "flops": int(4 * D * rows * (min(seen, W + S) if W else seen))}
    if op == "fork":
        B, N = case["seqs"], case["tile"]
        length = (case["len_min"] + case["len_max"]) / 2
        entries, raw = B * length / P, B * case["kv_heads"] * case["dim"] * min(length, N / 2)
        return {"bytes": int(8 * entries + 10 * case["len_max"] / P * B * 1.25 + 8 * raw), "flops": int(4 * entries)}
    n, live = case["pages"], case["live"]
    return {"bytes": int(2 * n * live * (1 - live) * case["page_bytes"] + 12 * n + 8 * case["seqs"] * case["columns"]),
            "flops": 4 * n}


# -------------------------------------------------------- the outputs in 64 bits
def _norm_exact(case, seed):
    xs, dys, ws, pos, inv_freq = _norm_inputs(case, seed)
    z = torch.polar(torch.full((), case["scale"], dtype=torch.float64, device=DEV), pos.double()[:, :, None, None] * inv_freq)
    r, outs = case["rope_dim"], []

    def forward(x, w):
        y = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / case["dim"] + 1e-6) * (w + case["offset"])
        pair = y[..., :r].unflatten(-1, (-1, 2)) if case["interleaved"] else y[..., :r].unflatten(-1, (2, -1)).mT
        t = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * z)
        return torch.cat([t.flatten(-2) if case["interleaved"] else t.mT.flatten(-2), y[..., r:]], -1)

    for i, (x, w) in enumerate(zip(xs, ws)):
        x, w = x.double(), w.double()
        if case["grad"]:
            x.requires_grad_(True), w.requires_grad_(True)
            outs.append(torch.autograd.grad(forward(x, w), (x, w), dys[i].double()))
        else:
            outs.append(forward(x, w))
    return outs


def _code_values(x, code):
    """The block codec value by value: the fp32 quotients and product it is defined with, rounded in 64 bits."""
    top = x.double().abs().flatten(-2).max(-1).values.clamp(min=TINY)
    scale, inverse = ((a).float().double()[..., None, None] for a in (top / TOP[code], TOP[code] / top))
    y = (x.double() * inverse).float().double()
    if code == "e4m3":
        step = 2.0 ** (torch.frexp(y).exponent.clamp(min=-5) - 4).double()  # eight steps to an octave, down to 2^-6
        return torch.round(y / step) * step * scale
    return torch.round(y) * scale


def _decode_exact(case, seed):
    s = _decode_inputs(case, seed, with_pages=False)
    H, Q, D, W, S = case["kv_heads"], case["queries"], case["dim"], case["window"], case["sinks"]
    G = case["q_heads"] // H
    outs, lses, tails = [], [], [s["tail_k"].clone().double(), s["tail_v"].clone().double()]
    for b, L in enumerate(s["lens"].tolist()):
        done = max(0, L - Q + 1) // P
        whole = (L - 1) // P if case["append"] else done
        unit = s["unit"][b, :whole]
        have = unit >= 0
        at = (torch.arange(whole, device=DEV)[have][:, None] * P + torch.arange(P, device=DEV)).flatten()
        at = torch.cat([at, torch.arange(whole * P, L, device=DEV)])
        kvs = []
        for n, (y, a) in enumerate(s["sides"]):
            x = (y[unit[have]].double() * a[unit[have]].double()[..., None, None]).transpose(0, 1).reshape(H, -1, D)
            rest = s["tail_kv"[:5] + "kv"[n]][b].clone()
            if case["append"]:
                rest[:, (L - 1) % P] = s["kv"[n]][b]
                if L % P:
                    tails[n][b] = rest.double()
                else:
                    rest = _code_values(rest[:, :P], case["code"])
            kvs.append(torch.cat([x, rest[:, :L - whole * P].double()], 1))
        q = s["q"][b].double().view(Q, H, G, D).transpose(0, 1)  # [H, Q, G, D]
        t = torch.einsum("hqgd,hld->hqgl", q, kvs[0]) / math.sqrt(D)
        p = L - Q + torch.arange(Q, device=DEV)[:, None]
        hidden = at > p
        if W:
            hidden |= (at >= S) & (at <= p - W)
        t = t.masked_fill(hidden[None, :, None], -math.inf)
        lse = torch.logsumexp(t, -1)
        outs.append(torch.einsum("hqgl,hld->qhgd", torch.exp(t - lse[..., None]), kvs[1]).reshape(Q, -1, D))
        lses.append(lse.transpose(0, 1).reshape(Q, -1))
    out = (torch.stack(outs), torch.stack(lses))
    return (*out, *tails) if case["append"] else out


def _fork_exact(case, seed):
    s = {n: t.cpu() for n, t in _fork_inputs(case, seed).items()}
    N, n, refs = case["tile"], case["tile"] // P, s["refs"].clone().numpy()
    lens, table = torch.zeros_like(s["lens"]), torch.full_like(s["table"], -1)
    tails = [torch.zeros_like(s["tail_k"], dtype=torch.float64), torch.zeros_like(s["tail_v"], dtype=torch.float64)]
    old = s["table"].numpy()
    for a, L in enumerate(s["lens"].tolist()):
        for page in old[a, :L // N * n]:
            refs[page] -= page >= 0
    for b, a in enumerate(s["parents"].tolist()):
        if a < 0:
            continue
        L = lens[b] = int(s["lens"][a])
        for i in range(L // N * n):
            t = i // n * N
            if not case["window"] or t < case["sinks"] or t + N > L + 1 - case["window"]:
                table[b, i] = page = int(old[a, i])
                refs[page] += page >= 0
        for new, x in zip(tails, (s["tail_k"], s["tail_v"])):
            new[b, :, :L % N] = x[a, :, :L % N].double()
    gone = [i for i, (x, y) in enumerate(zip(s["refs"].tolist(), refs.tolist())) if x > 0 and y <= 0]
    freed = torch.full_like(s["refs"], -1)
    freed[:len(gone)] = torch.tensor(gone, dtype=torch.int32)
    return lens, table, torch.from_numpy(refs), freed, torch.tensor([len(gone)], dtype=torch.int32), *tails


def exact(case, seed):
    op = case["op"]
    if op == "norm":
        return _norm_exact(case, seed)
    if op == "store":
        k, v, _, _ = _store_inputs(case, seed)
        return [_code_values(x.unflatten(2, (-1, P)), case["code"]).flatten(2, 3) for x in (k, v)]
    if op == "decode":
        return _decode_exact(case, seed)
    if op == "fork":
        return _fork_exact(case, seed)
    return None  # pages and whole numbers alone
