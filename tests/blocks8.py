"""Plain 64-bit statement of the 8-bit block cache and of its attention, for the tests: written from the
definitions in include/kvarn.h, one loop per index, sharing no code with the library."""
import math

import numpy as np
import torch

E4M3, INT8 = 0, 1
P = 16


def e4m3_values():
    """Value of every e4m3 byte: 1 sign, 4 exponent bits of bias 7, 3 mantissa bits; no infinities."""
    out = np.zeros(256)
    for b in range(256):
        e, m = b >> 3 & 15, b & 7
        v = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        out[b] = math.nan if b & 127 == 127 else -v if b & 128 else v
    return out


def code_bytes(x, code):
    """(code bytes, scale) of blocks x [..., 16, D] (float32 holding 16-bit values): the fp32 quotients and products of
    the definition are IEEE operations of numpy's float32."""
    x = np.asarray(x, np.float32)
    fine = np.isfinite(x).all((-2, -1))
    top = np.where(fine, np.maximum(np.abs(np.where(np.isfinite(x), x, 0)).max((-2, -1)), np.float32(2.0 ** -100)), 1)
    top = top.astype(np.float32)
    M, one = np.float32(127 if code == INT8 else 448), np.float32(1)
    scale, inv = np.where(fine, top * (one / M), np.float32(np.nan)).astype(np.float32), ((one / top) * M).astype(np.float32)
    y = (np.where(np.isfinite(x), x, 0) * inv[..., None, None]).astype(np.float32).astype(np.float64)
    y = np.where(fine[..., None, None], y, 0.0)
    if code == INT8:
        return (np.rint(y) + 128).astype(np.uint8), scale
    values = e4m3_values()[:127]  # the positive codes, ascending
    hi = np.clip(np.searchsorted(values, np.abs(y)), 0, 126)
    lo = np.maximum(hi - 1, 0)
    below, above = np.abs(y) - values[lo], values[hi] - np.abs(y)
    pick = np.where((below < above) | ((below == above) & (lo % 2 == 0)), lo, hi).astype(np.uint8)
    pick = np.where(np.abs(y) >= values[126], 126, pick).astype(np.uint8)
    return pick | np.where(np.signbit(y), 128, 0).astype(np.uint8), scale


def byte_values(b, code):
    return b.astype(np.float64) - 128 if code == INT8 else e4m3_values()[b]


def page_bytes(D):
    return 32 * D + 32


def pack_page(kb, ks, vb, vs):
    """One page from code bytes [16, D] of keys and values and their scales."""
    D = kb.shape[1]
    page = np.zeros(page_bytes(D), np.uint8)
    for tok in range(P):
        for ch in range(D):
            page[tok * D + 16 * ((ch // 16) ^ (4 * (tok % 2))) + ch % 16] = kb[tok, ch]
            nc, g, h, t, j = ch // 8, ch % 8, tok // 8, tok % 8 // 2, tok % 2
            page[16 * D + 16 * (32 * (nc // 4) + 4 * g + t) + 4 * (nc % 4) + j + 2 * h] = vb[tok, ch]
    page[32 * D:32 * D + 8] = np.array([ks, vs], np.float32).view(np.uint8)
    return page


def page_order(D):
    """Byte offsets within a page of key and value code (token, channel): two [16, D] arrays."""
    tok, ch = np.mgrid[0:P, 0:D]
    k = tok * D + 16 * ((ch // 16) ^ (4 * (tok % 2))) + ch % 16
    v = 16 * D + 16 * (32 * (ch // 32) + 4 * (ch % 8) + tok % 8 // 2) + 4 * (ch // 8 % 4) + tok % 2 + 2 * (tok // 8)
    return k, v


def values_of_cache(cache, D, code):
    """Keys and values [pages, heads, 16, D] in float64 of cache bytes [pages, heads, page]."""
    ko, vo = page_order(D)
    scales = np.ascontiguousarray(cache[..., 32 * D:32 * D + 8]).view(np.float32).astype(np.float64)
    return (byte_values(cache[..., ko], code) * scales[..., 0, None, None],
            byte_values(cache[..., vo], code) * scales[..., 1, None, None])


def attend(q, k, v, sm, L, window=0, sinks=0):
    """One sequence: q [Q, Hq, D], k and v [Hkv, L, D] in float64 -> out [Q, Hq, D], lse [Q, Hq], and how far fp32
    arithmetic may be from either.

    A score is a sum of D products in fp32: each of D / 16 tensor-core steps is off by at most 2^-23 of the sum of the
    products' magnitudes (truncation), each of D single additions of the raw rows by 2^-24, and scaling rounds three
    times: ds = sm (D / 2 + 4) 2^-23 sum |q_d k_d|. A weight then is off by ds + 2^-21 of itself (exp2, hi + lo operands,
    the scale's mantissa), the accumulators of the sum and the output by (n / 16 + 8) 2^-23 for n tokens, so an output,
    a quotient of two such sums, by twice that of the sum of its shares' magnitudes."""
    Q, Hq, D = q.shape
    G = Hq // k.shape[0]
    out, lse = np.zeros((Q, Hq, D)), np.full((Q, Hq), -math.inf)
    off, off_lse = np.zeros((Q, Hq, D)), np.zeros((Q, Hq))
    for j in range(Q):
        p = L - Q + j
        i = np.arange(L)
        seen = i <= p
        if window:
            seen &= (i < sinks) | (i > p - window)
        if not seen.any():
            continue
        for h in range(Hq):
            keys, values = k[h // G][seen], v[h // G][seen]
            s = sm * (keys @ q[j, h])
            m = s.max()
            w = np.exp(s - m)
            out[j, h] = w @ values / w.sum()
            lse[j, h] = m + np.log(w.sum())
            ds = abs(sm) * (D / 2 + 4) * 2.0 ** -23 * (np.abs(keys) @ np.abs(q[j, h]))
            # only the shares that count bring their error in
            each = (w @ ds / w.sum()) + 2.0 ** -21 + (len(s) / 16 + 8) * 2.0 ** -23
            off[j, h] = (w * ds) @ np.abs(values) / w.sum() + each * (w @ np.abs(values)) / w.sum() + 1e-30
            off_lse[j, h] = each + 2.0 ** -22 * abs(lse[j, h])
    return out, lse, off, off_lse


class Batch:
    """A batch on the GPU: raw keys and values of every sequence, the blocks that are whole before the newest Q
    tokens coded into pages in a random order, the rest in tails. Entries of the table for blocks that no query
    sees, and tail rows behind the last token, hold what must not be looked at."""

    def __init__(self, lens, Hq, Hkv, D, Q=1, window=0, sinks=0, code=E4M3, bf16=False, seed=0, cap=None, pad_columns=0):
        rng = np.random.default_rng(seed)
        self.lens, self.Hq, self.Hkv, self.D, self.Q, self.window, self.sinks, self.code = lens, Hq, Hkv, D, Q, window, sinks, code
        self.dt = torch.bfloat16 if bf16 else torch.float16
        self.bf16, self.sm = bf16, 1 / math.sqrt(D)
        B, self.max_len = len(lens), max(max(lens), 1)

        def half(x):
            return torch.from_numpy(np.asarray(x, np.float32)).to(self.dt).float().numpy()

        chan = np.exp(0.5 * rng.standard_normal((2, 1, Hkv, 1, D)))
        self.kv = [half(rng.standard_normal((B, Hkv, self.max_len, D)) * chan[n]) for n in (0, 1)]
        self.q = half(1.5 * rng.standard_normal((B, Q, Hq, D)))
        T = max(1, max(0, self.max_len - Q + 1) // P)
        done = [max(0, L - Q + 1) // P for L in lens]
        pages = max(1, sum(done))
        ids = rng.permutation(pages)
        cache = rng.integers(0, 120, (pages, Hkv, page_bytes(D))).astype(np.uint8)
        table = np.full((B, T + pad_columns), 0x7fffffff, np.int32)
        ko, vo = page_order(D)
        n = 0
        self.k, self.v = [], []  # what the queries attend over, float64 [Hkv, L, D]
        for b, L in enumerate(lens):
            parts = [[], []]
            for u in range(done[b]):
                page = ids[n]
                n += 1
                for side, order, x in ((0, ko, self.kv[0]), (1, vo, self.kv[1])):
                    block = x[b, :, u * P:u * P + P]
                    c, s = code_bytes(block, code)
                    cache[page][:, order] = c
                    cache[page, :, 32 * D + 4 * side:32 * D + 4 * side + 4] = s[:, None].view(np.uint8)
                    parts[side].append(byte_values(c, code) * s.astype(np.float64)[:, None, None])
                first = L - Q + 1 - window  # the first token that a window sees
                if not window or u * P < sinks or (u + 1) * P > first:
                    table[b, u] = page
            for side in (0, 1):
                parts[side].append(self.kv[side][b, :, done[b] * P:L].astype(np.float64))
            self.k.append(np.concatenate(parts[0], 1))
            self.v.append(np.concatenate(parts[1], 1))
        self.done, self.cache, self.table = done, cache, table
        cap = cap or P + Q - 1
        tails = np.full((2, B, Hkv, cap, D), np.nan, np.float32)
        for b, L in enumerate(lens):
            for side in (0, 1):
                tails[side, b, :, :L - done[b] * P] = self.kv[side][b, :, done[b] * P:L]
        self.tails = tails

    def expected(self):
        """out, lse and the largest errors of either."""
        rows = [attend(self.q[b].astype(np.float64), self.k[b], self.v[b], self.sm, L, self.window, self.sinks)
                for b, L in enumerate(self.lens)]
        return tuple(np.stack(x) for x in zip(*rows))

    def gpu(self, kv):
        """Tensors and the layout, as attributes."""
        B = len(self.lens)
        self.layout = kv.q8_layout(self.D, self.Hkv, self.cache.shape[0], kv.BF16 if self.bf16 else kv.FP16)
        self.t = dict(q=torch.from_numpy(self.q).to(self.dt).cuda(), cache=torch.from_numpy(self.cache).cuda(),
                      table=torch.from_numpy(self.table).cuda(), lens=torch.tensor(self.lens, dtype=torch.int32).cuda(),
                      tail_k=torch.from_numpy(self.tails[0]).to(self.dt).cuda(),
                      tail_v=torch.from_numpy(self.tails[1]).to(self.dt).cuda(), err=kv.new_error_word(),
                      out=torch.full((B, self.Q, self.Hq, self.D), 7.0, device="cuda"),
                      lse=torch.full((B, self.Q, self.Hq), 7.0, device="cuda"))
        n = kv.q8_decode_workspace_bytes(self.layout, B, self.Hq, self.Q, self.max_len, self.window, self.sinks)
        self.t["space"] = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
        return self

    def decode(self, kv, **more):
        t = {**self.t, **more}
        kv.q8_decode(t["q"], self.layout, self.code, t["cache"], t["table"], t["lens"], self.max_len, t["out"], t["space"],
                     t["err"], self.sm, t["tail_k"], t["tail_v"], t["lse"], window=self.window, sink_tokens=self.sinks,
                     stream=t.get("stream"))
        return t["out"], t["lse"]
