"""Inputs and error bounds shared by the tests of the serving operators
around the cache (shared-prefix decode, tile masses, eviction)."""
from __future__ import annotations

import numpy as np
import torch

import quantized_kv_cache_kvarn_gb300 as kv
from oracle import attention, layout
from tests import parity


class Batch:
    """Sequences over pages the oracle wrote: a shared prefix (whole tiles,
    possibly none) and each sequence's own tokens, the last ones raw."""

    def __init__(self, D, N, Hq, Hkv, lens, Q=1, prefix=0, dtype=torch.float16, widths=(4, 2, 4), seed=0, peak=2.0,
                 size=1.0, first=1.0):
        g = torch.Generator().manual_seed(seed)
        kb, vb, sb = widths
        self.D, self.N, self.Hq, self.Hkv, self.Q, self.prefix, self.dtype = D, N, Hq, Hkv, Q, prefix, dtype
        self.lens = np.array(lens, np.int32)
        B = len(lens)
        self.lay = layout.DenseLayout(D, N, kb, vb, sb)
        self.widths = widths
        ppt = N // 16
        ends = [max(prefix, attention.verify_committed(int(L), Q, N)) for L in lens]
        tiles = prefix // N + sum((e - prefix) // N for e in ends)
        num_pages = max(1, tiles * ppt)
        order = np.random.default_rng(seed).permutation(num_pages).astype(np.int32)
        self.cache = np.zeros((num_pages, Hkv, self.lay.page_bytes), np.uint8)
        longest = max([prefix] + ends)
        self.bt = np.full((B, max(1, longest // 16)), -1, np.int32)
        self.prefix_table = order[:prefix // 16].copy()

        def rows(n):  # [1, Hkv, n, D], one channel of ten larger; the values' size, and the first tile's
            x = size * torch.randn((1, Hkv, n, D), generator=g)
            x[..., ::10] *= 3.0
            x[:, :, :N] *= first if n == prefix else 1.0
            return x.to(dtype)

        if prefix:
            attention.encode_into_cache(self.cache, self.lay, parity.f64(rows(prefix)), parity.f64(rows(prefix)),
                                        self.prefix_table[None], [0])
        at = prefix // 16
        cap = N + Q - 1  # decode_mass takes N rows, the others at least N + Q - 2
        self.tail_k = torch.full((B, Hkv, cap, D), float("nan"), dtype=dtype)  # rows past a tail are never read
        self.tail_v = torch.full_like(self.tail_k, float("nan"))
        for b, (L, e) in enumerate(zip(lens, ends)):
            n = (e - prefix) // 16
            if n:
                self.bt[b, prefix // 16:e // 16] = order[at:at + n]
                own = rows(e - prefix), rows(e - prefix)
                attention.encode_into_cache(self.cache, self.lay, parity.f64(own[0]), parity.f64(own[1]),
                                            self.bt[b:b + 1], [prefix // N])
                at += n
            if L > e:
                self.tail_k[b, :, :L - e], self.tail_v[b, :, :L - e] = rows(L - e)[0], rows(L - e)[0]
        self.q = (peak / size * torch.randn((B, Q, Hq, D), generator=g)).to(dtype)
        self.sm = 1.0 / np.sqrt(D)

    def full_table(self):
        """Block table whose rows name the prefix's pages too."""
        t = self.bt.copy()
        t[:, :self.prefix // 16] = self.prefix_table
        return t

    def layout_of(self):
        kb, vb, sb = self.widths
        return kv.dense_layout(self.D, self.N, self.Hkv, self.cache.shape[0],
                               kv.BF16 if self.dtype == torch.bfloat16 else kv.FP16, k_bits=kb, v_bits=vb,
                               fp16_scales=sb == 2)

    def oracle(self):
        tk, tv = (np.nan_to_num(parity.f64(t)) for t in (self.tail_k, self.tail_v))
        return attention.decode_verify(parity.f64(self.q), self.cache, self.lay, self.full_table(), self.lens, self.sm,
                                       tk, tv)

    def reference(self, device="cuda"):
        """oracle() for many rows over a long prefix: the same definition, the
        prefix dequantised once and the sums in 64 bits on the GPU."""
        B, Q, Hq, Hkv, D, P = len(self.lens), self.Q, self.Hq, self.Hkv, self.D, self.prefix
        G = Hq // Hkv
        out, lse = np.zeros((B, Q, Hq, D)), np.full((B, Q, Hq), -np.inf)
        q = torch.from_numpy(parity.f64(self.q)).to(device)
        tk, tv = (np.nan_to_num(parity.f64(t)) for t in (self.tail_k, self.tail_v))
        for h in range(Hkv):
            pk, pv = (torch.from_numpy(np.ascontiguousarray(x)).to(device)
                      for x in attention.sequence_kv(self.cache, self.lay, self.prefix_table, P, h))
            for b, L in enumerate(self.lens):
                if L == 0:
                    continue
                end = max(P, attention.verify_committed(int(L), Q, self.N))
                ok, ov = attention.sequence_kv(self.cache, self.lay, self.bt[b, P // 16:], end - P, h) if end > P else \
                    (np.zeros((0, D)), np.zeros((0, D)))
                k, v = (torch.cat([a, torch.from_numpy(np.concatenate([o, t[b, h, :L - end]])).to(device)])
                        for a, o, t in ((pk, ok, tk), (pv, ov, tv)))
                qb = q[b, :, h * G:(h + 1) * G]  # [Q, G, D]
                s = self.sm * torch.einsum("qgd,ld->qgl", qb, k)
                seen = torch.tensor([attention.verify_visible(int(L), Q, j) for j in range(Q)], device=device)
                s = s.masked_fill(torch.arange(len(k), device=device) >= seen[:, None, None], -torch.inf)
                z = torch.logsumexp(s, -1)
                out[b, :, h * G:(h + 1) * G] = torch.einsum("qgl,ld->qgd", torch.exp(s - z[..., None]), v).cpu().numpy()
                lse[b, :, h * G:(h + 1) * G] = z.cpu().numpy()
        return out, lse

    def bounds(self):
        """(score error, output error) bounds of the decode arithmetic. A
        score is a sum of 2^-22-exact products and of at most 64 fp32 or
        tensor-core accumulation steps, each off by at most 2^-23 of the sum
        of magnitudes A = sum_j |q'_j| c_j (|a| code + |b|): (1/4 + 64) 2^-23
        A < 2^-17 A, A over the largest code, the largest scales and the
        longest query. The weights are then off by 2^-17 A + 2^-20 relative
        (exp2, sums), the output by twice that plus the same kind of
        accumulation error, 2^-17, of the largest value magnitude."""
        qmax_k, qmax_v = (1 << self.widths[0]) - 1, (1 << self.widths[1]) - 1
        q1 = float(np.abs(parity.f64(self.q) @ _hadamard(self.D)).sum(-1).max())
        raw_q1 = float(np.abs(parity.f64(self.q)).sum(-1).max())
        A = V = 0.0
        ppt = self.N // 16
        for row in [self.prefix_table] + [r[self.prefix // 16:] for r in self.bt]:
            pages = [int(x) for x in row if x >= 0]
            for t in range(len(pages) // ppt):
                for h in range(self.Hkv):
                    k, v = layout.read_tile(self.cache, self.lay, pages[t * ppt:(t + 1) * ppt], h)
                    A = max(A, q1 * float(np.abs(k["c"]).max() * (np.abs(k["a"]).max() * qmax_k + np.abs(k["b"]).max())))
                    V = max(V, float(np.abs(v["c"]).max() * (np.abs(v["a"]).max() * qmax_v + np.abs(v["b"]).max())))
        raw_k, raw_v = (np.abs(np.nan_to_num(parity.f64(t))).max() for t in (self.tail_k, self.tail_v))
        A = max(A, raw_q1 * float(raw_k)) * self.sm
        V = max(V, float(raw_v))
        score = 2.0 ** -17 * A
        return score, (2 * (score + 2.0 ** -20) + 2.0 ** -17) * V


def _hadamard(n):
    h = np.ones((1, 1))
    while h.shape[0] < n:
        h = np.block([[h, h], [h, -h]])
    return h / np.sqrt(n)


def run_shared(x: Batch, dev="cuda", stream=None, ws=None):
    lay = x.layout_of()
    B = len(x.lens)
    Lmax = int(x.lens.max())
    out = torch.full((B, x.Q, x.Hq, x.D), float("nan"), dtype=torch.float32, device=dev)
    lse = torch.full((B, x.Q, x.Hq), float("nan"), dtype=torch.float32, device=dev)
    n = kv.decode_shared_workspace_bytes(lay, B, x.Hq, x.Q, Lmax, x.prefix)
    ws = torch.full((n,), 0xff, dtype=torch.uint8, device=dev)  # nothing in it needs to start at zero
    err = kv.new_error_word(dev)
    kv.decode_shared(x.q.to(dev), lay, torch.from_numpy(x.cache).to(dev), torch.from_numpy(x.prefix_table).to(dev),
                     x.prefix, torch.from_numpy(x.bt).to(dev), torch.from_numpy(x.lens).to(dev), Lmax, out, ws, err,
                     x.sm, x.tail_k.to(dev), x.tail_v.to(dev), lse, stream=stream)
    torch.cuda.synchronize()
    return out, lse, kv.read_error_flags(err)


def run_mass(x: Batch, mass, decay, dev="cuda"):
    lay = x.layout_of()
    B, Lmax = len(x.lens), int(x.lens.max())
    out = torch.full((B, x.Hq, x.D), float("nan"), dtype=torch.float32, device=dev)
    lse = torch.full((B, x.Hq), float("nan"), dtype=torch.float32, device=dev)
    ws = torch.full((kv.decode_mass_workspace_bytes(lay, B, x.Hq, Lmax),), 0xff, dtype=torch.uint8, device=dev)
    err = kv.new_error_word(dev)
    mass = mass.to(dev)
    new = torch.full_like(mass, float("nan"))
    kv.decode_mass(x.q[:, 0].contiguous().to(dev), lay, torch.from_numpy(x.cache).to(dev),
                   torch.from_numpy(x.bt).to(dev), torch.from_numpy(x.lens).to(dev), Lmax, out, mass, new, ws, err, x.sm,
                   x.tail_k.to(dev), x.tail_v.to(dev), lse, decay=decay)
    torch.cuda.synchronize()
    return out, lse, new, kv.read_error_flags(err)


def evicted(mass, table, lens, N, keep, sink, recent):
    """The eviction's definition, sequence by sequence (numpy inputs): (mass,
    table, lens, freed, count)."""
    n = N // 16
    T = mass.shape[1]
    new_mass, new_table = np.zeros_like(mass), np.full_like(table, -1)
    freed, count, new_lens = np.full_like(table, -1), np.zeros_like(lens), lens.copy()
    for b, L in enumerate(lens):
        done = int(L) // N
        gone = []
        if done > keep:
            key = [float("-inf") if np.isnan(m) else float(m) for m in mass[b]]
            nan = [bool(np.isnan(m)) for m in mass[b]]
            free = range(sink, done - recent)
            gone = sorted(sorted(free, key=lambda t: (not nan[t], key[t], -t))[:done - keep])
        left = [t for t in range(done) if t not in set(gone)]
        new_mass[b, :len(left)] = mass[b, left]
        pages = table[b, :T * n].reshape(T, n)
        new_table[b, :len(left) * n] = pages[left].ravel()
        freed[b, :len(gone) * n] = pages[gone].ravel()
        count[b] = len(gone) * n
        new_lens[b] = L - len(gone) * N
    return new_mass, new_table, new_lens, freed, count
