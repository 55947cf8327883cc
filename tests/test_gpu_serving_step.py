"""The serving calls together, as a decode loop uses them: queries and keys
turned to their positions, the key appended (and the tile it completes
encoded), attention over the shared prefix, attention with tile masses, and
from time to time the eviction of the lightest tiles. Every step is checked
against the oracle's decode of the pages and tails the GPU holds; the same
step replayed from a CUDA graph gives the same bits."""
import numpy as np
import pytest
import torch

import quantized_kv_cache_kvarn_gb300 as kv
from oracle import attention, layout
from tests import parity, serving

pytestmark = pytest.mark.gpu

B, Hq, Hkv, D, N = 3, 8, 2, 128, 64
PREFIX, KEEP, LONGEST = 2 * N, 5, 9 * N
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_kv_cache_kvarn_gb300 import build
    build.build()
    kv.lib()


class Loop:
    """State of the decode loop: buffers a serving program keeps."""

    def __init__(self, seed):
        g = torch.Generator().manual_seed(seed)
        ppt, T = N // 16, LONGEST // N
        pages = (PREFIX // N + B * T) * ppt
        self.lay = kv.dense_layout(D, N, Hkv, pages)
        self.cache, self.err = kv.alloc_cache(self.lay, DEV), kv.new_error_word(DEV)
        perm = torch.randperm(pages, generator=g).to(torch.int32)
        self.prefix_table = perm[:PREFIX // 16].to(DEV)
        bt = perm[PREFIX // 16:].view(B, T * ppt)[:, :(LONGEST - PREFIX) // 16]
        self.table = torch.cat([self.prefix_table[None].repeat(B, 1), bt.to(DEV)], 1).contiguous()
        self.inv_freq, self.scale = kv.rope_frequencies(D, 10000.0, yarn=(4.0, 256), device=DEV)
        # the prefix: keys at positions 0.., encoded once
        pk, pv = (torch.randn((1, PREFIX, Hkv, D), generator=g).half().to(DEV) for _ in range(2))
        kv.rope(pk, pk, torch.arange(PREFIX, dtype=torch.int32, device=DEV)[None], self.inv_freq, scale=self.scale)
        kv.encode_tiles(pk.transpose(1, 2).contiguous(), pv.transpose(1, 2).contiguous(), self.lay,
                        torch.zeros(1, dtype=torch.int32, device=DEV), self.prefix_table[None], self.cache, self.err)
        self.lens = torch.full((B,), PREFIX, dtype=torch.int32, device=DEV)  # tokens held
        self.pos = torch.full((B, 1), PREFIX, dtype=torch.int32, device=DEV)  # position of the next one
        self.tail_k, self.tail_v = (torch.zeros((B, Hkv, N, D), dtype=torch.float16, device=DEV) for _ in range(2))
        self.mass = torch.zeros((B, T), device=DEV)
        # a step's inputs and outputs
        self.q, self.k, self.v = (torch.empty((B, 1, h, D), dtype=torch.float16, device=DEV) for h in (Hq, Hkv, Hkv))
        self.qr, self.kr = torch.empty_like(self.q), torch.empty_like(self.k)
        self.out, self.out_shared = torch.empty((B, Hq, D), device=DEV), torch.empty((B, 1, Hq, D), device=DEV)
        self.ws = torch.empty(kv.decode_mass_workspace_bytes(self.lay, B, Hq, LONGEST), dtype=torch.uint8, device=DEV)
        self.ws_shared = torch.empty(kv.decode_shared_workspace_bytes(self.lay, B, Hq, 1, LONGEST, PREFIX),
                                     dtype=torch.uint8, device=DEV)
        self.freed, self.count = torch.empty_like(self.table), torch.empty_like(self.lens)
        self.sm = 1.0 / np.sqrt(D)

    def step(self):
        kv.rope([self.q, self.k], [self.qr, self.kr], self.pos, self.inv_freq, scale=self.scale)
        self.pos += 1
        self.lens += 1
        kv.append(self.kr[:, 0], self.v[:, 0], self.lens, LONGEST, self.tail_k, self.tail_v, self.table, self.lay,
                  self.cache, self.err)
        kv.decode_shared(self.qr, self.lay, self.cache, self.prefix_table, PREFIX, self.table, self.lens, LONGEST,
                         self.out_shared, self.ws_shared, self.err, self.sm, self.tail_k, self.tail_v)
        kv.decode_mass(self.qr[:, 0], self.lay, self.cache, self.table, self.lens, LONGEST, self.out, self.mass, self.mass,
                       self.ws, self.err, self.sm, self.tail_k, self.tail_v, decay=0.9)

    def evict(self):
        kv.evict_tiles(self.mass, self.table, self.lens, self.lay, LONGEST, KEEP, self.mass, self.table, self.lens, self.freed,
                       self.count, self.err, sink_tiles=PREFIX // N, recent_tiles=1)

    def inputs(self, g):
        for t in (self.q, self.k, self.v):
            t.copy_(torch.randn(t.shape, generator=g))


def expected(x):
    """Oracle output and tile masses of a step's queries over what the GPU holds."""
    lay = layout.DenseLayout(D, N)
    cache, table, lens = x.cache.cpu().numpy(), x.table.cpu().numpy(), x.lens.cpu().numpy()
    q, tk, tv = parity.f64(x.qr[:, 0]), parity.f64(x.tail_k), parity.f64(x.tail_v)
    out, _ = attention.decode(q, cache, lay, table, lens, x.sm, tk, tv)
    mass = np.zeros((B, LONGEST // N))
    for b, L in enumerate(lens):
        for h in range(Hq):
            k, _ = attention.sequence_kv(cache, lay, table[b], int(L), h * Hkv // Hq, tk[b, h * Hkv // Hq], tv[b, h * Hkv // Hq])
            s = x.sm * (k @ q[b, h])
            p = np.exp(s - s.max())
            p /= p.sum()
            for t in range(int(L) // N):
                mass[b, t] += p[t * N:(t + 1) * N].sum()
    return out, mass


def test_loop_of_rope_append_shared_mass_and_eviction():
    x, g = Loop(3), torch.Generator().manual_seed(4)
    tiles_freed = 0
    for i in range(5 * N + 7):
        x.inputs(g)
        before = x.mass.double().cpu().numpy()
        x.step()
        if i % 37 == 0 or i % N in (N - 1, 0):  # and around every tile's end
            out, mass = expected(x)
            # parity's bound of the decode, 2e-3, holds 100 times over here:
            # scores of a few units are off by at most 2^-17 of 128 sums of
            # magnitude below 64, values below 8
            assert np.abs(parity.f64(x.out) - out).max() < 2e-3
            assert np.abs(parity.f64(x.out_shared[:, 0]) - out).max() < 2e-3
            done = x.lens.cpu().numpy()[:, None] // N > np.arange(LONGEST // N)
            want = np.where(done, 0.9 * before + mass, 0.0)
            assert np.abs(parity.f64(x.mass) - want).max() <= 2e-3 * max(1.0, want.max())
        if i % 50 == 49:
            m, t, l = x.mass.cpu().numpy(), x.table.cpu().numpy(), x.lens.cpu().numpy()
            x.evict()
            want = serving.evicted(m, t, l, N, KEEP, PREFIX // N, 1)
            for a, b in zip((x.mass, x.table, x.lens, x.freed, x.count), want):
                np.testing.assert_array_equal(a.cpu().numpy(), b)
            # a freed page may be used again: give it back behind the row's kept pages
            for b in range(B):
                n, c = int(x.lens[b]) // N * (N // 16), int(x.count[b])
                x.table[b, n:n + c] = x.freed[b, :c]
                x.table[b, n + c:] = torch.from_numpy(t[b, n + c:]).to(DEV)
                tiles_freed += c // (N // 16)
    assert tiles_freed > 0
    assert kv.read_error_flags(x.err) == 0


def test_the_step_replays_from_a_graph():
    eager, g = Loop(5), torch.Generator().manual_seed(6)
    graphed = Loop(5)
    rows = [[torch.randn(t.shape, generator=g) for t in (eager.q, eager.k, eager.v)] for _ in range(N + 5)]
    keep = [t.clone() for t in (graphed.lens, graphed.pos, graphed.mass)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graphed.inputs(torch.Generator().manual_seed(1))
        graphed.step()  # the library's one-time launch set-up
    torch.cuda.current_stream().wait_stream(s)
    for t, old in zip((graphed.lens, graphed.pos, graphed.mass), keep):
        t.copy_(old)
    graphed.tail_k.zero_()
    graphed.tail_v.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        graphed.step()
    for row in rows:
        for x in (eager, graphed):
            for t, r in zip((x.q, x.k, x.v), row):
                t.copy_(r)
        eager.step()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in ((eager.out, graphed.out), (eager.out_shared, graphed.out_shared), (eager.mass, graphed.mass)):
            assert torch.equal(a, b)
    assert torch.equal(eager.cache, graphed.cache)
    assert kv.read_error_flags(eager.err) == 0 and kv.read_error_flags(graphed.err) == 0
