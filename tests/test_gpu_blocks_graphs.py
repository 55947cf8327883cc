"""Blocks written and read back, norms, fork and compaction captured into graphs and replayed over new inputs, and two of
them on the GPU at once, each with buffers of its own: the bits of calls made one after another."""
import pytest
import torch

import quantized_kv_cache_kvarn_gb300 as kv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_kv_cache_kvarn_gb300 import build
    build.build()
    kv.lib()


class Work:
    """A chunk normed, written, read back; its rows forked, half of them ended; the cache compacted."""

    def __init__(self, code, pages=60, B=4, H=2, C=128, D=128):
        self.code, self.lay = code, kv.q8_layout(D, H, pages)
        i32 = dict(dtype=torch.int32, device="cuda")
        self.shape, self.B, self.T = (B, C, H, D), B, C // 16
        self.k, self.v = (torch.zeros(self.shape, dtype=torch.float16, device="cuda") for _ in range(2))
        self.k2, self.v2 = torch.zeros_like(self.k), torch.zeros_like(self.v)
        self.cache, self.err = kv.alloc_q8_cache(self.lay), kv.new_error_word()
        self.pos, self.inv = torch.arange(C, **i32)[None], kv.rope_frequencies(D)[0]
        self.start, self.table = torch.zeros(B, **i32), torch.full((B, self.T), -1, **i32)
        self.lens, self.parents, self.new_lens = torch.full((B,), C, **i32), torch.zeros(B, **i32), torch.zeros(B, **i32)
        self.new_table = torch.zeros_like(self.table)
        self.refs, self.freed, self.count = torch.zeros(pages, **i32), torch.zeros(pages, **i32), torch.zeros(1, **i32)
        self.remap, self.live = torch.zeros(pages, **i32), torch.zeros(1, **i32)
        self.space = torch.zeros(kv.compact_pages_workspace_bytes(pages), dtype=torch.uint8, device="cuda")

    def inputs(self, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.k.copy_(torch.randn(self.shape, generator=g, device="cuda"))
        self.v.copy_(torch.randn(self.shape, generator=g, device="cuda"))
        pages = self.refs.numel()
        self.table.copy_(torch.randperm(pages, generator=g, device="cuda")[:self.table.numel()].view(self.table.shape))
        self.refs.zero_()
        self.refs[self.table.flatten().long()] = 1
        self.parents.copy_(torch.tensor([(seed + i) % self.B // 2 * 2 for i in range(self.B)]))
        self.cache.fill_(seed % 100)

    def run(self):
        kv.norm_rope(self.k, self.k2, None, self.pos, self.inv)
        kv.q8_encode_blocks(self.k2.transpose(1, 2), self.v.transpose(1, 2), self.lay, self.code, self.start, self.table, self.cache, self.err)
        kv.fork_sequences(self.parents, self.lens, self.table, self.refs, self.lay, 16 * self.T, self.new_lens, self.new_table, self.refs,
                          self.freed, self.count, self.err)
        kv.compact_pages(self.cache, self.refs, self.new_table, self.refs, self.new_table, self.remap, self.live, self.space, self.err)
        kv.q8_read_blocks(self.k2.transpose(1, 2), self.v2.transpose(1, 2), self.lay, self.code, self.start, self.new_table, self.cache, self.err)

    def results(self):
        return [t.clone() for t in (self.k2, self.v2, self.cache, self.new_lens, self.new_table, self.refs, self.freed, self.count, self.remap,
                                    self.live, self.err)]


def test_replayed_and_at_once():
    seeds = (1, 2, 3)
    eager = {}
    for code in (0, 1):
        w = Work(code)
        for s in seeds:
            w.inputs(s)
            w.run()
            eager[code, s] = w.results()
            assert kv.read_error_flags(w.err) == 0 and 0 < int(w.live) < w.B * w.T and int(w.count) > 0
    works, graphs = [Work(0), Work(1)], []
    for w in works:
        w.inputs(1)
        w.run()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            w.run()
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in works]
    for s in seeds:
        for w in works:
            w.inputs(s)
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for code, w in enumerate(works):
            assert all(torch.equal(a, b) for a, b in zip(w.results(), eager[code, s])), (code, s)
    # eagerly, on streams of their own
    for s in seeds:
        for w in works:
            w.inputs(s)
        torch.cuda.synchronize()
        for w, st in zip(works, streams):
            with torch.cuda.stream(st):
                w.run()
        torch.cuda.synchronize()
        for code, w in enumerate(works):
            assert all(torch.equal(a, b) for a, b in zip(w.results(), eager[code, s])), (code, s)
