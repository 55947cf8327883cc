"""Append, decode, fork and compaction issued in a row without a pause, each starting while the one before it ends
(programmatic launches), over a cache in which blocks complete, pages are given back and pages move: the same bits as
with the GPU waited for after every call."""
import pytest
import torch

import quantized_kv_cache_kvarn_gb300 as kv
from tests import blocks8 as b8

pytestmark = pytest.mark.gpu

STEPS, W, S = 40, 64, 4
LENS = [47, 200, 31, 90]


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_kv_cache_kvarn_gb300 import build
    build.build()
    kv.lib()


def run(D, code, wait):
    """Outputs of every step, and what was done in all: blocks completed, pages freed, pages moved."""
    x = b8.Batch(LENS, 4, 2, D, window=W, sinks=S, code=code, seed=4).gpu(kv)
    most, B = max(LENS) + STEPS, len(LENS)
    T, pages = most // 16, x.cache.shape[0] + 24
    i32 = dict(dtype=torch.int32, device="cuda")
    lay = kv.q8_layout(D, 2, pages)
    cache = torch.cat([x.t["cache"], torch.zeros((24, *x.t["cache"].shape[1:]), dtype=torch.uint8, device="cuda")])
    table = torch.full((B, T), -1, **i32)
    table[:, :x.table.shape[1]] = x.t["table"]
    table[table >= pages] = -1  # blocks behind the windows: their pages are free
    lens, tails = x.t["lens"].clone(), [x.t[n].nan_to_num(0) for n in ("tail_k", "tail_v")]
    refs = torch.bincount(table[table >= 0], minlength=pages).int()
    # rows change places, then one ends and another forks
    turns = [torch.tensor(p, **i32) for p in ([1, 0, 2, 3], [0, 1, 3, 2], [2, 1, 0, 3], [0, 1, 2, 2])]
    live, count, err = torch.zeros(1, **i32), torch.zeros(1, **i32), kv.new_error_word()
    remap, freed, places = torch.zeros(pages, **i32), torch.zeros(pages, **i32), torch.arange(pages, **i32)
    space = torch.empty(kv.q8_decode_workspace_bytes(lay, B, 4, 1, most, W, S), dtype=torch.uint8, device="cuda")
    cspace = torch.empty(kv.compact_pages_workspace_bytes(pages), dtype=torch.uint8, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    outs, totals = [], torch.zeros(3, dtype=torch.int64, device="cuda")

    def made(calls):
        for call in calls:
            call()
            if wait:
                torch.cuda.synchronize()

    # to begin with, a cache without holes
    kv.compact_pages(cache, refs, table, refs, table, remap, live, cspace, err)
    for i in range(STEPS):
        # the next token of every row; pages behind those in use for the blocks that it completes
        lens += 1
        full = lens % 16 == 0
        page = (live + torch.cumsum(full, 0) - 1).int()
        at = (lens // 16 - 1).clamp(min=0).long()[:, None]
        table.scatter_(1, at, torch.where(full[:, None], page[:, None], table.gather(1, at)))
        refs.scatter_add_(0, torch.where(full, page, 0).long(), full.int())
        k, v, k2 = (torch.randn((B, 2, D), generator=g, device="cuda").half() for _ in range(3))
        q = torch.randn((B, 1, 4, D), generator=g, device="cuda").half()
        new_tails, new_table, new_lens = [torch.zeros_like(t) for t in tails], torch.full_like(table, -1), torch.empty_like(lens)
        o = [torch.empty((B, 1, 4, D), device="cuda") for _ in range(2)] + [torch.empty((B, 1, 4), device="cuda") for _ in range(2)]
        # k2: all rows the same token, so that rows that share a page of a block just completed write the same bytes
        k2[:] = k2[:1]
        parents = turns[i % len(turns)]
        made([
            lambda: kv.q8_append(k, v, lay, code, lens, most, *tails, table, cache, err),
            lambda: kv.q8_decode(q, lay, code, cache, table, lens, most, o[0], space, err, 0.1, *tails, o[2], window=W, sink_tokens=S),
            lambda: kv.fork_sequences(parents, lens, table, refs, lay, most, new_lens, new_table, refs, freed, count, err,
                                      tails=tuple(zip(tails, new_tails)), window=W, sink_tokens=S),
            lambda: kv.compact_pages(cache, refs, new_table, refs, new_table, remap, live, cspace, err),
            # the newest token again, another one: into tails and pages where fork and compaction have just put them (its
            # window is one token shorter: the fork keeps what the next token sees)
            lambda: kv.q8_append(k2, k2, lay, code, new_lens, most, *new_tails, new_table, cache, err),
            lambda: kv.q8_decode(q, lay, code, cache, new_table, new_lens, most, o[1], space, err, 0.1, *new_tails, o[3], window=W - 1,
                                 sink_tokens=S)])
        totals += torch.stack([full.sum(), count[0].long(), ((remap >= 0) & (remap != places)).sum()])
        tails, table, lens = new_tails, new_table, new_lens
        outs += [*o, count.clone(), live.clone(), freed.clone(), remap.clone()]
    torch.cuda.synchronize()
    assert kv.read_error_flags(err) == 0
    return outs + [*tails, table, lens, refs], totals.tolist()


@pytest.mark.parametrize("D,code", [(128, b8.E4M3), (256, b8.INT8)])
def test_a_chain_that_completes_blocks_frees_and_moves_pages(D, code):
    first, totals = run(D, code, True)
    assert all(n >= 5 for n in totals), totals
    for _ in range(3):
        again, _ = run(D, code, False)
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    assert all(t.isfinite().all() for t in first[:4])
