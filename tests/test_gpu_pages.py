"""Sequences that fork, end and leave their windows, and the compaction of a cache, against plain loops: tables, counts
and copies are whole, so everything has to be equal."""
import numpy as np
import pytest
import torch

import quantized_kv_cache_kvarn_gb300 as kv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_kv_cache_kvarn_gb300 import build
    build.build()
    kv.lib()


def layout(N, pages):
    return kv.q8_layout(128, 2, pages) if N == 16 else kv.dense_layout(128, N, 2, pages)


def gpu(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def rows_of(rng, B, N, T, pages, lens, share):
    """Tables whose rows share some pages, with places without one, and the counts that go with them."""
    n = N // 16
    table = rng.integers(0, pages, (B, T * n)).astype(np.int32)
    if B > 1:
        table[1::2, :share] = table[0:B - B % 2:2, :share]
    table[rng.random(table.shape) < 0.1] = -1
    refs = np.zeros(pages, np.int32)
    for b in range(B):
        for p in table[b, :max(0, lens[b]) // N * n]:
            if p >= 0:
                refs[p] += 1
    return table, refs


def fork(parents, lens, table, refs, N, T, window, sinks, recent):
    n = N // 16
    out_lens, out, counts = np.zeros(len(parents), np.int32), np.full((len(parents), T * n), -1, np.int32), refs.copy()

    def held(a):
        return max(0, lens[a] - recent) // N * n

    for a in range(len(lens)):
        for e in range(held(a)):
            if table[a, e] >= 0:
                counts[table[a, e]] -= 1
    for b, a in enumerate(parents):
        if a < 0:
            continue
        out_lens[b] = lens[a]
        for e in range(held(a)):
            t = e // n * N
            if window == 0 or t < sinks or t + N > lens[a] + 1 - window:
                out[b, e] = table[a, e]
                if table[a, e] >= 0:
                    counts[table[a, e]] += 1
    freed = np.flatnonzero((refs > 0) & (counts <= 0)).astype(np.int32)
    return out_lens, out, counts, freed


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,out,N,T,pages,window,sinks,recent,seed", [
    (1, 1, 16, 1, 1, 0, 0, 0, 0), (5, 7, 16, 9, 40, 0, 0, 0, 1), (8, 8, 128, 5, 500, 0, 0, 0, 2), (33, 20, 64, 40, 9000, 0, 0, 0, 3),
    (12, 12, 16, 70, 1000, 100, 4, 0, 4), (12, 17, 64, 20, 2000, 300, 130, 0, 5), (6, 6, 128, 12, 700, 1, 0, 256, 6),
    (40, 40, 16, 600, 70000, 2000, 20, 0, 7), (3, 0, 16, 4, 30, 0, 0, 0, 8), (300, 500, 16, 3, 333, 0, 0, 5, 9)])
def test_fork(B, out, N, T, pages, window, sinks, recent, seed, in_place):
    rng = np.random.default_rng(seed)
    most = T * N + N - 1
    lens = rng.integers(0, most + 1, B).astype(np.int32)
    lens[-1] = most
    table, refs = rows_of(rng, B, N, T, pages, lens, T * (N // 16) // 2)
    extra = 3
    refs[rng.random(pages) < 0.1] += 2  # held by others as well
    parents = rng.integers(-1, B, out).astype(np.int32)
    cap, D = N + recent, 24
    tails = [rng.standard_normal((B, 2, cap, D)).astype(np.float16), rng.standard_normal((B, 1, cap, 8)).astype(np.float32)]
    sink = rng.standard_normal((B, 2, 5, 8)).astype(np.float16)
    if seed == 7:
        tails, sink = [], None
    wide = np.full((B, table.shape[1] + extra), 12345, np.int32)
    wide[:, :table.shape[1]] = table
    lay = layout(N, pages)
    want = fork(parents, lens, table, refs, N, T, window, sinks, recent)
    t = dict(lens=gpu(lens), table=gpu(wide), refs=gpu(refs), parents=gpu(parents), err=kv.new_error_word())
    new_lens, new_table = torch.full((out,), 77, dtype=torch.int32, device="cuda"), torch.full((out, wide.shape[1]), 99, dtype=torch.int32, device="cuda")
    new_refs = t["refs"] if in_place else torch.full_like(t["refs"], 55)
    freed, count = torch.full_like(t["refs"], 44), torch.full((1,), 3, dtype=torch.int32, device="cuda")
    pairs = [(gpu(x), torch.full((out, *x.shape[1:]), 7.0, dtype=torch.from_numpy(x).dtype, device="cuda")) for x in tails]
    sinks_pair = [] if sink is None else [(gpu(sink), torch.full((out, *sink.shape[1:]), 7.0, dtype=torch.float16, device="cuda"))]
    kv.fork_sequences(t["parents"], t["lens"], t["table"], t["refs"], lay, most, new_lens, new_table, new_refs, freed, count,
                      t["err"], tails=pairs, sinks=sinks_pair, recent_tokens=recent, window=window, sink_tokens=sinks)
    assert kv.read_error_flags(t["err"]) == 0
    assert np.array_equal(new_lens.cpu().numpy(), want[0])
    assert np.array_equal(new_table.cpu().numpy()[:, :T * (N // 16)], want[1]) and (new_table[:, T * (N // 16):] == 99).all()
    assert np.array_equal(new_refs.cpu().numpy(), want[2])
    n = int(count)
    assert n == len(want[3]) and np.array_equal(freed.cpu().numpy()[:n], want[3]) and (freed[n:] == -1).all()
    for (old, new), x in zip(pairs, tails):
        for b, a in enumerate(parents):
            live = 0 if a < 0 else min(cap, lens[a] - max(0, lens[a] - recent) // N * N)
            assert np.array_equal(new[b, :, :live].cpu().numpy(), x[a, :, :live]) and (new[b, :, live:] == 7).all(), (b, a)
    for old, new in sinks_pair:
        for b, a in enumerate(parents):
            assert (new[b] == 7).all() if a < 0 else torch.equal(new[b], old[a])


def test_fork_of_bad_inputs_is_flagged():
    lay = layout(16, 10)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731

    def run(parents, lens, table):
        out, err = [torch.empty(len(parents), dtype=torch.int32, device="cuda"), torch.empty((len(parents), 2), dtype=torch.int32, device="cuda")], kv.new_error_word()
        refs, freed, count = torch.ones(10, dtype=torch.int32, device="cuda"), torch.empty(10, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
        kv.fork_sequences(i32(parents), i32(lens), i32(table), refs, lay, 40, out[0], out[1], refs, freed, count, err)
        return kv.read_error_flags(err), out[0].tolist(), out[1].tolist(), freed[:int(count)].tolist()

    assert run([0, 2], [32, 5], [[1, 2], [3, 4]]) == (kv.DEVERR_INDEX, [32, 0], [[1, 2], [-1, -1]], [])
    assert run([0, 1], [41, -3], [[1, 2], [3, 4]]) == (kv.DEVERR_SEQ_LEN, [40, 0], [[1, 2], [-1, -1]], [])
    assert run([0, 0], [32, 5], [[1, 10], [3, 4]]) == (kv.DEVERR_PAGE_RANGE, [32, 32], [[1, -1], [1, -1]], [])
    assert run([-1, -1], [32, 16], [[9, 0], [3, 4]]) == (0, [0, 0], [[-1, -1], [-1, -1]], [0, 3, 9])


def test_counts_that_do_not_agree_with_the_rows():
    """A count below its rows' number passes through 0 on its way: what it comes to decides."""
    lay, err = layout(16, 4), kv.new_error_word()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    refs, freed, count = i32([1, 1, 0, 2]), i32([0] * 4), i32([0])
    lens, table = i32([0] * 8), i32([[0]] * 8)
    # rows 0..6 hold page 0 and all but row 6 end; row 6 goes on eight times; row 7 holds page 3
    kv.fork_sequences(i32([6] * 8), i32([16] * 8), i32([[0]] * 7 + [[3]]), refs, lay, 16, lens, table, refs, freed, count, err)
    assert refs.tolist() == [2, 1, 0, 1] and int(count) == 0 and freed.tolist() == [-1] * 4


def compact(refs, table):
    live = np.flatnonzero(refs > 0)
    n = len(live)
    remap = np.full(len(refs), -1, np.int32)
    holes = [i for i in range(n) if refs[i] <= 0]
    for p in live:
        remap[p] = p if p < n else holes.pop(0)
    new_refs = np.zeros_like(refs)
    new_refs[remap[live]] = refs[live]
    return n, remap, new_refs, np.where(table >= 0, remap[np.maximum(table, 0)], -1)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("pages,live,page_bytes,rows,entries", [
    (1, 1.0, 16, 1, 1), (1, 0.0, 16, 1, 3), (17, 0.5, 48, 3, 5), (2048, 0.5, 4096, 2, 700), (2049, 0.3, 4112, 1, 9), (6000, 0.9, 8256, 40, 33),
    (20000, 0.02, 1920, 5, 1000), (5000, 1.0, 64, 4, 4), (4096, 0.0, 32, 4, 4), (100000, 0.5, 16, 7, 3)])
def test_compact(pages, live, page_bytes, rows, entries, in_place):
    rng = np.random.default_rng(pages)
    refs = np.where(rng.random(pages) < live, rng.integers(1, 5, pages), rng.integers(-1, 1, pages)).astype(np.int32)
    used = np.flatnonzero(refs > 0)
    table = rng.choice(used, (rows, entries)).astype(np.int32) if len(used) else np.full((rows, entries), -5, np.int32)
    table[rng.random(table.shape) < 0.2] = -7
    cache = rng.integers(0, 256, (pages, page_bytes)).astype(np.uint8)
    n, remap, new_refs, new_table = compact(refs, table)
    c, r, tb, err = gpu(cache), gpu(refs), gpu(table), kv.new_error_word()
    r2, t2 = (r, tb) if in_place else (torch.full_like(r, 9), torch.full_like(tb, 9))
    out, count = torch.full_like(r, 9), torch.full((1,), 9, dtype=torch.int32, device="cuda")
    space = torch.full((kv.compact_pages_workspace_bytes(pages),), 255, dtype=torch.uint8, device="cuda")
    kv.compact_pages(c, r, tb, r2, t2, out, count, space, err)
    assert kv.read_error_flags(err) == 0 and int(count) == n
    assert np.array_equal(out.cpu().numpy(), remap) and np.array_equal(r2.cpu().numpy(), new_refs)
    assert np.array_equal(t2.cpu().numpy(), new_table)
    got = c.cpu().numpy()
    assert np.array_equal(got[remap[used]], cache[used]) and np.array_equal(got[n:], cache[n:])


def test_compact_flags_bad_entries_and_takes_no_table():
    cache = torch.arange(6, dtype=torch.uint8, device="cuda").repeat_interleave(32).view(6, 32).contiguous()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    refs, err, count, remap = i32([0, 1, 0, 0, 2, 1]), kv.new_error_word(), i32([0]), i32([0] * 6)
    space = torch.empty(kv.compact_pages_workspace_bytes(6), dtype=torch.uint8, device="cuda")
    table, out = i32([[4, 0, 6, 5, -1]]), i32([[0] * 5])
    kv.compact_pages(cache.clone(), refs, table, i32([0] * 6), out, remap, count, space, err)
    assert kv.read_error_flags(err) == kv.DEVERR_PAGE_RANGE and out.tolist() == [[0, -1, -1, 2, -1]]
    err.zero_()
    kv.compact_pages(cache, refs, None, refs, None, remap, count, space, err)
    assert kv.read_error_flags(err) == 0 and remap.tolist() == [-1, 1, -1, -1, 0, 2] and refs.tolist() == [2, 1, 1, 0, 0, 0]
    assert cache[:, 0].tolist() == [4, 1, 5, 3, 4, 5]


def test_an_empty_cache():
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    count, err = torch.full((1,), 4, dtype=torch.int32, device="cuda"), kv.new_error_word()
    space = torch.empty(kv.compact_pages_workspace_bytes(0), dtype=torch.uint8, device="cuda")
    kv.compact_pages(torch.empty((0, 64), dtype=torch.uint8, device="cuda"), e, None, e, None, e.clone(), count, space, err)
    assert int(count) == 0 and kv.read_error_flags(err) == 0


def test_graphs_of_both():
    """Captured with workspaces of their own, replayed with other inputs."""
    rng = np.random.default_rng(5)
    B, N, T, pages = 20, 16, 50, 3000
    lay, most = layout(N, pages), T * N + 9
    lens = rng.integers(0, most, B).astype(np.int32)
    table, refs = rows_of(rng, B, N, T, pages, lens, 20)
    parents = gpu(np.arange(B, dtype=np.int32))
    t = dict(lens=gpu(lens), table=gpu(table), refs=gpu(refs), err=kv.new_error_word())
    out = dict(lens=torch.empty_like(t["lens"]), table=torch.empty_like(t["table"]), refs=torch.empty_like(t["refs"]),
               freed=torch.empty_like(t["refs"]), count=torch.empty_like(t["err"]), remap=torch.empty_like(t["refs"]),
               live=torch.empty_like(t["err"]), refs2=torch.empty_like(t["refs"]), table2=torch.empty_like(t["table"]))
    cache = gpu(rng.integers(0, 256, (pages, 160)).astype(np.uint8))
    first = cache.clone()
    space = torch.empty(kv.compact_pages_workspace_bytes(pages), dtype=torch.uint8, device="cuda")

    def both():
        kv.fork_sequences(parents, t["lens"], t["table"], t["refs"], lay, most, out["lens"], out["table"], out["refs"],
                          out["freed"], out["count"], t["err"])
        kv.compact_pages(cache, out["refs"], out["table"], out["refs2"], out["table2"], out["remap"], out["live"], space, t["err"])

    both()  # the attributes of the kernels are set before a capture
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        both()
    for seed in range(3):
        p = np.random.default_rng(seed).integers(-1, B, B).astype(np.int32)
        parents.copy_(torch.from_numpy(p))
        cache.copy_(first)
        g.replay()
        torch.cuda.synchronize()
        want = fork(p, lens, table, refs, N, T, 0, 0, 0)
        n, remap, new_refs, new_table = compact(want[2], want[1])
        assert np.array_equal(out["table2"].cpu().numpy(), new_table) and np.array_equal(out["refs2"].cpu().numpy(), new_refs)
        assert int(out["live"]) == n and int(out["count"]) == len(want[3])
        used = np.flatnonzero(want[2] > 0)
        assert np.array_equal(cache.cpu().numpy()[remap[used]], first.cpu().numpy()[used])
    assert kv.read_error_flags(t["err"]) == 0
