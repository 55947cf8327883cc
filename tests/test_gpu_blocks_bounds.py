"""The ends of what the 8-bit block cache's, the norms' and the pages' calls take: offsets past 32 bits, empty batches,
many sequences, waits that run out in the wide kernel, calls of several host threads at once, tensors elsewhere."""
import threading

import numpy as np
import pytest
import torch

import quantized_kv_cache_kvarn_gb300 as kv
from tests import blocks8 as b8
from tests.test_gpu_q8 import check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_kv_cache_kvarn_gb300 import build
    build.build()
    kv.lib()


def test_pages_past_32_bits():
    """A cache of more than 2^32 bytes whose pages in use lie at both of its ends: appended to, read and decoded."""
    x = b8.Batch([64, 100, 17], 4, 1, 128, seed=5)
    n, many = x.cache.shape[0], (1 << 32) // 4128 + 300
    far = np.where(np.arange(n) % 2 == 0, np.arange(n), many - 1 - np.arange(n)).astype(np.int64)
    x.gpu(kv)
    big = torch.zeros((many, 1, 4128), dtype=torch.uint8, device="cuda")
    big[torch.from_numpy(far).cuda()] = x.t["cache"]
    table = np.where(x.table < n, far[np.minimum(x.table, n - 1)], -1).astype(np.int32)
    x.layout = kv.q8_layout(128, 1, many)
    x.t["cache"], x.t["table"] = big, torch.from_numpy(table).cuda()
    check(x)
    k, v = (torch.empty((1, 1, 64, 128), dtype=torch.float16, device="cuda") for _ in range(2))
    kv.q8_read_blocks(k, v, x.layout, 0, torch.zeros(1, dtype=torch.int32, device="cuda"), x.t["table"][:1, :4].contiguous(),
                      big, x.t["err"])
    assert np.array_equal(k[0].cpu().numpy(), x.k[0].astype(np.float32).astype(np.float16))
    kv.q8_encode_blocks(k, v, x.layout, 0, torch.zeros(1, dtype=torch.int32, device="cuda"),
                        torch.arange(many - 4, many, dtype=torch.int32, device="cuda")[None], big, x.t["err"])
    k2, v2 = torch.empty_like(k), torch.empty_like(v)
    kv.q8_read_blocks(k2, v2, x.layout, 0, torch.zeros(1, dtype=torch.int32, device="cuda"),
                      torch.arange(many - 4, many, dtype=torch.int32, device="cuda")[None], big, x.t["err"])
    # values of codes are coded as themselves, but for the roundings of scales (fp16 outputs: one step)
    assert (k2.float() - k.float()).abs().max() <= 2.0 ** -10 * k.float().abs().max() * 2
    assert kv.read_error_flags(x.t["err"]) == 0


def test_moves_past_32_bits():
    pages, size = 700, 8 << 20  # 5.9 GB
    cache = torch.zeros((pages, size), dtype=torch.uint8, device="cuda")
    cache[690, ::4096], cache[699, ::4096], cache[600, -1], cache[2, 5] = 11, 12, 13, 14
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    refs[[2, 600, 690, 699]] = torch.tensor([1, 2, 3, 4], dtype=torch.int32, device="cuda")
    out, remap = torch.empty_like(refs), torch.empty_like(refs)
    live, err = torch.zeros(1, dtype=torch.int32, device="cuda"), kv.new_error_word()
    space = torch.empty(kv.compact_pages_workspace_bytes(pages), dtype=torch.uint8, device="cuda")
    kv.compact_pages(cache, refs, None, out, None, remap, live, space, err)
    assert int(live) == 4 and out[:5].tolist() == [2, 3, 1, 4, 0] and kv.read_error_flags(err) == 0
    assert cache[0, -1] == 13 and (cache[1, ::4096] == 11).all() and cache[2, 5] == 14 and (cache[3, ::4096] == 12).all()
    assert int(cache[1].count_nonzero()) == size // 4096 and int(cache[0].count_nonzero()) == 1


def test_norms_past_32_bits():
    """More than 2^31 elements: the last tokens against the definition."""
    S, H, D = 131100, 128, 128
    x = torch.empty((1, S, H, D), dtype=torch.float16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(0)
    for i in range(0, S, 16384):
        x[:, i:i + 16384] = torch.randn(x[:, i:i + 16384].shape, generator=g, device="cuda").half()
    y, pos = torch.empty_like(x), torch.arange(S, dtype=torch.int32, device="cuda")[None]
    inv, _ = kv.rope_frequencies(D)
    kv.norm_rope(x, y, None, pos, inv)
    z, p = x[:, -7:].double(), pos[:, -7:].double()[..., None, None] * inv
    z = z * (z.square().mean(-1, keepdim=True) + 1e-6).rsqrt()
    a, b = z[..., :64], z[..., 64:]
    want = torch.cat([a * p.cos() - b * p.sin(), a * p.sin() + b * p.cos()], -1)
    assert ((y[:, -7:].double() - want).abs() <= 2.0 ** -11 * want.abs() + 2.0 ** -18 * 8).all()


@pytest.mark.parametrize("D,Q", [(128, 1), (256, 3)])
def test_batches_of_nothing(D, Q):
    x = b8.Batch([0, 0, 0], 4, 1, D, Q=Q, seed=1).gpu(kv)
    out, lse = x.decode(kv)
    assert (out == 0).all() and torch.isneginf(lse).all() and kv.read_error_flags(x.t["err"]) == 0
    x.lens = [0, 1, 0]
    x.t["lens"].copy_(torch.tensor(x.lens))
    x.t["q"] = x.t["q"][:0]
    kv.q8_decode(x.t["q"], x.layout, 0, x.t["cache"], x.t["table"][:0], x.t["lens"][:0], 16, x.t["out"][:0], x.t["space"], x.t["err"],
                 1.0, x.t["tail_k"][:0], x.t["tail_v"][:0], x.t["lse"][:0])


def test_thousands_of_sequences():
    """More sequences than a CTA has threads, some empty, behind a window."""
    rng = np.random.default_rng(0)
    lens = rng.integers(0, 90, 1500).tolist()
    check(b8.Batch(lens, 2, 1, 128, Q=2, window=30, sinks=3, seed=2).gpu(kv))


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("cycles,withhold", [(1, False), (300, False), (3000, False), (30000, False), (200000, True)])
def test_waits_that_run_out_anywhere(D, cycles, withhold):
    """Short limits run out in any warp and at any item: the call flags it or is complete, and the next call is right."""
    x = b8.Batch([1500, 40, 700], 12, 2, D, Q=2, seed=3).gpu(kv)
    first = x.decode(kv)[0].clone()
    assert kv.read_error_flags(x.t["err"]) == 0
    kv.set_copy_wait_test(cycles, withhold)
    try:
        for _ in range(5):
            out = x.decode(kv)[0]
            flags = kv.read_error_flags(x.t["err"])
            assert flags == kv.DEVERR_TIMEOUT or (flags == 0 and torch.equal(out, first) and not withhold)
            x.t["err"].zero_()
    finally:
        kv.set_copy_wait_test(0)
    assert torch.equal(x.decode(kv)[0], first) and kv.read_error_flags(x.t["err"]) == 0


def test_several_host_threads():
    """Decodes of different layouts from threads of their own, each on its stream with its workspace."""
    batches = [b8.Batch([500, 33], 8, 2, 128, seed=1), b8.Batch([300, 200], 6, 1, 256, Q=3, code=1, bf16=True, seed=2),
               b8.Batch([700], 16, 2, 128, Q=2, window=100, sinks=4, seed=3)]
    failures, results = [], [None] * len(batches)
    for x in batches:
        x.gpu(kv)
    torch.cuda.synchronize()

    def work(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(50):
                    batches[i].decode(kv, stream=s)
            s.synchronize()
            results[i] = [t.clone() for t in (batches[i].t["out"], batches[i].t["lse"])]
        except Exception as e:  # a thread's failure is the test's
            failures.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(batches))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failures, failures
    for x, r in zip(batches, results):
        check(x, *r)


def test_tensors_elsewhere_are_refused():
    x = b8.Batch([40], 2, 1, 128, seed=1).gpu(kv)
    for name in ("q", "cache", "table", "lens", "out", "space", "tail_k", "lse"):
        with pytest.raises(kv.KvarnError):
            x.decode(kv, **{name: x.t[name].cpu()})
    t = torch.zeros((1, 1, 1, 128))
    with pytest.raises(kv.KvarnError):
        kv.norm_rope(t, t, None, None, None)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(kv.KvarnError):
        kv.fork_sequences(i, i, i[None], i, kv.q8_layout(128, 1, 1), 16, i, i[None], i, i, i, i)
    with pytest.raises(kv.KvarnError):
        kv.compact_pages(torch.zeros((1, 16), dtype=torch.uint8), i, None, i, None, i, i, i, i)


def test_a_chain_of_calls_without_a_pause():
    """Each call starts while the one before ends (programmatic launches): append, decode, fork and compaction issued
    many times in a row give what they give with the GPU waited for in between."""
    def run(wait):
        x = b8.Batch([47, 200, 31], 4, 2, 128, window=64, sinks=4, seed=4, pad_columns=4).gpu(kv)
        t = x.t
        pages = x.cache.shape[0]
        refs, freed = torch.ones(pages, dtype=torch.int32, device="cuda"), torch.empty(pages, dtype=torch.int32, device="cuda")
        count, remap, live = torch.empty(1, dtype=torch.int32, device="cuda"), torch.empty_like(freed), torch.empty(1, dtype=torch.int32, device="cuda")
        space = torch.empty(kv.compact_pages_workspace_bytes(pages), dtype=torch.uint8, device="cuda")
        table, lens = t["table"].clone(), t["lens"].clone()
        table[table >= pages] = -1
        tk, tv = t["tail_k"].nan_to_num(0), t["tail_v"].nan_to_num(0)
        parents = torch.tensor([1, 0, 2], dtype=torch.int32, device="cuda")
        outs = []
        g = torch.Generator(device="cuda").manual_seed(1)
        for i in range(12):
            k = torch.randn((3, 2, 128), generator=g, device="cuda").half()
            tk2, tv2, table2, lens2 = torch.zeros_like(tk), torch.zeros_like(tv), torch.full_like(table, -1), torch.empty_like(lens)
            out, lse = torch.empty_like(t["out"]), torch.empty_like(t["lse"])
            calls = [
                lambda: kv.q8_append(k, k, x.layout, 0, lens, 200, tk, tv, table, t["cache"], t["err"]),
                lambda: kv.q8_decode(t["q"], x.layout, 0, t["cache"], table, lens, 200, out, t["space"], t["err"], 0.1, tk, tv, lse,
                                     window=64, sink_tokens=4),
                lambda: kv.fork_sequences(parents, lens, table, refs, x.layout, 200, lens2, table2, refs, freed, count, t["err"],
                                          tails=((tk, tk2), (tv, tv2)), window=64, sink_tokens=4),
                lambda: kv.compact_pages(t["cache"], refs, table2, refs, table2, remap, live, space, t["err"])]
            for call in calls:
                call()
                if wait:
                    torch.cuda.synchronize()
            tk, tv, table, lens = tk2, tv2, table2, lens2
            outs += [out, lse, count.clone(), live.clone()]
        torch.cuda.synchronize()
        assert kv.read_error_flags(t["err"]) == 0
        return outs + [tk, tv, table, lens, refs]

    assert all(torch.equal(a, b) for a, b in zip(run(True), run(False)))
