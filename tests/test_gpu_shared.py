"""kvarn_decode_shared against the oracle's decode of every sequence over the
same tokens: layouts, widths, group sizes, several queries, padding rows,
ragged own tokens, capture, and the errors it flags."""
import numpy as np
import pytest
import torch

import quantized_kv_cache_kvarn_gb300 as kv
from tests import parity, serving

pytestmark = pytest.mark.gpu

h, b16 = torch.float16, torch.bfloat16
CASES = {
    # D, N, Hq, Hkv, prefix, own tokens of each sequence (None: padding row), Q, dtype, widths
    "pair": (128, 128, 4, 1, 128, [1, 130], 1, h, (4, 2, 4)),
    "one_row": (128, 128, 1, 1, 256, [7], 1, h, (4, 2, 4)),
    "nothing_own": (128, 128, 8, 2, 384, [0, 0, 5], 1, h, (4, 2, 4)),
    "padding_rows": (128, 128, 16, 2, 256, [None, 300, None, 12, 0], 1, h, (4, 2, 4)),
    "g8_many": (128, 128, 16, 2, 640, list(range(0, 19 * 9, 9)), 1, h, (4, 2, 4)),
    "odd_group_tile64": (128, 64, 6, 2, 320, [1, 64, 63, 200, 129], 1, h, (4, 2, 4)),
    "verify3_tile64": (128, 64, 12, 4, 192, [2, 66, 67, 130, 3, 4, 5], 3, b16, (4, 2, 4)),
    "verify8": (128, 128, 8, 2, 256, [7, 135, 8, None, 300], 8, h, (4, 2, 4)),
    "wide": (256, 128, 12, 4, 256, [33, 260, 1], 1, b16, (4, 2, 4)),
    "wide_verify_tile64": (256, 64, 7, 7, 128, [5, 64], 2, h, (4, 2, 4)),
    "k6v6": (128, 128, 32, 8, 256, [100, 3], 1, h, (6, 6, 2)),
    "k2v8": (128, 64, 8, 1, 192, [64, 3, 2, 1], 1, h, (2, 8, 4)),
    "k3v5": (128, 128, 4, 2, 384, [64, 3, 2, 1] * 5, 1, b16, (3, 5, 2)),
    "k8v3": (128, 128, 8, 1, 128, [10] * 17, 1, h, (8, 3, 2)),
    "k5v4_wide": (256, 128, 4, 2, 128, [10, 140], 1, h, (5, 4, 2)),
    "many_rows": (128, 128, 8, 1, 512, [(7 * i) % 40 for i in range(37)], 1, h, (4, 2, 4)),
    "many_rows_verify": (128, 64, 8, 1, 448, [4 + (7 * i) % 90 for i in range(20)], 4, h, (4, 2, 4)),
}


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_kv_cache_kvarn_gb300 import build
    build.build()
    kv.lib()


def batch(name, seed=0):
    D, N, Hq, Hkv, prefix, own, Q, dtype, widths = CASES[name]
    lens = [0 if n is None else prefix + n for n in own]
    return serving.Batch(D, N, Hq, Hkv, lens, Q=Q, prefix=prefix, dtype=dtype, widths=widths, seed=seed)


@pytest.mark.parametrize("name", list(CASES))
def test_matches_oracle(name):
    x = batch(name)
    ref, rlse = x.oracle()
    out, lse, flags = serving.run_shared(x)
    assert flags == 0
    score, tol = x.bounds()
    out, lse = parity.f64(out), parity.f64(lse)
    print(f"\n{name}: max |out - oracle| = {np.abs(out - ref).max():.3e} (bound {tol:.3e})")
    assert np.abs(out - ref).max() <= tol
    fin = np.isfinite(rlse)
    np.testing.assert_array_equal(np.isfinite(lse), fin)
    assert np.abs(lse[fin] - rlse[fin]).max() <= score + 2.0 ** -20 * (1 + np.abs(rlse[fin]).max())


# Batches large enough that the tensor-core kernel takes the prefix (its rule:
# 4.5 to 13.5 ns per eight rows and 128 tokens, by the widths, above 10 us and
# 11.5 ns per 128 rows and 64 tokens): every width of K and of V, both tile
# sizes and scale types, blocks of 128 rows that are not full, odd groups,
# caches of large and of small values, and a first tile far from the others.
LARGE = {
    # N, Hq, Hkv, prefix, sequences, own tokens past the queries at most, Q, dtype, widths, more
    "k4v2": (128, 8, 1, 8192, 61, 200, 2, h, (4, 2, 4), {}),
    "k4v2_tile64_bf16": (64, 8, 1, 4096, 61, 90, 2, b16, (4, 2, 4), {}),
    "k4v2_group7_two_heads": (128, 14, 2, 4096, 70, 140, 1, h, (4, 2, 4), {}),
    "k6v6": (128, 8, 2, 4096, 50, 5, 1, h, (6, 6, 2), {}),
    "k8v8_fp32_scales": (128, 8, 1, 8192, 20, 129, 1, h, (8, 8, 4), {}),
    "k2v8_tile64": (64, 8, 1, 8192, 40, 3, 1, h, (2, 8, 2), {}),
    "k3v5": (128, 8, 1, 8192, 30, 20, 1, b16, (3, 5, 2), {}),
    "k8v3": (128, 8, 1, 8192, 30, 20, 1, h, (8, 3, 4), {}),
    "k5v4": (128, 8, 1, 8192, 40, 20, 1, h, (5, 4, 2), {}),
    "large_values": (128, 8, 1, 8192, 61, 9, 2, h, (4, 2, 4), dict(size=300.0)),
    "small_values": (128, 8, 1, 8192, 61, 9, 2, h, (4, 2, 4), dict(size=2.0 ** -9)),
    "first_tile_large": (128, 8, 1, 8192, 61, 9, 2, h, (4, 2, 4), dict(first=200.0, peak=0.05)),
    "first_tile_small": (64, 8, 1, 8192, 61, 9, 2, h, (4, 2, 4), dict(first=2.0 ** -9)),
    "sharp": (128, 8, 1, 8192, 61, 9, 2, h, (4, 2, 4), dict(peak=12.0)),
    "padding_verify": (128, 8, 1, 8192, 33, 150, 4, b16, (4, 2, 4), dict(pad=True)),
}


@pytest.mark.parametrize("name", list(LARGE))
def test_large_batches_match_the_definition(name):
    N, Hq, Hkv, prefix, B, most, Q, dtype, widths, more = LARGE[name]
    more = dict(more)
    pad = more.pop("pad", False)
    lens = [0 if pad and b % 5 == 3 else prefix + Q + (37 * b) % (most + 1) for b in range(B)]
    x = serving.Batch(128, N, Hq, Hkv, lens, Q=Q, prefix=prefix, dtype=dtype, widths=widths, seed=4, **more)
    ref, rlse = x.reference()
    out, lse, flags = serving.run_shared(x)
    assert flags == 0
    score, tol = x.bounds()
    out, lse = parity.f64(out), parity.f64(lse)
    print(f"\n{name}: max |out - definition| = {np.abs(out - ref).max():.3e} (bound {tol:.3e}), relative "
          f"{np.linalg.norm(out - ref) / np.linalg.norm(ref):.2e}")
    assert np.abs(out - ref).max() <= tol
    fin = np.isfinite(rlse)
    np.testing.assert_array_equal(np.isfinite(lse), fin)
    assert np.abs(lse[fin] - rlse[fin]).max() <= score + 2.0 ** -20 * (1 + np.abs(rlse[fin]).max())
    # the norm over the whole batch, where errors do not all add up: operands
    # split to 2^-22, a few hundred truncated fp32 accumulation steps
    assert np.linalg.norm(out - ref) <= 2.0 ** -14 * np.linalg.norm(ref)


def test_long_own_tokens():
    """Own tokens long enough for equal ranges of the tile list (six rounds
    of tiles per CTA) instead of pieces of units: only whole tiles differ, so
    the plain decode over the same pages is the reference."""
    own, B, Hkv, N = 64 * 64, 64, 8, 64
    lay = kv.dense_layout(128, N, Hkv, 64 * 40)
    g = torch.Generator(device="cuda").manual_seed(2)
    k, v = (torch.randn((1, Hkv, lay.num_pages * 16, 128), generator=g, device="cuda").half() for _ in range(2))
    cache, err = kv.alloc_cache(lay), kv.new_error_word()
    pages = torch.arange(lay.num_pages, dtype=torch.int32, device="cuda")
    kv.encode_tiles(k, v, lay, torch.zeros(1, dtype=torch.int32, device="cuda"), pages[None], cache, err)
    prefix, L = 2 * N, 2 * N + own
    tiles = torch.randint(0, lay.num_pages // 4, (B, L // N), generator=g, device="cuda")
    tiles[:, :2] = tiles[0, :2]
    bt = (tiles[..., None] * 4 + torch.arange(4, device="cuda")).flatten(1).to(torch.int32).contiguous()
    lens = torch.full((B,), L, dtype=torch.int32, device="cuda") - torch.arange(B, device="cuda", dtype=torch.int32) % 5 * N
    q = torch.randn((B, 1, 8, 128), generator=g, device="cuda").half()
    outs = []
    for shared in (True, False):
        out, lse = torch.empty((B, 1, 8, 128), device="cuda"), torch.empty((B, 1, 8), device="cuda")
        if shared:
            ws = torch.empty(kv.decode_shared_workspace_bytes(lay, B, 8, 1, L, prefix), dtype=torch.uint8, device="cuda")
            kv.decode_shared(q, lay, cache, bt[0, :prefix // 16].contiguous(), prefix, bt, lens, L, out, ws, err, 0.1, lse=lse)
        else:
            ws = torch.empty(kv.decode_verify_workspace_bytes(lay, B, 8, 1, L), dtype=torch.uint8, device="cuda")
            kv.decode_verify(q, lay, cache, bt, lens, L, out, ws, err, 0.1, lse=lse)
        torch.cuda.synchronize()
        outs.append((out, lse))
    assert kv.read_error_flags(err) == 0
    # both sides: 64 accumulation steps of 2^-23 and exponents off by 2^-17
    # of scores below 16
    assert float((outs[0][0] - outs[1][0]).norm()) <= 2.0 ** -13 * float(outs[1][0].norm())
    assert float((outs[0][1] - outs[1][1]).abs().max()) <= 2.0 ** -13


def test_bad_pages_are_flagged_by_the_large_path():
    x = serving.Batch(128, 64, 8, 1, [4096 + 3] * 61, Q=2, prefix=4096, seed=4)
    good = x.prefix_table.copy()
    for at, page in ((200, x.cache.shape[0]), (0, -1), (255, 2 ** 31 - 1)):
        x.prefix_table[:] = good
        x.prefix_table[at] = page
        assert serving.run_shared(x)[2] == kv.DEVERR_PAGE_RANGE


def test_infinite_and_nan_queries_stay_in_their_rows():
    x = serving.Batch(128, 64, 8, 1, [4096 + 3] * 61, Q=2, prefix=4096, seed=4)
    want, _, _ = serving.run_shared(x)
    x.q[7, 1, 3, 5], x.q[20, 0, 0, 100] = float("nan"), float("inf")
    got, _, flags = serving.run_shared(x)
    assert flags == 0
    bad = torch.zeros(want.shape[:3], dtype=torch.bool, device="cuda")
    bad[7, 1, 3] = bad[20, 0, 0] = True
    assert torch.equal(got[~bad], want[~bad])
    assert not torch.isfinite(got[bad]).any()


def test_agrees_with_the_decode_that_reads_the_prefix_per_sequence():
    x = batch("g8_many")
    out, lse, _ = serving.run_shared(x)
    lay, B, Lmax = x.layout_of(), len(x.lens), int(x.lens.max())
    o2, l2 = torch.empty((B, x.Hq, x.D), device="cuda"), torch.empty((B, x.Hq), device="cuda")
    ws = torch.empty(kv.decode_workspace_bytes(lay, B, x.Hq, Lmax), dtype=torch.uint8, device="cuda")
    err = kv.new_error_word()
    kv.decode(x.q[:, 0].contiguous().cuda(), lay, torch.from_numpy(x.cache).cuda(), torch.from_numpy(x.full_table()).cuda(),
              torch.from_numpy(x.lens).cuda(), Lmax, o2, ws, err, x.sm, x.tail_k.cuda(), x.tail_v.cuda(), l2)
    torch.cuda.synchronize()
    score, tol = x.bounds()
    assert float((out[:, 0] - o2).abs().max()) <= 2 * tol
    assert float((lse[:, 0] - l2).abs().max()) <= 2 * (score + 2.0 ** -16)


def test_without_lse_and_tails():
    x = batch("pair")
    x.lens[:] = 128  # the prefix alone: no tail needed
    lay = x.layout_of()
    out = torch.empty((2, 1, 4, 128), device="cuda")
    ws = torch.empty(kv.decode_shared_workspace_bytes(lay, 2, 4, 1, 128, 128), dtype=torch.uint8, device="cuda")
    err = kv.new_error_word()
    kv.decode_shared(x.q.cuda(), lay, torch.from_numpy(x.cache).cuda(), torch.from_numpy(x.prefix_table).cuda(), 128,
                     torch.from_numpy(x.bt).cuda(), torch.from_numpy(x.lens).cuda(), 128, out, ws, err, x.sm)
    torch.cuda.synchronize()
    assert kv.read_error_flags(err) == 0
    ref, _ = x.oracle()
    assert np.abs(parity.f64(out) - ref).max() <= x.bounds()[1]


def test_capture_replays_and_two_captures_share_a_workspace():
    x = batch("many_rows")
    lay, B, Lmax = x.layout_of(), len(x.lens), int(x.lens.max())
    q = x.q.cuda()
    args = [lay, torch.from_numpy(x.cache).cuda(), torch.from_numpy(x.prefix_table).cuda(), x.prefix,
            torch.from_numpy(x.bt).cuda(), torch.from_numpy(x.lens).cuda(), Lmax]
    ws = torch.empty(kv.decode_shared_workspace_bytes(lay, B, x.Hq, 1, Lmax, x.prefix), dtype=torch.uint8, device="cuda")
    err, tk, tv = kv.new_error_word(), x.tail_k.cuda(), x.tail_v.cuda()
    eager, _, _ = serving.run_shared(x)
    graphs, outs = [], [torch.empty_like(eager) for _ in range(2)]
    for o in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            kv.decode_shared(q, *args, o, ws, err, x.sm, tk, tv)
        graphs.append(g)
    for o in outs:
        o.fill_(float("nan"))
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], eager) and torch.equal(outs[1], eager)
    q.copy_(torch.randn(q.shape, generator=torch.Generator().manual_seed(8)).to(q.dtype))
    x.q = q.cpu()
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], serving.run_shared(x)[0])
    assert kv.read_error_flags(err) == 0


def test_another_stream():
    x = batch("k6v6")
    want, _, _ = serving.run_shared(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got, _, flags = serving.run_shared(x)
    assert flags == 0 and torch.equal(got, want)


@pytest.mark.parametrize("name", ["pair", "many_rows", "wide", "verify8"])
def test_bad_pages_and_lengths_are_flagged(name):
    x = batch(name)
    good = x.prefix_table.copy()
    x.prefix_table[3] = x.cache.shape[0] + 5
    assert serving.run_shared(x)[2] == kv.DEVERR_PAGE_RANGE
    x.prefix_table[:] = good
    x.prefix_table[0] = -1
    assert serving.run_shared(x)[2] == kv.DEVERR_PAGE_RANGE
    x.prefix_table[:] = good
    x.lens[0] = x.prefix - 1  # does not hold the prefix
    assert serving.run_shared(x)[2] == kv.DEVERR_SEQ_LEN
