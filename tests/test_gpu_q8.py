"""The 8-bit block cache: blocks written, read back and completed by appended tokens, bit for bit; attention over
them against its definition in 64 bits, over windows, sinks, lengths, head layouts and types."""
import numpy as np
import pytest
import torch

import quantized_kv_cache_kvarn_gb300 as kv
from tests import blocks8 as b8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_kv_cache_kvarn_gb300 import build
    build.build()
    kv.lib()


def np32(t):
    return t.detach().float().cpu().numpy()


def blocks(B, H, C, D, dt, seed, heads_first):
    """Keys and values with a zero block, a tiny one, one of the largest magnitudes, one with an infinity and one
    with a NaN, and values half-way between codes."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((2, B, H, C, D)) * np.exp(rng.standard_normal((2, B, H, 1, D)))
    x = x.reshape(2, B, H, C // 16, 16, D)
    x[0, 0, 0, 0] = 0
    x[1, 0, 0, 0] *= 2.0 ** -20
    if C >= 64:
        x[0, 0, 0, 1] *= 60000 / np.abs(x[0, 0, 0, 1]).max()
        x[1, 0, 0, 1, 3, 5] = np.inf
        x[0, 0, 0, 2, 15, D - 1] = np.nan
        x[1, 0, 0, 2] = np.round(x[1, 0, 0, 2] * 2) / 2
        x[1, 0, 0, 2, 0, 0] = 127 / 2  # halves of an int8 step
        x[0, 0, 0, 3] = -2.0 ** -14 * np.abs(x[0, 0, 0, 3])
    t = torch.from_numpy(x.reshape(2, B, H, C, D).astype(np.float32)).to(dt).cuda()
    if not heads_first:
        t = t.transpose(2, 3).contiguous().transpose(2, 3)
    return t[0], t[1]


@pytest.mark.parametrize("code", [b8.E4M3, b8.INT8])
@pytest.mark.parametrize("B,H,C,D,bf16,heads_first", [(1, 1, 16, 128, False, True), (3, 2, 64, 128, True, False),
                                                      (2, 3, 80, 256, False, False), (2, 1, 64, 256, True, True)])
def test_blocks_are_written_and_read_bit_for_bit(B, H, C, D, bf16, heads_first, code):
    dt = torch.bfloat16 if bf16 else torch.float16
    k, v = blocks(B, H, C, D, dt, 5, heads_first)
    n = C // 16
    starts = [2, -1, 0][:B]
    table = torch.randperm(B * (n + 3), generator=torch.Generator().manual_seed(1)).to(torch.int32).view(B, n + 3)
    lay = kv.q8_layout(D, H, B * (n + 3), kv.BF16 if bf16 else kv.FP16)
    cache = torch.full((lay.num_pages, H, kv.q8_page_bytes(lay)), 171, dtype=torch.uint8, device="cuda")
    start, err = torch.tensor(starts, dtype=torch.int32).cuda(), kv.new_error_word()
    kv.q8_encode_blocks(k, v, lay, code, start, table.cuda(), cache, err)
    got = cache.cpu().numpy()
    assert kv.read_error_flags(err) == 0
    written = np.zeros(lay.num_pages, bool)
    values = {}
    for b, s in enumerate(starts):
        for u in range(n if s >= 0 else 0):
            page = int(table[b, s + u])
            written[page] = True
            for h in range(H):
                sides = [b8.code_bytes(np32(x[b, h, 16 * u:16 * u + 16]), code) for x in (k, v)]
                want = b8.pack_page(sides[0][0], sides[0][1], sides[1][0], sides[1][1])
                assert np.array_equal(got[page, h][:32 * D], want[:32 * D]), (b, u, h)
                a, w = got[page, h][32 * D:32 * D + 8].copy().view(np.float32), want[32 * D:32 * D + 8].copy().view(np.float32)
                assert np.array_equal(a, w, equal_nan=True), (b, u, h)
                values[b, h, u] = [(b8.byte_values(c, code) * np.float64(s)) for c, s in sides]
    assert (got[~written] == 171).all()  # nothing else is touched
    ko, vo = (torch.full_like(k, 3.0), torch.full_like(v, 3.0))
    kv.q8_read_blocks(ko, vo, lay, code, start, table.cuda(), cache, err)
    for b, s in enumerate(starts):
        if s < 0:
            assert (ko[b] == 3).all() and (vo[b] == 3).all()
            continue
        for h in range(H):
            for u in range(n):
                for x, want in zip((ko, vo), values[b, h, u]):
                    # code * scale is exact in 64 bits; the kernel rounds it to fp32 and then to the type
                    w = torch.from_numpy(want).float().to(dt)
                    assert torch.equal(x[b, h, 16 * u:16 * u + 16].cpu().nan_to_num(777), w.nan_to_num(777)), (b, h, u)
    assert kv.read_error_flags(err) == 0


def test_bad_pages_are_flagged_and_skipped():
    k, v = blocks(2, 1, 64, 128, torch.float16, 6, True)
    lay = kv.q8_layout(128, 1, 8)
    cache, err = torch.full((8, 1, 4128), 9, dtype=torch.uint8, device="cuda"), kv.new_error_word()
    table = torch.tensor([[0, 8, 1, 2], [-1, 3, 4, 5]], dtype=torch.int32).cuda()
    kv.q8_encode_blocks(k, v, lay, 0, torch.tensor([0, 1], dtype=torch.int32).cuda(), table, cache, err)
    assert kv.read_error_flags(err) == kv.DEVERR_PAGE_RANGE
    touched = [(cache[i] != 9).any().item() for i in range(8)]
    assert touched == [True, True, True, True, True, True, False, False]


RAGGED = [0, 1, 2, 15, 16, 17, 31, 32, 33, 47, 100, 257, 1000]


@pytest.mark.parametrize("code", [b8.E4M3, b8.INT8])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("Hq,Hkv,D,Q", [(4, 1, 128, 1), (8, 1, 128, 1), (4, 4, 128, 1), (6, 2, 128, 3), (8, 1, 128, 8), (16, 2, 128, 2),
                                        (3, 1, 256, 1), (12, 2, 256, 1), (10, 2, 256, 3), (8, 1, 256, 8)])
def test_decode_of_ragged_lengths(Hq, Hkv, D, Q, bf16, code):
    x = b8.Batch(RAGGED, Hq, Hkv, D, Q=Q, code=code, bf16=bf16, seed=Hq + D + Q).gpu(kv)
    check(x)


@pytest.mark.parametrize("window,sinks", [(1, 0), (2, 1), (5, 4), (16, 16), (17, 3), (64, 37), (100, 0), (300, 128), (999, 5),
                                          (1000, 5), (2000, 9), (3, 5000)])
@pytest.mark.parametrize("Hq,Hkv,D,Q,code", [(8, 2, 128, 1, b8.E4M3), (8, 1, 128, 5, b8.INT8), (6, 1, 256, 2, b8.E4M3)])
def test_windows_and_sinks(Hq, Hkv, D, Q, code, window, sinks):
    check(b8.Batch(RAGGED, Hq, Hkv, D, Q=Q, window=window, sinks=sinks, code=code, seed=window + sinks, pad_columns=3).gpu(kv))


def check(x, out=None, lse=None):
    if out is None:
        out, lse = x.decode(kv)
    want, want_lse, off, off_lse = x.expected()
    assert kv.read_error_flags(x.t["err"]) == 0
    got, got_lse = out.cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= off).all(), (np.abs(got - want) / np.maximum(off, 1e-300)).max()
    fine = np.isfinite(want_lse)
    assert np.array_equal(np.isneginf(got_lse), ~fine)
    assert (np.abs(got_lse[fine] - want_lse[fine]) <= off_lse[fine]).all()
    assert (got[~fine] == 0).all()


@pytest.mark.parametrize("lens,Hq,Hkv", [([40000], 8, 1), ([5] * 700, 4, 2), ([3000, 7, 0, 9000, 12], 16, 2)])
def test_long_and_many(lens, Hq, Hkv):
    check(b8.Batch(lens, Hq, Hkv, 128, seed=3).gpu(kv))


def test_append_fills_tails_and_completes_blocks():
    for D, bf16, code in ((128, False, b8.E4M3), (256, True, b8.INT8)):
        dt = torch.bfloat16 if bf16 else torch.float16
        lens, H, cap = [0, 1, 15, 16, 17, 32, 160, 33], 3, 19
        B = len(lens)
        g = torch.Generator().manual_seed(D)
        k, v = (torch.randn((B, H, D), generator=g).to(dt).cuda() for _ in range(2))
        tk, tv = (torch.randn((B, H, cap, D), generator=g).to(dt).cuda() for _ in range(2))
        tk0, tv0 = tk.clone(), tv.clone()
        table = torch.randperm(B * 10, generator=g).to(torch.int32).view(B, 10).cuda()
        lay = kv.q8_layout(D, H, B * 10, kv.BF16 if bf16 else kv.FP16)
        cache, err = kv.alloc_q8_cache(lay).fill_(5), kv.new_error_word()
        kv.q8_append(k, v, lay, code, torch.tensor(lens, dtype=torch.int32).cuda(), 160, tk, tv, table, cache, err)
        assert kv.read_error_flags(err) == 0
        got, pages = cache.cpu().numpy(), set()
        for b, L in enumerate(lens):
            row = (L - 1) % 16
            if L and row < 15:
                tk0[b, :, row], tv0[b, :, row] = k[b], v[b]
            elif L:
                page = int(table[b, L // 16 - 1])
                pages.add(page)
                for h in range(H):
                    sides = [b8.code_bytes(np.concatenate([np32(t[b, h, :15]), np32(x[b, h])[None]]), code)
                             for t, x in ((tk0, k), (tv0, v))]
                    want = b8.pack_page(sides[0][0], sides[0][1], sides[1][0], sides[1][1])
                    assert np.array_equal(got[page, h][:32 * D + 8], want[:32 * D + 8]), (b, h)
        assert torch.equal(tk, tk0) and torch.equal(tv, tv0)
        rest = [i for i in range(B * 10) if i not in pages]
        assert (got[rest] == 5).all()


def test_append_of_bad_lengths_is_flagged():
    lay = kv.q8_layout(128, 1, 4)
    cache, err = kv.alloc_q8_cache(lay), kv.new_error_word()
    k = torch.ones((2, 1, 128), dtype=torch.float16, device="cuda")
    tk, tv = (torch.zeros((2, 1, 16, 128), dtype=torch.float16, device="cuda") for _ in range(2))
    kv.q8_append(k, k, lay, 0, torch.tensor([33, -4], dtype=torch.int32).cuda(), 32, tk, tv,
                 torch.zeros((2, 2), dtype=torch.int32).cuda(), cache, err)
    assert kv.read_error_flags(err) == kv.DEVERR_SEQ_LEN
    assert not tk.any() and not cache.any()


def test_hidden_values_do_not_matter():
    """Infinities and NaN in tokens that a query does not see: behind its window, between the sinks and the window in
    a page that both touch, under verification after it, and behind the last token."""
    Q, W, S = 4, 20, 5
    x = b8.Batch([39, 64, 70, 200], 8, 2, 128, Q=Q, window=W, sinks=S, seed=8).gpu(kv)
    first, first_lse = (t.clone() for t in x.decode(kv))
    check(x, first, first_lse)
    D = 128
    for b, L in enumerate(x.lens):
        # blocks of which query 0 sees nothing, but which lie in an item with others
        for u in range(x.done[b]):
            lo, hi = 16 * u, 16 * u + 16
            seen = any(i < S or i > L - Q - W for i in range(lo, hi))
            if not seen and x.table[b, u] != 0x7fffffff:
                x.t["cache"][int(x.table[b, u]), :, 32 * D:32 * D + 8] = 255  # scales NaN
    # the tokens under verification after query 0: its row stays as it was, the later ones become NaN
    for bad in (float("nan"), float("inf")):
        tk, tv = x.t["tail_k"].clone(), x.t["tail_v"].clone()
        for b, L in enumerate(x.lens):
            at = L - Q + 1 - 16 * x.done[b]
            tk[b, :, at:], tv[b, :, at:] = bad, bad
        out, lse = x.decode(kv, tail_k=tk, tail_v=tv)
        assert torch.equal(out[:, 0], first[:, 0]) and torch.equal(lse[:, 0], first_lse[:, 0])
        assert out[:, 1:].isnan().all()


def test_a_block_of_nan_is_nan_where_it_is_seen():
    x = b8.Batch([100, 64], 4, 1, 128, seed=2).gpu(kv)
    x.t["cache"][int(x.table[0, 3]), :, 32 * 128:32 * 128 + 4] = 255
    out, lse = x.decode(kv)
    assert out[0].isnan().all() and lse[0].isnan().all() and not out[1].isnan().any()
    x.t["q"][1, 0, 2, 7] = float("inf")
    out, _ = x.decode(kv)
    assert out[1, 0, 2].isnan().all() and not out[1, 0, :2].isnan().any() and not out[1, 0, 3].isnan().any()


@pytest.mark.parametrize("k_power,v_power,q_power", [(-60, 40, 0), (60, -90, 0), (0, 0, -30), (0, 100, 20)])
def test_scales_of_any_size(k_power, v_power, q_power):
    """Blocks and queries a power of two apart (bf16, which holds them): the softmax of the scaled scores."""
    x = b8.Batch([333, 50], 4, 1, 128, bf16=True, seed=4)
    D = 128
    for n, p in ((0, k_power), (4, v_power)):
        s = np.ascontiguousarray(x.cache[..., 32 * D + n:32 * D + n + 4]).view(np.float32) * np.float32(2.0 ** p)
        x.cache[..., 32 * D + n:32 * D + n + 4] = s.view(np.uint8)
    x.tails[0] *= np.float32(2.0 ** k_power)
    x.tails[1] *= np.float32(2.0 ** v_power)
    x.q *= np.float32(2.0 ** q_power)
    x.k, x.v = [k * 2.0 ** k_power for k in x.k], [v * 2.0 ** v_power for v in x.v]
    x.sm = float(np.float32(x.sm * 2.0 ** (-k_power - q_power)))
    check(x.gpu(kv))


def test_values_of_blocks_far_apart():
    """A block whose values are 2^60 times the others': the output is its share of them, to the weights' 2^-36."""
    x = b8.Batch([160], 4, 1, 128, bf16=True, seed=11)
    D, page = 128, int(x.table[0, 4])
    s = np.ascontiguousarray(x.cache[page, :, 32 * D + 4:32 * D + 8]).view(np.float32) * np.float32(2.0 ** 60)
    x.cache[page, :, 32 * D + 4:32 * D + 8] = s.view(np.uint8)
    x.v[0][:, 64:80] *= 2.0 ** 60
    check(x.gpu(kv))


def test_bad_pages_and_lengths_in_decode():
    x = b8.Batch([100, 64], 4, 1, 128, seed=2).gpu(kv)
    first = x.decode(kv)[0].clone()
    table = x.t["table"].clone()
    table[0, 2] = -1
    out, _ = x.decode(kv, table=table)
    assert kv.read_error_flags(x.t["err"]) == kv.DEVERR_PAGE_RANGE
    assert torch.equal(out[1], first[1])
    x.t["err"].zero_()
    x.decode(kv, lens=torch.tensor([101, -5], dtype=torch.int32).cuda())
    assert kv.read_error_flags(x.t["err"]) == kv.DEVERR_SEQ_LEN
    x.t["err"].zero_()
    x.decode(kv, tail_k=None, tail_v=None)
    assert kv.read_error_flags(x.t["err"]) == kv.DEVERR_NO_TAIL
    x.t["err"].zero_()
    out, _ = x.decode(kv)
    assert kv.read_error_flags(x.t["err"]) == 0 and torch.equal(out, first)


def test_streams_graphs_and_repeats():
    """The same bits again, on another stream, and from two captured graphs with workspaces of their own."""
    x = b8.Batch([777, 0, 90, 3000], 16, 2, 128, Q=2, window=500, sinks=4, seed=6).gpu(kv)
    first, lse = (t.clone() for t in x.decode(kv))
    check(x, first, lse)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, _ = x.decode(kv, out=torch.zeros_like(first), stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(out, first)
    graphs, outs = [], []
    for _ in range(2):
        outs.append(torch.zeros_like(first))
        g = torch.cuda.CUDAGraph()
        space = torch.empty_like(x.t["space"])
        with torch.cuda.graph(g):
            x.decode(kv, out=outs[-1], space=space)
        graphs.append((g, space))
    for _ in range(3):
        for g, _ in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], first) and torch.equal(outs[1], first)


def test_waits_that_run_out_are_flagged():
    x = b8.Batch([3000, 500], 8, 2, 128, seed=9).gpu(kv)
    first = x.decode(kv)[0].clone()
    torch.cuda.synchronize()
    kv.set_copy_wait_test(1000000, True)
    try:
        x.decode(kv)
        assert kv.read_error_flags(x.t["err"]) == kv.DEVERR_TIMEOUT
    finally:
        kv.set_copy_wait_test(0)
    x.t["err"].zero_()
    assert torch.equal(x.decode(kv)[0], first) and kv.read_error_flags(x.t["err"]) == 0
