"""Attention over the 8-bit block cache at the ends of what its numbers may be: queries, keys, values and scales of any
size in coded blocks and in the raw tail, scores of any size, sinks up to the largest length, waits that run out."""
import ctypes

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


def scaled(lens, Hq, Hkv, D, Q, k_power, v_power, q_power, seed):
    """A bf16 batch whose keys, values and queries are a power of two of those of another one, the softmax's scale such
    that the scores are the other one's (but for what queries lose below the smallest bf16 number)."""
    x = b8.Batch(lens, Hq, Hkv, D, Q=Q, bf16=True, seed=seed)
    for n, p in ((0, k_power), (4, v_power)):
        at = slice(32 * D + n, 32 * D + n + 4)
        with np.errstate(over="ignore"):  # pages that hold no block hold any bytes
            s = np.ascontiguousarray(x.cache[..., at]).view(np.float32) * np.float32(2.0 ** p)
        x.cache[..., at] = s.view(np.uint8)
    x.tails[0] *= np.float32(2.0 ** k_power)
    x.tails[1] *= np.float32(2.0 ** v_power)
    x.q = torch.from_numpy(x.q.astype(np.float64) * 2.0 ** q_power).to(torch.bfloat16).float().numpy()
    x.k, x.v = [k * 2.0 ** k_power for k in x.k], [v * 2.0 ** v_power for v in x.v]
    x.sm = float(np.float32(x.sm * 2.0 ** (-k_power - q_power)))
    return x


HEADS = [(4, 1, 128, 1), (8, 1, 128, 3), (3, 1, 256, 1), (6, 1, 256, 3)]  # Hq, Hkv, D, Q: eight rows and sixteen


@pytest.mark.parametrize("Hq,Hkv,D,Q", HEADS[::2])
@pytest.mark.parametrize("k_power,q_power", [(122, 0), (122, -100), (120, -126), (-95, 110), (-90, 0), (60, -126), (0, -128), (0, 123)])
def test_scores_of_blocks_of_any_size(k_power, q_power, Hq, Hkv, D, Q):
    """Without a tail."""
    check(scaled([320, 48], Hq, Hkv, D, Q, k_power, 0, q_power, 7).gpu(kv))


@pytest.mark.parametrize("Hq,Hkv,D,Q", HEADS)
@pytest.mark.parametrize("k_power,v_power,q_power", [(122, 0, 0), (122, 0, -100), (-95, 0, 110), (0, 123, 0), (0, -90, 0), (110, 120, -126),
                                                     (122, 123, -122), (0, 0, 123), (0, 0, -128)])
@pytest.mark.parametrize("lens", [[13, 15, 1], [333, 50, 9]])
def test_raw_tails_of_any_size(lens, k_power, v_power, q_power, Hq, Hkv, D, Q):
    """Tails alone, and behind coded blocks of the same sizes."""
    check(scaled(lens, Hq, Hkv, D, Q, k_power, v_power, q_power, 9).gpu(kv))


@pytest.mark.parametrize("Hq,Hkv,D,Q", HEADS)
@pytest.mark.parametrize("power", [-90, -40, 20, 71, 72, 73, 110])
def test_a_block_of_other_values_than_the_rest(power, Hq, Hkv, D, Q):
    """Values of one block a power of two of the others': the output is the sum of the shares, the larger ones' to what fp32
    counts (a share of less than 2^-36 of the largest is within what the largest may be off by)."""
    x = b8.Batch([160 + Q - 1, 77], Hq, Hkv, D, Q=Q, bf16=True, seed=11)
    page = int(x.table[0, 4])
    s = np.ascontiguousarray(x.cache[page, :, 32 * D + 4:32 * D + 8]).view(np.float32) * np.float32(2.0 ** power)
    x.cache[page, :, 32 * D + 4:32 * D + 8] = s.view(np.uint8)
    x.v[0][:, 64:80] *= 2.0 ** power
    check(x.gpu(kv))


@pytest.mark.parametrize("Hq,Hkv,D,Q", HEADS)
@pytest.mark.parametrize("power", [20, 22, 24])
@pytest.mark.parametrize("lens", [[320, 64], [13, 7], [333, 50]])
def test_scores_beyond_what_fp32_counts(lens, power, Hq, Hkv, D, Q):
    """Scores of 2^24 and more, which fp32 holds in steps of two and more: where one token is ahead of the others by more
    than what scores may be off by, the output is its value (the weight is hi + lo and the scale's mantissa a product:
    2^-20 of it) and the lse its score."""
    x = b8.Batch([L + Q - 1 for L in lens], Hq, Hkv, D, Q=Q, seed=3)
    x.sm *= 2.0 ** power
    x.gpu(kv)
    out, lse = (t.cpu().numpy().astype(np.float64) for t in x.decode(kv))
    assert kv.read_error_flags(x.t["err"]) == 0
    seen = 0
    for b, L in enumerate(x.lens):
        for j in range(Q):
            for h in range(Hq):
                k, v, q = x.k[b][h // (Hq // Hkv)][:L - Q + j + 1], x.v[b][h // (Hq // Hkv)], x.q[b, j, h].astype(np.float64)
                s = x.sm * (k @ q)
                off = x.sm * (D / 2 + 4) * 2.0 ** -23 * (np.abs(k) @ np.abs(q))
                i = int(s.argmax())
                if len(s) > 1 and s[i] - off[i] - 200 <= np.delete(s + off, i).max():
                    continue
                seen += abs(s[i]) > 2.0 ** (power + 1)
                assert (np.abs(out[b, j, h] - v[i]) <= 2.0 ** -20 * np.abs(v[i])).all(), (b, j, h, s[i])
                assert abs(lse[b, j, h] - s[i]) <= off[i] + 2.0 ** -22 * abs(s[i])
    assert seen >= Q


@pytest.mark.parametrize("sinks", [(1 << 31) - 16, (1 << 31) - 15, (1 << 31) - 1])
def test_sinks_up_to_the_largest_length(sinks):
    """max_seq_len of 2^31 - 1: every token is one of the sinks."""
    x = b8.Batch([100, ], 4, 1, 128, seed=2).gpu(kv)
    t, most = x.t, (1 << 31) - 1
    P = ctypes.c_void_p
    # the table's row is as long as the stride says; entries behind the sequence's blocks are not read
    code = kv.lib().kvarn_q8_decode(P(t["q"].data_ptr()), 4, 1, x.sm, P(t["cache"].data_ptr()), ctypes.byref(x.layout), x.code,
                                    P(t["table"].data_ptr()), most // 16, P(t["lens"].data_ptr()), most, P(t["tail_k"].data_ptr()),
                                    P(t["tail_v"].data_ptr()), t["tail_k"].shape[2], 20, sinks, 1, P(t["out"].data_ptr()),
                                    P(t["lse"].data_ptr()), P(t["space"].data_ptr()), t["space"].numel(), P(t["err"].data_ptr()),
                                    P(torch.cuda.current_stream().cuda_stream))
    assert code == 0
    check(x, t["out"], t["lse"])


def test_a_pair_that_gives_up_leaves_at_once():
    """At head_dim 256 two warps share an item; where one's wait runs out both leave as soon as the copies that were asked
    for have landed, long before the 1e8 cycles (48 ms) that a copy that never comes would be waited for."""
    B, Hq, Hkv, D, L = 16, 8, 2, 256, 16384
    pages = B * L // 16  # 270 MB: pages come from memory, and waits are long wherever a warp is
    g = torch.Generator(device="cuda").manual_seed(0)
    lay = kv.q8_layout(D, Hkv, pages)
    cache = torch.randint(0, 100, (pages, Hkv, kv.q8_page_bytes(lay)), generator=g, device="cuda", dtype=torch.uint8)
    cache[..., 32 * D:] = torch.tensor([0.01, 0.01] + [0.0] * 6, device="cuda").view(torch.uint8)
    table = torch.randperm(pages, generator=g, device="cuda").int().view(B, L // 16)
    lens, err = torch.full((B,), L, dtype=torch.int32, device="cuda"), kv.new_error_word()
    q = torch.randn((B, 1, Hq, D), generator=g, device="cuda").half()
    out = torch.empty((B, 1, Hq, D), device="cuda")
    space = torch.empty(kv.q8_decode_workspace_bytes(lay, B, Hq, 1, L), dtype=torch.uint8, device="cuda")

    def call():
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        kv.q8_decode(q, lay, 0, cache, table, lens, L, out, space, err, D ** -0.5)
        b.record()
        torch.cuda.synchronize()
        flags = kv.read_error_flags(err)
        err.zero_()
        return a.elapsed_time(b), flags

    for _ in range(3):
        assert call()[1] == 0
    first = out.clone()
    assert first.isfinite().all()
    gave_up, slowest = 0, 0.0
    try:
        for cycles in (1, 50, 200, 500, 1000, 2000, 3000, 5000, 8000):
            kv.set_copy_wait_test(cycles)
            for _ in range(5):
                ms, flags = call()
                assert flags == kv.DEVERR_TIMEOUT or (flags == 0 and torch.equal(out, first))
                gave_up, slowest = gave_up + (flags != 0), max(slowest, ms)
    finally:
        kv.set_copy_wait_test(0)
    assert gave_up > 0 and slowest < 20, (gave_up, slowest)
    assert call()[1] == 0 and torch.equal(out, first)
