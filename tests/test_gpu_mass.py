"""kvarn_decode_mass: the decode's outputs bit for bit, and every tile's
attention mass against the softmax of the dequantised cache in 64 bits."""
import numpy as np
import pytest
import torch

import quantized_kv_cache_kvarn_gb300 as kv
from oracle import attention
from tests import parity, serving

pytestmark = pytest.mark.gpu

CASES = {
    # D, N, Hq, Hkv, lens, dtype, widths
    "g8": (128, 128, 16, 2, [700, 128, 127, 0, 1290], torch.float16, (4, 2, 4)),
    "tile64": (128, 64, 6, 2, [1, 64, 333, 65, 640], torch.float16, (4, 2, 4)),
    "wide_bf16": (256, 128, 12, 4, [517, 384], torch.bfloat16, (4, 2, 4)),
    "k6v6_group1": (128, 128, 7, 7, [400, 256], torch.bfloat16, (6, 6, 2)),
    "k4v2_fp16_scales_tile64": (128, 64, 14, 2, [400, 256, 63], torch.float16, (4, 2, 2)),
    "k4v4_wide": (256, 128, 8, 2, [300, 256], torch.float16, (4, 4, 2)),
    "k8v8": (128, 128, 8, 1, [700, 128], torch.float16, (8, 8, 2)),
    "k8v8_wide_tile64": (256, 64, 8, 1, [200, 70], torch.float16, (8, 8, 2)),
    "only_tails": (128, 128, 4, 1, [5, 127], torch.float16, (4, 2, 4)),
}


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_kv_cache_kvarn_gb300 import build
    build.build()
    kv.lib()


def tile_masses(x):
    """Weights per tile summed over heads, [B, T], in 64 bits."""
    T = int(x.lens.max()) // x.N
    out = np.zeros((len(x.lens), max(1, T)))
    G = x.Hq // x.Hkv
    for b, L in enumerate(x.lens):
        for h in range(x.Hq if L else 0):
            k, _ = attention.sequence_kv(x.cache, x.lay, x.bt[b], int(L), h // G, np.nan_to_num(parity.f64(x.tail_k[b, h // G])),
                                         np.nan_to_num(parity.f64(x.tail_v[b, h // G])))
            s = x.sm * (k @ parity.f64(x.q[b, 0, h]))
            p = np.exp(s - s.max())
            p /= p.sum()
            for t in range(int(L) // x.N):
                out[b, t] += p[t * x.N:(t + 1) * x.N].sum()
    return out


@pytest.mark.parametrize("name", list(CASES))
def test_masses_match_the_weights(name):
    D, N, Hq, Hkv, lens, dtype, widths = CASES[name]
    x = serving.Batch(D, N, Hq, Hkv, lens, dtype=dtype, widths=widths, seed=3)
    ref = tile_masses(x)
    T = ref.shape[1]
    before = torch.rand((len(lens), T), generator=torch.Generator().manual_seed(1)) * 3
    out, lse, new, flags = serving.run_mass(x, before, 0.75)
    assert flags == 0
    done = x.lens // N
    want = np.where(np.arange(T) < done[:, None], 0.75 * before.double().numpy() + ref, 0.0)
    if int(x.lens.max()) // N == 0:  # no tile at all: nothing is written
        assert torch.isnan(new).all()
    else:
        # a weight is off by its score's error and 2^-20 (exp2, lse), a
        # mass by that of its weights, and the sum with decay by 2^-23 more
        score, _ = x.bounds()
        tol = ref * (2 * score + 2.0 ** -19) + want * 2.0 ** -22
        assert (np.abs(parity.f64(new) - want) <= tol + 1e-30).all(), np.abs(parity.f64(new) - want).max()
    # the decode itself is untouched
    lay = x.layout_of()
    Lmax = int(x.lens.max())
    o2, l2 = torch.empty_like(out), torch.empty_like(lse)
    ws = torch.empty(kv.decode_workspace_bytes(lay, len(lens), Hq, Lmax), dtype=torch.uint8, device="cuda")
    err = kv.new_error_word()
    kv.decode(x.q[:, 0].contiguous().cuda(), lay, torch.from_numpy(x.cache).cuda(), torch.from_numpy(x.bt).cuda(),
              torch.from_numpy(x.lens).cuda(), Lmax, o2, ws, err, x.sm, x.tail_k.cuda(), x.tail_v.cuda(), l2)
    torch.cuda.synchronize()
    assert torch.equal(out, o2) and torch.equal(lse, l2)


def test_accumulates_in_place_without_lse_and_repeats_exactly():
    x = serving.Batch(128, 128, 8, 2, [900, 260], seed=5)
    lay, B = x.layout_of(), 2
    ref = tile_masses(x)
    q, cache, bt, lens = x.q[:, 0].contiguous().cuda(), torch.from_numpy(x.cache).cuda(), torch.from_numpy(x.bt).cuda(), \
        torch.from_numpy(x.lens).cuda()
    tk, tv = x.tail_k.cuda(), x.tail_v.cuda()
    out = torch.empty((B, 8, 128), device="cuda")
    ws = torch.empty(kv.decode_mass_workspace_bytes(lay, B, 8, 900), dtype=torch.uint8, device="cuda")
    err = kv.new_error_word()
    runs = []
    for _ in range(2):
        mass = torch.zeros((B, 12), device="cuda")[:, :9]  # rows further apart than their tiles
        for _ in range(3):
            kv.decode_mass(q, lay, cache, bt, lens, 900, out, mass, mass, ws, err, x.sm, tk, tv)
        torch.cuda.synchronize()
        runs.append(mass.clone())
    assert kv.read_error_flags(err) == 0
    assert torch.equal(*runs)
    score, _ = x.bounds()
    assert (np.abs(parity.f64(runs[0][:, :7]) - 3 * ref) <= 3 * ref * (2 * score + 2.0 ** -18) + 1e-30).all()
    assert not runs[0][:, 7:].any()
    # rows add up to the heads' weight in the pages, at most one each
    assert (runs[0].sum(1) <= 3 * 8 * (1 + 1e-5)).all()


def test_decay_zero_forgets_whatever_was_there():
    x = serving.Batch(128, 128, 8, 2, [900, 260], seed=5)
    ref = tile_masses(x)
    _, _, new, flags = serving.run_mass(x, torch.full((2, 7), float("nan")), 0.0)
    assert flags == 0
    score, _ = x.bounds()
    assert (np.abs(parity.f64(new) - ref) <= ref * (2 * score + 2.0 ** -19) + 1e-30).all()


def test_length_out_of_range_is_flagged():
    x = serving.Batch(128, 128, 4, 1, [300, 256], seed=6)
    lens = torch.tensor([300, 1000], dtype=torch.int32).cuda()
    lay = x.layout_of()
    out = torch.empty((2, 4, 128), device="cuda")
    mass = torch.zeros((2, 2), device="cuda")
    ws = torch.empty(kv.decode_mass_workspace_bytes(lay, 2, 4, 300), dtype=torch.uint8, device="cuda")
    err = kv.new_error_word()
    kv.decode_mass(x.q[:, 0].contiguous().cuda(), lay, torch.from_numpy(x.cache).cuda(), torch.from_numpy(x.bt).cuda(), lens,
                   300, out, mass, mass, ws, err, x.sm, x.tail_k.cuda(), x.tail_v.cuda())
    torch.cuda.synchronize()
    assert kv.read_error_flags(err) & kv.DEVERR_SEQ_LEN
