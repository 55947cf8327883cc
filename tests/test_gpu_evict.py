"""Eviction of tiles by mass against its definition: budgets, protected tiles,
ties, NaN, in place, long rows, and the decode over the shortened sequence."""
import numpy as np
import pytest
import torch

import quantized_kv_cache_kvarn_gb300 as kv
from oracle import attention
from tests import parity, serving

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_kv_cache_kvarn_gb300 import build
    build.build()
    kv.lib()


def run(mass, table, lens, N, max_len, keep, sink, recent, inplace=False):
    m, t, l = (torch.from_numpy(a.copy()).cuda() for a in (mass, table, lens))
    mo, to, lo = (m, t, l) if inplace else (torch.full_like(m, float("nan")), torch.full_like(t, -7), torch.full_like(l, -7))
    freed, count = torch.full_like(t, -7), torch.full_like(l, -7)
    err = kv.new_error_word()
    kv.evict_tiles(m, t, l, kv.dense_layout(128, N, 1, 1 << 20), max_len, keep, mo, to, lo, freed, count, err,
                   sink_tiles=sink, recent_tiles=recent)
    torch.cuda.synchronize()
    return [x.cpu().numpy() for x in (mo, to, lo, freed, count)], kv.read_error_flags(err)


def inputs(lens, N, T, seed, kind):
    g = np.random.default_rng(seed)
    B = len(lens)
    mass = g.standard_normal((B, T)).astype(np.float32)
    if kind == "ties":
        mass = g.integers(0, 3, (B, T)).astype(np.float32)
        mass[mass == 0] = np.where(g.random((mass == 0).sum()) < 0.5, 0.0, -0.0)
    elif kind == "equal":
        mass[:] = 1.5
    elif kind == "odd":
        mass[g.random((B, T)) < 0.2] = np.nan
        mass[g.random((B, T)) < 0.1] = -np.nan
        mass[g.random((B, T)) < 0.2] = np.inf
        mass[g.random((B, T)) < 0.2] = -np.inf
        mass[g.random((B, T)) < 0.2] = np.finfo(np.float32).tiny / 4
    n = N // 16
    table = g.permutation(B * T * n).astype(np.int32).reshape(B, T * n)
    for b, L in enumerate(lens):
        mass[b, L // N:] = 0
        table[b, L // N * n:] = -1
    return mass, table, np.array(lens, np.int32)


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("kind", ["spread", "ties", "equal", "odd"])
@pytest.mark.parametrize("N,lens,keep,sink,recent", [
    (128, [0, 1, 127, 128, 1280, 1300, 5000], 4, 1, 2),
    (64, [64 * 9 + 3, 64 * 8, 64 * 5], 8, 0, 0),
    (64, [64 * 2500 + 7, 64 * 1025, 64 * 1024, 64 * 1023], 700, 3, 30),
    (128, [128 * 40, 128 * 3], 0, 0, 0),
    (128, [128 * 40, 128 * 3], 5, 2, 3),      # the protected ones alone
    (64, [64 * 33], 32, 0, 32),
    (64, [64 * 33], 32, 32, 0),
    (128, [128 * 20], 1000, 1, 1),
])
def test_matches_definition(N, lens, keep, sink, recent, kind, inplace):
    T = max(lens) // N
    mass, table, lens = inputs(lens, N, T, keep + T, kind)
    got, flags = run(mass, table, lens, N, int(lens.max()), keep, sink, recent, inplace)
    assert flags == 0
    for a, b in zip(got, serving.evicted(mass, table, lens, N, keep, sink, recent)):
        np.testing.assert_array_equal(a, b)


@pytest.mark.parametrize("T,inplace", [(26001, False), (83001, False), (83001, True)])
def test_long_rows(T, inplace):
    """Rows over a whole cluster's shared memory, and longer ones, which one
    CTA walks chunk by chunk."""
    N = 64
    mass, table, lens = inputs([64 * T, 64 * 25000 + 9], N, T, 4, "ties")
    got, flags = run(mass, table, lens, N, 64 * T, 13000, 4, 100, inplace)
    assert flags == 0
    want = []
    for b in range(2):  # the definition by sorting (stable: equal masses stay from the left)
        C = int(lens[b]) // N
        key = mass[b, :C].astype(np.float64) + 0.0
        key[:4], key[C - 100:] = np.inf, np.inf
        keep = np.sort(np.argsort(-key, kind="stable")[:13000])
        want.append(keep)
        np.testing.assert_array_equal(got[0][b, :13000], mass[b, keep])
        np.testing.assert_array_equal(got[1][b].reshape(T, 4)[:13000], table[b].reshape(T, 4)[keep])
        gone = np.setdiff1d(np.arange(C), keep)
        np.testing.assert_array_equal(got[3][b].reshape(T, 4)[:len(gone)], table[b].reshape(T, 4)[gone])
        assert got[4][b] == 4 * len(gone) and got[2][b] == lens[b] - N * len(gone)
        assert (got[3][b][4 * len(gone):] == -1).all() and (got[1][b][4 * 13000:] == -1).all()


def test_padding_columns_and_rows_stay():
    """Entries past max_seq_len's tiles are nobody's."""
    N, T = 128, 6
    mass, table, lens = inputs([6 * N + 5, 2 * N], N, T, 9, "spread")
    m = torch.full((3, 10), 77.0, device="cuda")
    t = torch.full((3, 64), 77, dtype=torch.int32, device="cuda")
    m[:2, :T], t[:2, :T * 8] = torch.from_numpy(mass).cuda(), torch.from_numpy(table).cuda()
    f = torch.full_like(t, 77)
    l = torch.from_numpy(lens).cuda()
    cnt, err = torch.zeros_like(l), kv.new_error_word()
    kv.evict_tiles(m[:2], t[:2], l, kv.dense_layout(128, N, 1, 1000), 6 * N + 5, 3, m[:2], t[:2], l, f[:2], cnt, err)
    torch.cuda.synchronize()
    want = serving.evicted(mass, table, lens, N, 3, 0, 0)
    np.testing.assert_array_equal(m[:2, :T].cpu().numpy(), want[0])
    np.testing.assert_array_equal(t[:2, :T * 8].cpu().numpy(), want[1])
    assert (m[:, T:] == 77).all() and (m[2] == 77).all() and (t[:, T * 8:] == 77).all() and (t[2] == 77).all()
    assert (f[:, T * 8:] == 77).all() and (f[2] == 77).all()


def test_length_out_of_range_is_flagged():
    mass, table, lens = inputs([128 * 4, 128 * 4], 128, 4, 2, "spread")
    lens[0] = 10 ** 6
    _, flags = run(mass, table, lens, 128, 512, 2, 0, 0)
    assert flags == kv.DEVERR_SEQ_LEN
    lens[0] = -5
    _, flags = run(mass, table, lens, 128, 512, 2, 0, 0)
    assert flags == kv.DEVERR_SEQ_LEN


def test_mass_then_evict_then_decode():
    """The masses choose the tiles; the decode over the shortened sequence is
    the attention over the tokens that are left."""
    x = serving.Batch(128, 64, 8, 2, [64 * 12 + 30, 64 * 5, 64 * 3 + 1], seed=11, peak=4.0)
    T = 12
    _, _, mass, flags = serving.run_mass(x, torch.zeros((3, T)), 1.0)
    assert flags == 0
    lay, keep = x.layout_of(), 4
    bt, lens = torch.from_numpy(x.bt).cuda(), torch.from_numpy(x.lens).cuda()
    m_before = mass.cpu().numpy()
    freed, count, err = torch.full_like(bt, -7), torch.zeros_like(lens), kv.new_error_word()
    kv.evict_tiles(mass, bt, lens, lay, int(x.lens.max()), keep, mass, bt, lens, freed, count, err, sink_tiles=1,
                   recent_tiles=1)
    out = torch.empty((3, 8, 128), device="cuda")
    ws = torch.empty(kv.decode_workspace_bytes(lay, 3, 8, int(x.lens.max())), dtype=torch.uint8, device="cuda")
    kv.decode(x.q[:, 0].contiguous().cuda(), lay, torch.from_numpy(x.cache).cuda(), bt, lens, int(x.lens.max()), out, ws, err,
              x.sm, x.tail_k.cuda(), x.tail_v.cuda())
    torch.cuda.synchronize()
    assert kv.read_error_flags(err) == 0
    want = serving.evicted(m_before, x.bt, x.lens, 64, keep, 1, 1)
    np.testing.assert_array_equal(bt.cpu().numpy(), want[1])
    np.testing.assert_array_equal(lens.cpu().numpy(), want[2])
    assert sorted(set(x.bt[0][x.bt[0] >= 0])) == sorted(list(want[1][0][want[1][0] >= 0]) + list(want[3][0][want[3][0] >= 0]))
    tk, tv = (np.nan_to_num(parity.f64(t)) for t in (x.tail_k, x.tail_v))
    ref, _ = attention.decode(parity.f64(x.q[:, 0]), x.cache, x.lay, want[1], want[2], x.sm, tk, tv)
    _, tol = x.bounds()
    assert np.abs(parity.f64(out) - ref).max() <= tol
