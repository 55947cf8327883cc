"""The decode loop of test_gpu_serving_step.py row by row and tile by tile:
outputs by the L2 norm of a row's error, masses relative to each tile's own,
against bounds formed from the step's weights in 64 bits."""
import numpy as np
import pytest
import torch

import quantized_kv_cache_kvarn_gb300 as kv
from oracle import attention, layout
from tests import parity, serving
from tests.test_gpu_serving_step import KEEP, LONGEST, PREFIX, B, D, Hkv, Hq, Loop, N

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_kv_cache_kvarn_gb300 import build
    build.build()
    kv.lib()


def expected(x):
    """(outputs, bound of each row's error, masses, bound of each mass
    relative to it). A score is a sum of products whose operands are split to
    2^-22 of each, in at most 24 fp32 or tensor-core steps off by 2^-23, with
    scales that add four roundings: below 2^-18 |q| max |k| sm. A weight is off
    by its own and its sum's score error and by 2^-20 (exp2, sums), a row by
    twice the scores' and the weights' errors of sum w |v|, the values' splits
    and 64 accumulation steps more: 2^-16. A mass adds up weights, and the sum
    over tokens, heads and slots is off by 2^-19."""
    lay = layout.DenseLayout(D, N)
    cache, table, lens = x.cache.cpu().numpy(), x.table.cpu().numpy(), x.lens.cpu().numpy()
    q, tk, tv = parity.f64(x.qr[:, 0]), parity.f64(x.tail_k), parity.f64(x.tail_v)
    T = LONGEST // N
    out, bound, mass, off = np.zeros((B, Hq, D)), np.zeros((B, Hq)), np.zeros((B, T)), np.zeros(B)
    for b, L in enumerate(lens):
        for g in range(Hkv):
            k, v = attention.sequence_kv(cache, lay, table[b], int(L), g, tk[b, g], tv[b, g])
            for h in range(g * Hq // Hkv, (g + 1) * Hq // Hkv):
                s = x.sm * (k @ q[b, h])
                p = np.exp(s - s.max())
                p /= p.sum()
                out[b, h] = p @ v
                score = 2.0 ** -18 * x.sm * np.linalg.norm(q[b, h]) * np.linalg.norm(k, axis=1).max()
                bound[b, h] = (2 * score + 2.0 ** -16) * (p @ np.linalg.norm(v, axis=1))
                off[b] = max(off[b], 2 * score + 2.0 ** -19)
                done = int(L) // N
                mass[b, :done] += p[:done * N].reshape(done, N).sum(1)
    return out, bound, mass, off


def test_rows_and_tiles_of_the_loop():
    x, g = Loop(13), torch.Generator().manual_seed(14)
    worst_row = worst_mass = 0.0
    evicted = 0
    for i in range(5 * N + 7):
        x.inputs(g)
        before = x.mass.double().cpu().numpy()
        x.step()
        if i % 29 == 0 or i % N in (N - 1, 0):  # and around every tile's end
            out, bound, mass, off = expected(x)
            for got in (x.out, x.out_shared[:, 0]):
                err = np.linalg.norm(parity.f64(got) - out, axis=-1)
                worst_row = max(worst_row, (err / bound).max())
                assert (err <= bound).all(), (i, (err / bound).max())
            done = x.lens.cpu().numpy()[:, None] // N > np.arange(LONGEST // N)
            want = np.where(done, 0.9 * before + mass, 0.0)
            err = np.abs(parity.f64(x.mass) - want)
            tol = mass * off[:, None] + want * 2.0 ** -22
            worst_mass = max(worst_mass, (err[done] / tol[done]).max() if done.any() else 0.0)
            assert (err <= tol).all(), (i, err.max())
        if i % 50 == 49:
            m, t, l = x.mass.cpu().numpy(), x.table.cpu().numpy(), x.lens.cpu().numpy()
            x.evict()
            want = serving.evicted(m, t, l, N, KEEP, PREFIX // N, 1)
            for a, b in zip((x.mass, x.table, x.lens, x.freed, x.count), want):
                np.testing.assert_array_equal(a.cpu().numpy(), b)
            for b in range(B):  # freed pages are used again, behind the row's kept ones
                n, c = int(x.lens[b]) // N * (N // 16), int(x.count[b])
                x.table[b, n:n + c] = x.freed[b, :c]
                x.table[b, n + c:] = torch.from_numpy(t[b, n + c:]).to(x.table.device)
                evicted += c // (N // 16)
    parity.report(f"decode loop with eviction: largest error of a row {worst_row:.3f} of its bound, of a mass {worst_mass:.3f}")
    assert evicted > 0
    assert kv.read_error_flags(x.err) == 0
