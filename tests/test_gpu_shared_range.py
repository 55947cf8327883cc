"""Shared prefix, tensor-core path: tiles whose values differ in size by up to
2^24, wherever a split meets them, and tiles of zeros, row by row against the
definition in 64 bits."""
import numpy as np
import pytest
import torch

import quantized_kv_cache_kvarn_gb300 as kv
from oracle import attention, layout
from tests import parity, serving

pytestmark = pytest.mark.gpu

# N, prefix, widths, dtype, exponent of the values of tile t
CASES = {
    "first_small": (128, 8192, (4, 2, 4), torch.float16, lambda t: -15 if t == 0 else 9),
    "first_large": (128, 8192, (4, 2, 4), torch.float16, lambda t: 9 if t == 0 else -15),
    "fifths_large": (128, 8192, (4, 2, 4), torch.float16, lambda t: 9 if t % 5 == 0 else -15),
    "fifths_small": (128, 8192, (4, 2, 4), torch.float16, lambda t: -15 if t % 5 == 0 else 9),
    "fifths_large_tile64": (64, 4096, (4, 2, 4), torch.bfloat16, lambda t: 12 if t % 5 == 0 else -12),
    "fifths_small_tile64": (64, 4096, (4, 2, 4), torch.bfloat16, lambda t: -12 if t % 5 == 0 else 12),
    "far_apart": (128, 8192, (4, 2, 4), torch.bfloat16, lambda t: 24 if t % 5 == 0 else -20),
    "growing": (128, 8192, (4, 2, 4), torch.float16, lambda t: -14 + t * 22 // 63),
    "shrinking": (128, 8192, (4, 2, 4), torch.float16, lambda t: 8 - t * 22 // 63),
    "fp16_scales_20": (128, 8192, (6, 6, 2), torch.float16, lambda t: 8 if t % 5 == 0 else -12),
    "fp16_scales_16": (64, 8192, (4, 4, 2), torch.float16, lambda t: -8 if t % 5 == 0 else 8),
    "zeros_first": (128, 8192, (4, 2, 4), torch.float16, lambda t: None if t < 2 else -12),
    "zeros_fifths": (128, 8192, (4, 2, 4), torch.float16, lambda t: None if t % 5 == 0 else 8 if t % 2 else -14),
    "huge_bf16": (128, 8192, (4, 2, 4), torch.bfloat16, lambda t: 104 if t % 5 == 0 else 90),
    "tiny_bf16": (64, 4096, (4, 2, 4), torch.bfloat16, lambda t: -86 if t % 5 == 0 else -80),
    "zeros_tiny_bf16": (128, 8192, (4, 2, 4), torch.bfloat16, lambda t: None if t % 5 == 0 else -80),
    "zeros_huge_bf16": (128, 8192, (4, 2, 4), torch.bfloat16, lambda t: None if t % 5 == 4 else 100),
    "zeros_only": (128, 8192, (4, 2, 4), torch.float16, lambda t: None),
}
B, Q, HQ, D, DIR = 61, 2, 8, 128, 10.6


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_kv_cache_kvarn_gb300 import build
    build.build()
    kv.lib()


def batch(name):
    """A batch whose even rows look at the tiles t % 5 == 0 and whose odd rows
    at the others (scores about 20 apart), a few tokens of a tile each."""
    N, prefix, widths, dtype, exponent = CASES[name]
    x = serving.Batch(D, N, HQ, 1, [prefix + Q - 1 + b % 3 for b in range(B)], Q=Q, prefix=prefix, dtype=dtype,
                      widths=widths, seed=7)
    g = torch.Generator().manual_seed(8)
    u = torch.sign(torch.randn(D, generator=g)) / D ** 0.5
    tile = torch.arange(prefix) // N
    k = 3.0 * torch.randn((prefix, D), generator=g) + torch.where(tile % 5 == 0, DIR, -DIR)[:, None] * u
    e = [exponent(t) for t in range(prefix // N)]
    size = torch.tensor([0.0 if v is None else 2.0 ** v for v in e], dtype=torch.float64)
    v = (torch.randn((prefix, D), generator=g).double() * size[tile][:, None])
    attention.encode_into_cache(x.cache, x.lay, parity.f64(k.to(dtype))[None, None], parity.f64(v.to(dtype))[None, None],
                                x.prefix_table[None], [0])
    sign = torch.where(torch.arange(B * Q * HQ) % 2 == 0, 1.0, -1.0)
    q = 0.5 * torch.randn((B * Q * HQ, D), generator=g) + sign[:, None] * DIR * u
    x.q = q.to(dtype).view(B, Q, HQ, D)
    # own tokens of the size of the smallest tile, so that they hide nothing
    own = min([v for v in e if v is not None], default=0)
    x.tail_v = (x.tail_v.double() * 2.0 ** own).to(dtype)
    return x


def definition(x):
    """(out, lse, bound) per row in 64 bits on the GPU. The bound is the L2
    norm of the output's error:
      scores      products of operands split to 2^-22 of each (hi hi + lo hi +
                  hi lo: three such errors) and a sum in eight truncated steps
                  of 2^-23 (the sixteen of the small products count 2^-11),
                  three more roundings: 17 2^-23 of sum_j |q_j k_j|, below
                  2^-18 |q| max |k| sm; and the smallest steps of the split
                  operands, 2^-25 of the row's and of the tile's unit on each
                  channel: a row's unit is at most 2 |q|, a tile's `unit` = 2
                  max |c| max |a code + b| (and more than a quarter of that),
                  so 2^-24 sm (unit |q|_1 + 2 |q| sqrt(D) max |k|)
      weights     off by their own and the sum's score errors, by 2^-20 (exp2
                  and sums) and 2^-22 (the split)
      values      2^-22, and 2^-25 of the tile's unit on each channel
      the sum     four truncated steps a stage over at most 64 stages in a
                  split, 2^-15, which covers the merge's sums too
      smallest    P is a weight times its tile's power of two, in units of at
      weights     most twice the row's largest such product (`share`), and
                  exact to 2^-25: a weight to 2^-25 2 share 4 / unit, or it
                  is lost"""
    G = HQ
    out, lse, bound = (np.zeros((B, Q, HQ, D)), np.zeros((B, Q, HQ)), np.zeros((B, Q, HQ)))
    pk, pv = (torch.from_numpy(np.ascontiguousarray(a)).cuda()
              for a in attention.sequence_kv(x.cache, x.lay, x.prefix_table, x.prefix, 0))
    ppt, tiles = x.N // 16, x.prefix // x.N
    unit = torch.zeros(2, tiles, dtype=torch.float64)
    for t in range(tiles):
        for i, (s, bits) in enumerate(zip(layout.read_tile(x.cache, x.lay, x.prefix_table[t * ppt:(t + 1) * ppt], 0),
                                          x.widths)):
            rows = np.maximum(np.abs(s["b"]), np.abs(s["a"] * ((1 << bits) - 1) + s["b"])).max()
            unit[i, t] = 2 * float(rows) * float(np.abs(s["c"]).max())
    unit = unit.cuda()
    q = torch.from_numpy(parity.f64(x.q)).cuda()
    tk, tv = (torch.from_numpy(np.nan_to_num(parity.f64(t))).cuda() for t in (x.tail_k, x.tail_v))
    # rotated rows: the arithmetic's operands
    H = torch.from_numpy(serving._hadamard(D)).cuda()
    for b, L in enumerate(x.lens):
        n = int(L) - x.prefix
        k, v = torch.cat([pk, tk[b, 0, :n]]), torch.cat([pv, tv[b, 0, :n]])
        qb = q[b]  # [Q, G, D]
        s = x.sm * torch.einsum("qgd,ld->qgl", qb, k)
        seen = torch.tensor([attention.verify_visible(int(L), Q, j) for j in range(Q)], device="cuda")
        s = s.masked_fill(torch.arange(len(k), device="cuda") >= seen[:, None, None], -torch.inf)
        z = torch.logsumexp(s, -1)
        w = torch.exp(s - z[..., None])
        norm = v.norm(dim=-1)
        q2, q1 = qb.norm(dim=-1), (qb @ H).abs().sum(-1)
        kunit = unit[0].max()
        score = x.sm * (2.0 ** -18 * q2 * k.norm(dim=-1).max() + 2.0 ** -24 * (kunit * q1 + 2 * q2 * D ** 0.5 * k.norm(dim=-1).max()))
        big = w[..., :x.prefix].unflatten(-1, (tiles, x.N)).amax(-1)
        share = (big * unit[1]).amax(-1)
        per = unit[1].repeat_interleave(x.N)
        floor = torch.minimum(w[..., :x.prefix], 2.0 ** -22 * share[..., None] / per.clamp(min=1e-300))
        err = (2 * score + 2.0 ** -20 + 2.0 ** -22 + 2.0 ** -15) * (w * norm).sum(-1)
        err += 2.0 ** -22 * (w * norm).sum(-1) + 2.0 ** -25 * D ** 0.5 * (w[..., :x.prefix] * per).sum(-1)
        err += (floor * norm[:x.prefix]).sum(-1)
        out[b] = torch.einsum("qgl,ld->qgd", w, v).cpu().numpy()
        lse[b] = z.cpu().numpy()
        bound[b] = err.cpu().numpy()
    return out, lse, bound


@pytest.mark.parametrize("name", list(CASES))
def test_rows_of_tiles_of_any_size(name):
    x = batch(name)
    ref, rlse, bound = definition(x)
    out, lse, flags = serving.run_shared(x)
    assert flags == 0
    out, lse = parity.f64(out), parity.f64(lse)
    assert np.isfinite(out).all() and np.isfinite(lse).all()
    err, size = np.linalg.norm(out - ref, axis=-1), np.linalg.norm(ref, axis=-1)
    rel = err / np.maximum(size, 1e-300)
    print(f"\n{name}: largest error of a row {rel.max():.2e} of it, bounds {(bound / np.maximum(size, 1e-300)).min():.2e} to "
          f"{(bound / np.maximum(size, 1e-300)).max():.2e}; largest error / bound {(err / np.maximum(bound, 1e-300)).max():.3f}")
    assert (err <= bound).all()
    assert np.abs(lse - rlse).max() <= x.bounds()[0] + 2.0 ** -20 * (1 + np.abs(rlse).max())
