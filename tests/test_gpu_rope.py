"""Rotary positions against their definition in extended precision: layouts,
types, part of the head, strides, positions to the ends of int32, in place,
the gradient against the formula's and against differences, capture."""
import numpy as np
import pytest
import torch

import quantized_kv_cache_kvarn_gb300 as kv

pytestmark = pytest.mark.gpu

# fp32 arithmetic, in units of 2^-24 scale (|x_a| + |x_b|): the fraction of a
# turn rounded to fp32 (pi: a relative 2^-24 of an angle of at most pi),
# sincospi (2 ulp below 1: 2), the scale's product (1), the product and the
# fused multiply-add (2): 8.2, and the phase itself 2^31 2^-65 turns.
UNITS = 9 * 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_kv_cache_kvarn_gb300 import build
    build.build()
    kv.lib()


def reference(x, pos, inv_freq, offset, interleaved, scale, inverse):
    """(y, sum of magnitudes) in extended precision. x [B, S, H, D] float64."""
    R = 2 * len(inv_freq)
    t = pos.astype(np.longdouble)[:, :, None, None] * inv_freq.astype(np.longdouble)
    c, s = (f.astype(np.float64) * scale for f in (np.cos(t), np.sin(t) * (-1 if inverse else 1)))
    y, mag = x.copy(), np.zeros_like(x)
    a = offset + (np.arange(0, R, 2) if interleaved else np.arange(R // 2))
    b = a + (1 if interleaved else R // 2)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., a] * s + x[..., b] * c
    mag[..., a] = mag[..., b] = scale * (np.abs(x[..., a]) + np.abs(x[..., b]))
    return y, mag


def tensor(B, S, H, D, dtype, order, g):
    x = torch.randn((B, H, S, D) if order == "heads" else (B, S, H, D), generator=g).to(dtype)
    return x.transpose(1, 2) if order == "heads" else x


def check(xs, outs, pos, inv_freq, offset, interleaved, scale, inverse):
    for x, y in zip(xs, outs):
        ref, mag = reference(x.double().cpu().numpy(), pos.cpu().numpy().astype(np.int64), inv_freq.cpu().numpy(), offset,
                             interleaved, scale, inverse)
        got = y.double().cpu().numpy()
        tol = UNITS * mag + (0 if x.dtype == torch.float32 else torch.finfo(x.dtype).eps / 2) * np.abs(ref) * (1 + 2.0 ** -10)
        # a pair's small difference may fall below the type's normal range
        tol = tol + (0 if x.dtype == torch.float32 else 2.0 ** -25 if x.dtype == torch.float16 else 0) + 1e-38
        bad = np.abs(got - ref) > np.where(mag > 0, tol, 0)
        assert not bad.any(), f"{bad.sum()} values off, worst {np.abs(got - ref).max():.3e}"


CASES = [
    # B, S, heads, D, R, offset, dtype, order, interleaved, scale, far
    (2, 5, (4, 1), 128, 128, 0, torch.float16, "tokens", False, 1.0, 4000),
    (1, 1, (64, 8), 128, 128, 0, torch.bfloat16, "tokens", True, 1.0, 1 << 30),
    (3, 17, (24, 4), 256, 64, 192, torch.bfloat16, "heads", True, 1.35, 1 << 20),
    (2, 9, (3, 3), 96, 48, 0, torch.float16, "heads", False, 0.5, 131072),
    (1, 700, (7, 2), 64, 64, 0, torch.float32, "tokens", False, 1.0, 1 << 24),
    (2, 33, (5,), 192, 64, 128, torch.float32, "heads", True, 2.0, 100),
    (1, 3, (2, 2), 20, 10, 3, torch.float16, "tokens", False, 1.0, 1000),   # no vector path
    (2, 2, (3, 1), 7, 2, 0, torch.float32, "tokens", True, 1.0, 1 << 29),
    (1, 4, (2,), 1024, 1024, 0, torch.float16, "heads", False, 1.0, 50000),
    (40, 64, (6, 2), 128, 32, 32, torch.float16, "heads", False, 1.0, 9000),
]


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_matches_definition(case, inverse):
    B, S, heads, D, R, offset, dtype, order, interleaved, scale, far = CASES[case]
    g = torch.Generator().manual_seed(case)
    xs = [tensor(B, S, h, D, dtype, order, g).cuda() for h in heads]
    pos = torch.randint(0, far, (B, S), generator=g).to(torch.int32).cuda()
    inv_freq, _ = kv.rope_frequencies(R, 10000.0)
    outs = [torch.full_like(x, float("nan")) for x in xs]
    call = kv.rope_backward if inverse else kv.rope
    call(xs, outs, pos, inv_freq, rope_offset=offset, interleaved=interleaved, scale=scale)
    torch.cuda.synchronize()
    check(xs, outs, pos, inv_freq, offset, interleaved, scale, inverse)
    # in place gives the same values
    same = [x.clone() for x in xs]
    same = [s if s.stride() == x.stride() else torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device=x.device).copy_(x)
            for s, x in zip(same, xs)]
    call(same, same, pos, inv_freq, rope_offset=offset, interleaved=interleaved, scale=scale)
    torch.cuda.synchronize()
    for a, b in zip(same, outs):
        assert torch.equal(a, b)


def test_ends_of_the_positions_and_unscaled_zero():
    x = torch.randn((1, 6, 2, 64), generator=torch.Generator().manual_seed(1)).cuda()
    pos = torch.tensor([[0, 1, -1, 2 ** 31 - 1, -2 ** 31, 12345678]], dtype=torch.int32, device="cuda")
    freqs = torch.cat([torch.tensor([0.0, 1e-300, 2.0 ** -70, 5.0, 7.5], dtype=torch.float64),
                       torch.rand(27, generator=torch.Generator().manual_seed(2), dtype=torch.float64)]).cuda()
    y = torch.empty_like(x)
    kv.rope(x, y, pos, freqs)
    torch.cuda.synchronize()
    check([x], [y], pos, freqs, 0, False, 1.0, False)
    assert torch.equal(y[:, 0], x[:, 0])  # position 0 turns nothing


def test_strided_views_and_shared_positions():
    """Queries and keys inside one fused projection, outputs into another
    layout, one row of positions for the batch."""
    g = torch.Generator().manual_seed(3)
    B, S, Hq, Hkv, D = 3, 10, 8, 2, 128
    qkv = torch.randn((B, S, (Hq + 2 * Hkv) * D), generator=g).half().cuda()
    q = qkv[..., :Hq * D].unflatten(-1, (Hq, D))
    k = qkv[..., Hq * D:(Hq + Hkv) * D].unflatten(-1, (Hkv, D))
    before = qkv.clone()
    pos = torch.arange(100, 100 + S, dtype=torch.int32, device="cuda")[None]
    inv_freq, _ = kv.rope_frequencies(D)
    qo = torch.empty_like(q)
    ko = torch.empty((B, Hkv, S, D), dtype=k.dtype, device="cuda").transpose(1, 2)
    kv.rope([q, k], [qo, ko], pos, inv_freq)
    torch.cuda.synchronize()
    check([q, k], [qo, ko], pos.expand(B, S), inv_freq, 0, False, 1.0, False)
    assert torch.equal(qkv, before)
    # the same through a misaligned view (element by element), and in place of it
    odd = torch.empty(q.numel() + 1, dtype=q.dtype, device="cuda")[1:].view(B, S, Hq, D).copy_(q)
    out = torch.empty_like(odd)
    kv.rope(odd, out, pos, inv_freq)
    torch.cuda.synchronize()
    check([odd], [out], pos.expand(B, S), inv_freq, 0, False, 1.0, False)
    # nothing past the rotated tensors is written
    kv.rope([q, k], [q, k], pos, inv_freq)
    torch.cuda.synchronize()
    assert torch.equal(qkv[..., (Hq + Hkv) * D:], before[..., (Hq + Hkv) * D:])
    assert torch.equal(q, qo) and torch.equal(k, ko)


def test_infinities_and_nan_stay_in_their_pairs():
    x = torch.ones((1, 2, 1, 128)).cuda()
    x[0, 0, 0, 5], x[0, 0, 0, 40] = float("inf"), float("nan")
    y = torch.empty_like(x)
    pos = torch.tensor([[3, 3]], dtype=torch.int32, device="cuda")
    inv_freq, _ = kv.rope_frequencies(128)
    kv.rope(x, y, pos, inv_freq)
    torch.cuda.synchronize()
    touched = [5, 69, 40, 104]
    rest = [i for i in range(128) if i not in touched]
    assert not torch.isfinite(y[0, 0, 0, touched]).any()
    assert torch.equal(y[0, 0, 0, rest], y[0, 1, 0, rest])


def test_gradient_against_differences():
    """fp32: the loss sum w rope(x) is linear in x, so a central difference of
    step h is exact up to the rounding of the outputs, whose size is 2 |w|_1
    |x| 2^-24 / h per component; w, x of size 1, 64 channels and h = 1 bound
    the error of a component by 64 * 2^-23 * 6 < 5e-5."""
    g = torch.Generator().manual_seed(5)
    x = torch.randn((1, 3, 2, 64), generator=g).cuda()
    w = torch.randn((1, 3, 2, 64), generator=g).cuda()
    pos = torch.tensor([[7, 900, 131071]], dtype=torch.int32, device="cuda")
    inv_freq, scale = kv.rope_frequencies(32, yarn=(4.0, 4096))
    kw = dict(rope_offset=16, interleaved=True, scale=scale)
    grad = torch.empty_like(x)
    kv.rope_backward(w, grad, pos, inv_freq, **kw)

    def loss(v):
        y = torch.empty_like(v)
        kv.rope(v, y, pos, inv_freq, **kw)
        return (y.double() * w.double()).sum()

    for idx in [(0, 0, 0, 0), (0, 0, 1, 16), (0, 1, 0, 17), (0, 2, 1, 30), (0, 2, 0, 47), (0, 1, 1, 63)]:
        e = torch.zeros_like(x)
        e[idx] = 1.0
        diff = (loss(x + e) - loss(x - e)) / 2
        assert abs(float(diff) - float(grad[idx])) < 5e-5


def test_capture_and_another_stream():
    g = torch.Generator().manual_seed(6)
    x = torch.randn((4, 1, 10, 128), generator=g).half().cuda()
    y, pos = torch.empty_like(x), torch.tensor([[5], [6], [70], [8000]], dtype=torch.int32, device="cuda")
    inv_freq, _ = kv.rope_frequencies(128)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    kv.rope(x, y, pos, inv_freq, stream=s)
    s.synchronize()
    eager = y.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kv.rope(x, y, pos, inv_freq)
    y.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, eager)
    pos += 1
    graph.replay()
    torch.cuda.synchronize()
    check([x], [y], pos, inv_freq, 0, False, 1.0, False)


def test_nothing_to_do():
    inv_freq, _ = kv.rope_frequencies(16)
    x = torch.empty((0, 4, 2, 16), device="cuda")
    kv.rope(x, x, torch.empty((0, 4), dtype=torch.int32, device="cuda"), inv_freq)
    x = torch.empty((2, 0, 2, 16), device="cuda")
    kv.rope(x, x, torch.empty((2, 0), dtype=torch.int32, device="cuda"), inv_freq)
