"""Norms of heads with their rotation in one pass, and the gradient, against the definition in 64 bits."""
import numpy as np
import pytest
import torch

import quantized_kv_cache_kvarn_gb300 as kv

pytestmark = pytest.mark.gpu

STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # half a step, relative
SMALL = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -126}  # half the smallest step


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_kv_cache_kvarn_gb300 import build
    build.build()
    kv.lib()


def turn(z, pos, inv, off, inter, scale):
    """z [B, S, H, D] turned by the positions, in float64; the gradient of a loss is turned by -inv."""
    if inv is None:
        return z
    a = pos.double()[..., None, None] * inv
    c, s = a.cos() * scale, a.sin() * scale
    n = inv.numel()
    i = torch.arange(n, device=z.device)
    ia, ib = (off + 2 * i, off + 2 * i + 1) if inter else (off + i, off + i + n)
    y = z.clone()
    y[..., ia] = z[..., ia] * c - z[..., ib] * s
    y[..., ib] = z[..., ia] * s + z[..., ib] * c
    return y


def spread(x, inv, off, inter):
    """|x_a| + |x_b| of a channel's pair, |x| of the others: what rounding errors of a rotation are relative to."""
    if inv is None:
        return x.abs()
    n = inv.numel()
    i = torch.arange(n, device=x.device)
    ia, ib = (off + 2 * i, off + 2 * i + 1) if inter else (off + i, off + i + n)
    y = x.abs().clone()
    y[..., ia] = y[..., ib] = x[..., ia].abs() + x[..., ib].abs()
    return y


# Relative error of r: a sum of D <= 1024 squares, at most 32 added one after another and five more times by a
# butterfly (37 roundings of 2^-24, halved by the root), the mean and the root (2^-22); then two products, the cosines and
# sines (2^-22 of one) and the turn's three roundings.
T = 40 * 2.0 ** -25 + 6 * 2.0 ** -23


def make(B, S, heads, D, dtype, wtype, rope, off, first, seed, offset=0.0, none=False):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def like(h):
        shape = (B, h, S, D) if first else (B, S, h, D)
        x = torch.randn(shape, generator=g, device="cuda") * torch.exp(torch.randn((*shape[:-1], 1), generator=g, device="cuda"))
        x = x.to(dtype)
        return x.transpose(1, 2) if first else x

    xs, dys = [like(h) for h in heads], [like(h) for h in heads]
    ws = [None if none else (1 - offset + 0.3 * torch.randn(D, generator=g, device="cuda")).to(wtype) for _ in heads]
    pos = torch.randint(-1000, 1 << 20, (B, S), generator=g, device="cuda", dtype=torch.int32)
    inv = 10000.0 ** (-torch.arange(rope // 2, device="cuda", dtype=torch.float64) / max(1, rope // 2)) if rope else None
    return xs, dys, ws, pos, inv


def reference(x, w, pos, inv, off, inter, scale, eps, offset):
    x, w = x.double(), (torch.ones((), dtype=torch.float64, device=x.device) if w is None else w.double()) + offset
    r = (x.square().mean(-1, keepdim=True) + eps).rsqrt()
    z = x * r * w
    return turn(z, pos, inv, off, inter, scale), T * abs(scale if inv is not None else 1) * spread(z, inv, off, inter) + T * z.abs()


def close(got, want, off):
    d = (got.double() - want).abs()
    assert (d <= off + STEP[got.dtype] * (want.abs() + off) + SMALL[got.dtype]).all(), (d / (off + STEP[got.dtype] * want.abs() + 1e-300)).max()


CASES = [
    # B, S, heads, D, rope, offset of the rope, interleaved, heads first
    (2, 5, (4, 1), 128, 128, 0, False, False), (1, 1, (64, 8), 128, 128, 0, True, False), (3, 7, (6, 2), 64, 32, 0, False, True),
    (2, 3, (5,), 256, 64, 16, True, False), (1, 4, (3, 2, 1), 96, 64, 8, False, False), (2, 33, (7, 7), 128, 0, 0, False, True),
    (1, 3, (2, 1), 512, 256, 128, False, False), (2, 2, (3,), 80, 20, 3, False, False), (1, 5, (2, 2), 33, 10, 1, True, False),
    (2, 3, (2,), 1024, 512, 0, False, False), (1, 2, (1,), 1, 0, 0, False, False), (1, 700, (9, 3), 128, 96, 32, False, False),
    (1, 2, (2,), 2, 2, 0, True, False),
]


@pytest.mark.parametrize("dtype,wtype", [(torch.float16, torch.float16), (torch.bfloat16, torch.float32), (torch.float32, torch.float32),
                                         (torch.float32, torch.bfloat16)])
@pytest.mark.parametrize("case", CASES)
def test_forward(case, dtype, wtype):
    B, S, heads, D, rope, off, inter, first = case
    xs, _, ws, pos, inv = make(B, S, heads, D, dtype, wtype, rope, off, first, D + S)
    outs = [torch.full_like(x, 9.0) for x in xs]
    more = dict(eps=1e-5, rope_offset=off, interleaved=inter, scale=1.25)
    kv.norm_rope(xs, outs, ws, pos, inv, **more)
    for x, y, w in zip(xs, outs, ws):
        close(y, *reference(x, w, pos, inv, off, inter, 1.25, 1e-5, 0.0))
    again = [x.clone() for x in xs]
    kv.norm_rope(again, again, ws, pos, inv, **more)  # in place: the same bits
    assert all(torch.equal(a, y) for a, y in zip(again, outs))


def gradients(x, dy, w, pos, inv, off, inter, scale, eps, offset):
    """dx, dw and how far fp32 may be from each: with eu what g is off by times the weight, mean(u h) is off by T of its
    terms' magnitudes and by eu; dx by those and by T of its two terms; dw by its terms' error and 200 additions."""
    x, dy = x.double(), dy.double()
    w = (torch.ones(x.shape[-1], dtype=torch.float64, device=x.device) if w is None else w.double()) + offset
    D = x.shape[-1]
    r = (x.square().mean(-1, keepdim=True) + eps).rsqrt()
    h = x * r
    g = turn(dy, pos, None if inv is None else -inv, off, inter, scale)
    eg = T * (abs(scale) if inv is not None else 1) * spread(dy, inv, off, inter)
    u, eu = g * w, eg * w.abs()
    m = (u * h).mean(-1, keepdim=True)
    em = (2 * T * u.abs() * h.abs() + eu * h.abs()).mean(-1, keepdim=True)
    dx = r * (u - h * m)
    ex = r * (eu + h.abs() * em + 2 * T * (u.abs() + (h * m).abs()))
    dw = (g * h).sum((0, 1, 2))
    ew = (eg * h.abs() + (2 * T + 200 * 2.0 ** -24) * (g * h).abs()).sum((0, 1, 2))
    return dx, ex, dw, ew


@pytest.mark.parametrize("dtype,wtype", [(torch.float16, torch.float16), (torch.bfloat16, torch.float32), (torch.float32, torch.float32)])
@pytest.mark.parametrize("case", CASES)
def test_backward(case, dtype, wtype):
    B, S, heads, D, rope, off, inter, first = case
    xs, dys, ws, pos, inv = make(B, S, heads, D, dtype, wtype, rope, off, first, D + S + 1, offset=1.0)
    outs, dws = [torch.full_like(x, 9.0) for x in xs], [torch.full((D,), 9.0, device="cuda") for _ in xs]
    space = torch.full((kv.norm_rope_backward_workspace_bytes(xs),), 255, dtype=torch.uint8, device="cuda")
    more = dict(eps=1e-5, weight_offset=1.0, rope_offset=off, interleaved=inter, scale=0.75)
    kv.norm_rope_backward(xs, dys, outs, ws, dws, pos, inv, space, **more)
    for x, dy, dx, w, dw in zip(xs, dys, outs, ws, dws):
        want, ex, want_w, ew = gradients(x, dy, w, pos, inv, off, inter, 0.75, 1e-5, 1.0)
        close(dx, want, ex)
        close(dw, want_w, ew)
    # over the gradients, some sums not wanted, then none: the same bits
    over, dw2 = [d.clone() for d in dys], [torch.empty(D, device="cuda")] + [None] * (len(xs) - 1)
    kv.norm_rope_backward(xs, over, over, ws, dw2, pos, inv, space, **more)
    assert all(torch.equal(a, b) for a, b in zip(over, outs)) and torch.equal(dw2[0], dws[0])
    over = [x.clone() for x in xs]
    kv.norm_rope_backward(over, dys, over, ws, None, pos, inv, None, **more)
    assert all(torch.equal(a, b) for a, b in zip(over, outs))


def test_the_formula_of_the_gradient_against_differences():
    xs, dys, ws, pos, inv = make(1, 3, (2,), 16, torch.float32, torch.float32, 8, 4, False, 3)
    x, dy, w = xs[0].double(), dys[0].double(), ws[0].double()

    def loss(x, w):
        return (reference(x, w, pos, inv, 4, True, 1.5, 1e-3, 0.0)[0] * dy).sum()

    dx, _, dw, _ = gradients(x, dy, w, pos, inv, 4, True, 1.5, 1e-3, 0.0)
    g = torch.Generator(device="cuda").manual_seed(0)
    for _ in range(5):
        ex, ew = torch.randn(x.shape, generator=g, device="cuda").double(), torch.randn(w.shape, generator=g, device="cuda").double()
        h = 1e-5
        slope = (loss(x + h * ex, w + h * ew) - loss(x - h * ex, w - h * ew)) / (2 * h)
        want = (dx * ex).sum() + (dw * ew).sum()
        # third derivatives times h^2, and 2^-53 / h of the loss's terms
        assert abs(slope - want) <= 1e-7 * ((dx * ex).abs().sum() + (dw * ew).abs().sum() + dy.abs().sum())


def test_shared_and_broadcast_inputs():
    """One position row for the batch; an input whose sequences are one; weights that are none."""
    xs, dys, _, pos, inv = make(3, 4, (4,), 128, torch.float32, torch.float32, 128, 0, False, 9)
    x, out = xs[0][:1].expand(3, -1, -1, -1), torch.empty_like(xs[0])
    kv.norm_rope(x, out, None, pos[:1], inv)
    close(out, *reference(x, None, pos[:1].expand(3, -1), inv, 0, False, 1.0, 1e-6, 0.0))
    dw, space = torch.empty(128, device="cuda"), torch.empty(kv.norm_rope_backward_workspace_bytes(x), dtype=torch.uint8, device="cuda")
    kv.norm_rope_backward(x, dys[0], out, None, dw, pos[:1], inv, space)
    want, ex, want_w, ew = gradients(x, dys[0], None, pos[:1].expand(3, -1), inv, 0, False, 1.0, 1e-6, 0.0)
    close(out, want, ex)
    close(dw, want_w, ew)
    with pytest.raises(kv.KvarnError):
        kv.norm_rope(xs[0], x, None, pos, inv)  # an output may not be broadcast


def test_views_with_odd_strides():
    """Queries and keys as slices of one projection, and one that starts at an odd channel."""
    g = torch.Generator(device="cuda").manual_seed(4)
    whole = torch.randn((2, 5, 10, 130), generator=g, device="cuda").to(torch.bfloat16)
    pos = torch.arange(10, device="cuda", dtype=torch.int32).view(2, 5)
    inv, _ = kv.rope_frequencies(64)
    for lo in (0, 1):
        xs = [whole[:, :, :8, lo:lo + 128], whole[:, :, 8:, lo:lo + 128]]
        outs = [torch.empty((2, 5, h, 128), dtype=torch.bfloat16, device="cuda") for h in (8, 2)]
        ws = [torch.ones(128, device="cuda"), torch.full((128,), 2.0, device="cuda")]
        kv.norm_rope(xs, outs, ws, pos, inv)
        for x, y, w in zip(xs, outs, ws):
            close(y, *reference(x, w, pos, inv, 0, False, 1.0, 1e-6, 0.0))


def test_values_at_the_ends():
    """A head of zeros, tiny and large ones, an infinity, a NaN: the others are not touched by them."""
    x = torch.randn((1, 1, 6, 128), device="cuda")
    x[0, 0, 0] = 0
    x[0, 0, 1] *= 2.0 ** -60
    x[0, 0, 2] *= 2.0 ** 40
    x[0, 0, 3, 5] = float("inf")
    x[0, 0, 4, 9] = float("nan")
    y = torch.empty_like(x)
    pos = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    inv, _ = kv.rope_frequencies(128)
    kv.norm_rope(x, y, None, pos, inv)
    assert (y[0, 0, 0] == 0).all() and y[0, 0, 4].isnan().all() and y[0, 0, 3, 5].isnan()
    fine = [1, 2, 5]
    want, off = reference(x[:, :, fine], None, pos, inv, 0, False, 1.0, 1e-6, 0.0)
    close(y[:, :, fine], want, off)


def test_eps_of_zero():
    """Heads and tokens that do not fill a CTA, with eps 0: rows that are not there bring nothing into the sums."""
    xs, dys, ws, pos, inv = make(1, 3, (3,), 128, torch.float32, torch.float32, 128, 0, False, 6)
    dx, dw = torch.empty_like(xs[0]), torch.empty(128, device="cuda")
    space = torch.empty(kv.norm_rope_backward_workspace_bytes(xs), dtype=torch.uint8, device="cuda")
    kv.norm_rope_backward(xs[0], dys[0], dx, ws[0], dw, pos, inv, space, eps=0.0)
    want, ex, want_w, ew = gradients(xs[0], dys[0], ws[0], pos, inv, 0, False, 1.0, 0.0, 0.0)
    close(dx, want, ex)
    close(dw, want_w, ew)


def test_nothing_to_do():
    inv, _ = kv.rope_frequencies(128)
    for B, S, H in ((0, 3, 2), (2, 0, 2), (2, 3, 0)):
        x = torch.empty((B, S, H, 128), device="cuda")
        pos = torch.zeros((B, S), dtype=torch.int32, device="cuda")
        kv.norm_rope(x, torch.empty_like(x), None, pos, inv)
        dw, space = torch.full((128,), 5.0, device="cuda"), torch.empty(max(1, kv.norm_rope_backward_workspace_bytes(x)), dtype=torch.uint8, device="cuda")
        kv.norm_rope_backward(x, torch.empty_like(x), torch.empty_like(x), None, dw, pos, inv, space)
        assert (dw == 0).all()  # a sum over nothing


def test_many_rows_streams_and_graphs():
    """More tokens than a CTA's share, the gradient replayed from a graph while eager calls go on elsewhere."""
    xs, dys, ws, pos, inv = make(2, 3001, (4, 1), 128, torch.bfloat16, torch.float32, 128, 0, False, 12)
    space = torch.empty(kv.norm_rope_backward_workspace_bytes(xs), dtype=torch.uint8, device="cuda")
    outs, dws = [torch.empty_like(x) for x in xs], [torch.empty(128, device="cuda") for _ in xs]
    kv.norm_rope_backward(xs, dys, outs, ws, dws, pos, inv, space)
    for x, dy, dx, w, dw in zip(xs, dys, outs, ws, dws):
        want, ex, want_w, ew = gradients(x, dy, w, pos, inv, 0, False, 1.0, 1e-6, 0.0)
        close(dx, want, ex)
        close(dw, want_w, ew)
    other, odw, ospace = [torch.zeros_like(x) for x in xs], [torch.zeros(128, device="cuda") for _ in xs], torch.empty_like(space)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kv.norm_rope_backward(xs, dys, other, ws, odw, pos, inv, ospace)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g.replay()
    kv.norm_rope_backward(xs, dys, outs, ws, dws, pos, inv, space, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(other + odw, outs + dws))
