"""The gradient of the norms' weights over many heads: the sums in fp32 stay short whatever the number of heads."""
import pytest
import torch

import quantized_kv_cache_kvarn_gb300 as kv
from tests.test_gpu_norm_rope import close, gradients, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_kv_cache_kvarn_gb300 import build
    build.build()
    kv.lib()


def backward(xs, dys, ws, pos, inv, **more):
    outs, dws = [torch.full_like(x, 9.0) for x in xs], [torch.full((x.shape[-1],), 9.0, device="cuda") for x in xs]
    space = torch.full((kv.norm_rope_backward_workspace_bytes(xs),), 255, dtype=torch.uint8, device="cuda")
    kv.norm_rope_backward(xs, dys, outs, ws, dws, pos, inv, space, **more)
    return outs, dws


@pytest.mark.parametrize("S,heads,D", [(1, 1 << 18, 64), (1, 1 << 18, 33), (3, 20001, 128), (2, 5003, 1000)])
def test_equal_terms(S, heads, D):
    """All terms of a sum are equal and a little more than a number that late additions of a long fp32 sum would round
    them to: a sum of n terms in a row is then off by up to n / 2 roundings, all of one sign. The tolerance is that of 200
    additions."""
    x = torch.ones((1, S, heads, D), device="cuda")
    dy = torch.full_like(x, 1 + 0.4 * 2.0 ** -10)
    outs, dws = backward([x], [dy], [None], None, None)
    want, ex, want_w, ew = gradients(x, dy, None, None, None, 0, False, 1.0, 1e-6, 0.0)
    close(dws[0], want_w, ew)
    close(outs[0], want, ex)


CASES = [
    # B, S, heads, D, rope, offset of the rope, interleaved, heads first
    (1, 3, (1500, 1), 512, 512, 0, False, False), (1, 2, (1024, 1025), 512, 64, 64, True, False), (2, 1, (9001,), 128, 64, 0, False, False),
    (1, 2, (3, 2500), 96, 20, 3, False, False), (1, 1, (1029,), 1000, 10, 1, True, True), (1, 4900, (131, 2), 512, 0, 0, False, False),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("case", CASES)
def test_many_heads(case, dtype):
    """More heads than one CTA adds up, beside tensors of few; some sums not wanted; the same bits again."""
    B, S, heads, D, rope, off, inter, first = case
    xs, dys, ws, pos, inv = make(B, S, heads, D, dtype, torch.float32, rope, off, first, D + S, offset=1.0)
    more = dict(eps=1e-5, weight_offset=1.0, rope_offset=off, interleaved=inter, scale=0.75)
    outs, dws = backward(xs, dys, ws, pos, inv, **more)
    for x, dy, dx, w, dw in zip(xs, dys, outs, ws, dws):
        want, ex, want_w, ew = gradients(x, dy, w, pos, inv, off, inter, 0.75, 1e-5, 1.0)
        close(dx, want, ex)
        close(dw, want_w, ew)
    again, dws2 = backward(xs, dys, ws, pos, inv, **more)
    assert all(torch.equal(a, b) for a, b in zip(outs + dws, again + dws2))
    over = [d.clone() for d in dys]
    kv.norm_rope_backward(xs, over, over, ws, None, pos, inv, None, **more)
    assert all(torch.equal(a, b) for a, b in zip(outs, over))
