"""Rotary positions where an axis has length one: its stride says nothing,
neither for turning in place nor for the vector path."""
import pytest
import torch

import quantized_kv_cache_kvarn_gb300 as kv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_kv_cache_kvarn_gb300 import build
    build.build()
    kv.lib()


@pytest.mark.parametrize("shape", [(1, 5, 3, 128), (4, 1, 3, 128), (4, 5, 1, 128), (1, 1, 3, 128), (1, 1, 1, 64)])
def test_strides_of_axes_of_length_one(shape):
    g = torch.Generator().manual_seed(1)
    x = torch.randn(shape, generator=g).half().cuda()
    pos = torch.randint(0, 5000, shape[:2], generator=g).to(torch.int32).cuda()
    inv_freq, _ = kv.rope_frequencies(64)
    want = torch.empty_like(x)
    kv.rope(x, want, pos, inv_freq)
    strides = [7 if n == 1 else s for n, s in zip(shape, x.stride())]  # odd: no multiple of 16 bytes
    odd = torch.empty_like(x).as_strided(shape, strides)
    kv.rope(x, odd, pos, inv_freq)
    same = x.clone()
    kv.rope(same.as_strided(shape, strides), same, pos, inv_freq)
    torch.cuda.synchronize()
    assert torch.equal(odd, want) and torch.equal(same, want)
