"""Arguments of the serving calls that name the same memory twice, refused by
the C ABI before any launch (fake addresses; no compute call is made)."""
import ctypes

import pytest

import quantized_kv_cache_kvarn_gb300 as kv
from quantized_kv_cache_kvarn_gb300 import build as kvbuild

P = ctypes.c_void_p
A = [P(i << 20) for i in range(1, 12)]
OK, EINVAL = 0, -1


@pytest.fixture(scope="module")
def L():
    kvbuild.build()
    return kv.lib()


def rope(L, pairs, heads=None):
    rows = [kv.RopeTensor(in_=a << 20, out=b << 20, in_seq_stride=384, in_token_stride=128, in_head_stride=128,
                          out_seq_stride=384, out_token_stride=128, out_head_stride=128,
                          num_heads=1 if heads is None else heads[i], head_dim=128) for i, (a, b) in enumerate(pairs)]
    return L.kvarn_rope((kv.RopeTensor * len(rows))(*rows), len(rows), 0, 2, 3, A[9], 3, A[10], 64, 0, 0, 1.0, 0, None)


@pytest.mark.parametrize("pairs", [
    [(1, 1), (1, 1)],            # one tensor turned twice in place
    [(1, 3), (2, 3)],            # two into one
    [(1, 2), (2, 3)],            # one's output is the other's input
    [(2, 3), (1, 2)],
    [(1, 2), (2, 1)],
    [(1, 1), (1, 2)],
    [(1, 2), (3, 4), (5, 4)],
    [(1, 2), (3, 4), (5, 5), (2, 2)],
])
def test_rope_outputs_of_a_call_are_tensors_of_their_own(L, pairs):
    assert rope(L, pairs) == EINVAL


def test_rope_looks_only_at_tensors_with_heads(L):
    assert rope(L, [(1, 1), (1, 1)], heads=(0, 0)) == OK


@pytest.mark.parametrize("lens,lens_out,count", [(A[6], A[7], A[7]), (A[6], A[6], A[6]), (A[6], A[7], A[6])])
def test_eviction_counts_into_a_buffer_of_its_own(L, lens, lens_out, count):
    lay = kv.dense_layout(128, 128, 8, 10)
    assert L.kvarn_evict_tiles(A[0], A[1], 8, A[2], A[3], A[4], 64, lens, lens_out, count, 1024, 2, ctypes.byref(lay), 4, 1, 1, A[8],
                               None) == EINVAL
