"""Decode calls that are the first CUDA work of a host thread, on a stream that
another thread made."""
import threading

import pytest
import torch

import quantized_kv_cache_kvarn_gb300 as kv
from tests import serving

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_kv_cache_kvarn_gb300 import build
    build.build()
    kv.lib()


@pytest.mark.parametrize("D,N,widths", [(128, 128, (4, 2, 4)), (128, 64, (4, 2, 4)), (256, 128, (4, 2, 4)),
                                        (128, 128, (6, 6, 2)), (128, 64, (8, 8, 2)), (256, 64, (5, 4, 2))])
def test_the_first_call_of_a_host_thread(D, N, widths):
    prefix = 2 * N
    x = serving.Batch(D, N, 8, 2, [prefix + 5, prefix + N + 1], prefix=prefix, widths=widths, seed=1)
    lay, L, stream = x.layout_of(), int(x.lens.max()), torch.cuda.Stream()
    q, cache, table, own, lens, tk, tv = (t.cuda() for t in (
        x.q, torch.from_numpy(x.cache), torch.from_numpy(x.full_table()), torch.from_numpy(x.prefix_table),
        torch.from_numpy(x.lens), x.tail_k[:, :, :N].contiguous(), x.tail_v[:, :, :N].contiguous()))
    outs = torch.zeros((4, 2, 1, 8, D), device="cuda")
    ws = torch.empty(max(kv.decode_workspace_bytes(lay, 2, 8, L), kv.decode_shared_workspace_bytes(lay, 2, 8, 1, L, prefix)),
                     dtype=torch.uint8, device="cuda")
    err = kv.new_error_word()
    torch.cuda.synchronize()

    def plain(out):
        kv.decode(q[:, 0], lay, cache, table, lens, L, out[:, 0], ws, err, x.sm, tk, tv, stream=stream)

    def shared(out):
        kv.decode_shared(q, lay, cache, own, prefix, table, lens, L, out, ws, err, x.sm, tk, tv, stream=stream)

    failures = []

    def in_thread(call, out):
        def run():
            try:
                call(out)
            except Exception as e:
                failures.append(e)
        t = threading.Thread(target=run)
        t.start()
        t.join()

    for i, call in enumerate((plain, shared)):
        call(outs[2 * i])
        in_thread(call, outs[2 * i + 1])
    stream.synchronize()
    assert not failures, failures
    assert kv.read_error_flags(err) == 0
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[2], outs[3]) and outs[0].any()
