"""Calls of kvarn_decode_shared from several host threads at once, on caches of
different layouts, each with its own stream, buffers and workspace."""
import ctypes
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


class Caller(threading.Thread):
    def __init__(self, N, widths, calls, start):
        super().__init__()
        x = serving.Batch(128, N, 8, 1, [8192 + 3] * 61, Q=2, prefix=8192, widths=widths, seed=N)
        self.lay, self.sm, self.calls, self.begin, self.failure = x.layout_of(), x.sm, calls, start, None
        self.stream = torch.cuda.Stream()
        with torch.cuda.stream(self.stream):
            self.args = [t.cuda() for t in (x.q, torch.from_numpy(x.cache), torch.from_numpy(x.prefix_table),
                                            torch.from_numpy(x.bt), torch.from_numpy(x.lens), x.tail_k, x.tail_v)]
            self.out = torch.empty((61, 2, 8, 128), device="cuda")
            n = kv.decode_shared_workspace_bytes(self.lay, 61, 8, 2, 8195, 8192)
            self.ws, self.err = torch.empty(n, dtype=torch.uint8, device="cuda"), kv.new_error_word()
        self.stream.synchronize()

        # the C entry itself, so that the threads spend most of their time in it
        p, i, f = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float
        q, cache, prefix, bt, lens, tk, tv = (p(t.data_ptr()) for t in self.args)
        self.row = (q, i(8), i(2), f(self.sm), cache, ctypes.byref(self.lay), prefix, i(8192), bt, i(self.args[3].shape[1]), lens,
                    i(8195), tk, tv, i(self.args[5].shape[2]), i(61), p(self.out.data_ptr()), None, p(self.ws.data_ptr()),
                    ctypes.c_int64(n), p(self.err.data_ptr()), p(self.stream.cuda_stream))

    def call(self):
        return kv.lib().kvarn_decode_shared(*self.row)

    def run(self):
        entry, row = kv.lib().kvarn_decode_shared, self.row
        self.begin.wait()
        for i in range(self.calls):
            code = entry(*row)
            if code:
                self.failure = (i, code)
                return
            if i % 64 == 63:
                self.stream.synchronize()


def test_threads_with_caches_of_different_layouts():
    layouts = [(128, (4, 2, 4)), (64, (4, 2, 4)), (128, (8, 8, 2)), (64, (2, 2, 2))]
    start = threading.Barrier(len(layouts))
    callers = [Caller(N, widths, 6000, start) for N, widths in layouts]
    want = []
    for c in callers:
        assert c.call() == 0
        c.stream.synchronize()
        assert kv.read_error_flags(c.err) == 0
        want.append(c.out.clone())
        c.out.fill_(float("nan"))
    torch.cuda.synchronize()
    for c in callers:
        c.start()
    for c in callers:
        c.join()
    torch.cuda.synchronize()
    for c, w in zip(callers, want):
        assert c.failure is None, c.failure
        assert kv.read_error_flags(c.err) == 0
        assert torch.equal(c.out, w)
