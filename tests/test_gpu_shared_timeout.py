"""The bounded waits of the tensor-core kernel over a shared prefix, driven as
those of the dense decode are (kvarn_set_copy_wait_test): with copies announced
larger than they are, so that none completes, and with limits so short that a
wait of any role runs out anywhere in the run while the copies land as usual.
The call flags KVARN_DEVERR_TIMEOUT and returns; the next one is right."""
import time

import pytest
import torch

import quantized_kv_cache_kvarn_gb300 as kv
from tests import parity, serving

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_kv_cache_kvarn_gb300 import build
    build.build()
    kv.lib()


class Call:
    """A call whose prefix goes to the tensor-core kernel (61 sequences: 122
    rows of eight, 4096 tokens), without tiles of its own (own below 64), so
    that no other kernel waits for a copy; or to the dense kernel (4)."""

    def __init__(self, own=3, sequences=61, dim=128):
        B = sequences
        x = serving.Batch(dim, 64, 8, 1, [4096 + own] * B, Q=2, prefix=4096, seed=4)
        self.lay, self.n = x.layout_of(), int(x.lens.max())
        self.cache, self.prefix, self.bt, self.lens, self.q, self.tk, self.tv = (
            t.cuda() for t in (torch.from_numpy(x.cache), torch.from_numpy(x.prefix_table), torch.from_numpy(x.bt),
                               torch.from_numpy(x.lens), x.q, x.tail_k, x.tail_v))
        self.sm = x.sm
        self.out = torch.empty((B, 2, 8, dim), device="cuda")
        self.ws = torch.empty(kv.decode_shared_workspace_bytes(self.lay, B, 8, 2, self.n, 4096), dtype=torch.uint8,
                              device="cuda")
        self.err = kv.new_error_word()

    def __call__(self):
        """(output, error word, seconds)"""
        self.err.zero_()
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        kv.decode_shared(self.q, self.lay, self.cache, self.prefix, 4096, self.bt, self.lens, self.n, self.out, self.ws,
                         self.err, self.sm, self.tk, self.tv)
        torch.cuda.synchronize()
        took = time.perf_counter() - t0
        return self.out.clone(), kv.read_error_flags(self.err), took


@pytest.mark.parametrize("own,sequences,dim", [(3, 61, 128), (70, 61, 128), (70, 4, 128), (3, 4, 256), (150, 4, 256)])
def test_copies_that_never_complete(own, sequences, dim):
    call = Call(own, sequences, dim)
    want, flags, _ = call()
    assert flags == 0
    for cycles in (1_000_000, 50_000):
        kv.set_copy_wait_test(cycles, withhold=True)
        try:
            _, flags, took = call()
        finally:
            kv.set_copy_wait_test(0, withhold=False)
        parity.report(f"shared-prefix time-out ({sequences} x {own} own tokens, head_dim {dim}, {cycles} cycles): error word "
                      f"{flags:#x} after {took * 1e3:.0f} ms")
        assert flags == kv.DEVERR_TIMEOUT
        assert took < 1.0  # the limit, 50 ms for the copies under way, launches
        got, flags, _ = call()
        assert flags == 0 and torch.equal(got, want)


def test_waits_that_run_out_anywhere():
    call = Call()
    want, flags, _ = call()
    assert flags == 0
    gave_up = 0
    for k in range(120):
        kv.set_copy_wait_test(1 + 37 * (k % 40) ** 2, withhold=False)  # 1 to 56,000 cycles; the whole run takes about 40,000
        try:
            got, flags, took = call()
        finally:
            kv.set_copy_wait_test(0, withhold=False)
        assert flags in (0, kv.DEVERR_TIMEOUT) and took < 1.0
        if flags:
            gave_up += 1
        else:
            assert torch.equal(got, want)
        if k % 10 == 0:
            got, flags, _ = call()
            assert flags == 0 and torch.equal(got, want)
    parity.report(f"shared-prefix waits of 1 to 56,000 cycles: {gave_up} of 120 calls gave up")
    assert 0 < gave_up < 120
