"""What the binding of the serving calls refuses and lets through, with the
library and the GPU replaced by fakes: the tensors here are on the CPU and no
call reaches the C ABI."""
import types

import pytest
import torch

import quantized_kv_cache_kvarn_gb300 as kv
from quantized_kv_cache_kvarn_gb300 import build


@pytest.fixture
def calls(monkeypatch):
    """Names of the C entries that the binding has called."""
    build.build()
    real, made = kv.lib(), []

    def entry(name):
        def call(*args):
            made.append(name)
            return 0
        return call

    fake = types.SimpleNamespace(**{n: entry(n) for n in ("kvarn_decode_mass", "kvarn_decode_shared", "kvarn_evict_tiles",
                                                          "kvarn_rope")},
                                 kvarn_page_bytes=real.kvarn_page_bytes, kvarn_status_string=real.kvarn_status_string)
    monkeypatch.setattr(kv, "lib", lambda: fake)
    monkeypatch.setattr(kv, "_device_of", lambda what, *tensors: 0)
    monkeypatch.setattr(kv, "_raw_stream", lambda what, stream, dev: 0)
    return made


def table(rows, columns, stride=None):
    """int32 [rows, columns], rows `stride` apart, at the end of its storage."""
    stride = stride or columns
    return torch.zeros((rows - 1) * stride + columns, dtype=torch.int32).as_strided((rows, columns), (stride, 1))


def decode_mass(block_table, longest):
    B, N = block_table.shape[0], 128
    lay = kv.dense_layout(128, N, 1, 8)
    q, out = torch.zeros((B, 4, 128), dtype=torch.float16), torch.zeros((B, 4, 128))
    mass = torch.zeros((B, max(1, longest // N)))
    kv.decode_mass(q, lay, torch.zeros(8 * kv.page_bytes(lay), dtype=torch.uint8), block_table, torch.zeros(B, dtype=torch.int32),
                   longest, out, mass, mass, torch.zeros(16, dtype=torch.uint8), torch.zeros(1, dtype=torch.int32), 0.1)


def decode_shared(block_table, longest, prefix=128, Q=1):
    B = block_table.shape[0]
    lay = kv.dense_layout(128, 128, 1, 8)
    q, out = torch.zeros((B, Q, 4, 128), dtype=torch.float16), torch.zeros((B, Q, 4, 128))
    kv.decode_shared(q, lay, torch.zeros(8 * kv.page_bytes(lay), dtype=torch.uint8), torch.zeros(prefix // 16, dtype=torch.int32),
                     prefix, block_table, torch.zeros(B, dtype=torch.int32), longest, out, torch.zeros(16, dtype=torch.uint8),
                     torch.zeros(1, dtype=torch.int32), 0.1)


@pytest.mark.parametrize("rows,columns,stride,longest,ok", [
    (2, 16, 16, 256, True), (2, 16, 40, 256, True), (2, 16, 40, 383, True), (1, 16, 16, 256, True),
    (2, 15, 40, 256, False), (2, 16, 40, 384, False), (3, 8, 24, 384, False), (1, 8, 8, 256, False),
])
def test_block_tables_hold_every_committed_page(calls, rows, columns, stride, longest, ok):
    for call in (decode_mass, decode_shared):
        if ok:
            call(table(rows, columns, stride), longest)
        else:
            with pytest.raises(kv.KvarnError, match="block_table"):
                call(table(rows, columns, stride), longest)
    assert calls == (["kvarn_decode_mass", "kvarn_decode_shared"] if ok else [])


def test_block_tables_of_a_prefix_and_queries(calls):
    decode_shared(table(2, 1, 4), 255)                    # no tile but the prefix's: the table is not read
    decode_shared(table(2, 8, 40), 258, prefix=128, Q=4)  # 255 tokens before the queries: one tile
    decode_shared(table(2, 16, 40), 259, prefix=128, Q=4)
    with pytest.raises(kv.KvarnError, match="block_table"):
        decode_shared(table(2, 15, 40), 259, prefix=128, Q=4)
    assert len(calls) == 3


def evict(mass_in, mass_out, block_table, table_out, freed):
    B = mass_in.shape[0]
    ints = [torch.zeros(B, dtype=torch.int32) for _ in range(3)]
    kv.evict_tiles(mass_in, block_table, ints[0], kv.dense_layout(128, 128, 1, 8), 256, 1, mass_out, table_out, ints[1], freed,
                   ints[2], torch.zeros(1, dtype=torch.int32))


def mass(rows, columns, stride=None):
    return table(rows, columns, stride).view(torch.float32)


def test_eviction_of_one_row_takes_any_distance_of_rows(calls):
    evict(mass(1, 2, 9), mass(1, 2, 2), table(1, 16, 99), table(1, 16), table(1, 16, 50))
    evict(mass(1, 2), mass(1, 2, 7), table(1, 16), table(1, 16, 40), table(1, 16))
    assert len(calls) == 2


@pytest.mark.parametrize("which", ["mass_out", "block_table_out", "freed"])
def test_eviction_of_several_rows_takes_one_distance(calls, which):
    made = dict(mass_out=mass(2, 2, 9), block_table_out=table(2, 16, 99), freed=table(2, 16, 99))
    evict(mass(2, 2, 9), made["mass_out"], table(2, 16, 99), made["block_table_out"], made["freed"])
    made[which] = mass(2, 2, 8) if which == "mass_out" else table(2, 16, 98)
    with pytest.raises(kv.KvarnError, match=which):
        evict(mass(2, 2, 9), made["mass_out"], table(2, 16, 99), made["block_table_out"], made["freed"])
    made[which] = (mass if which == "mass_out" else table)(2, 16 if which != "mass_out" else 2, 99)[:, ::2]
    with pytest.raises(kv.KvarnError, match=which):
        evict(mass(2, 2, 9), made["mass_out"], table(2, 16, 99), made["block_table_out"], made["freed"])
    assert len(calls) == 1


@pytest.mark.parametrize("base", [1.0, 0.5])
def test_yarn_needs_frequencies_that_fall(base):
    with pytest.raises(kv.KvarnError, match="base"):
        kv.rope_frequencies(64, base, yarn=(2.0, 4096), device="cpu")
