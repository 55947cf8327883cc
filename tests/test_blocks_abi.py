"""Refusals of the 8-bit block cache, the norms with rotary positions and the pages' calls, before any launch: by the C
ABI on fake addresses, and by the binding on what the C ABI can not see. No compute call is made here."""
import ctypes
import types

import numpy as np
import pytest
import torch

import quantized_kv_cache_kvarn_gb300 as kv
from quantized_kv_cache_kvarn_gb300 import build as kvbuild
from tests import blocks8 as b8

P = ctypes.c_void_p
BASE = 1 << 30


def at(i, off=0):
    """A fake address of its own."""
    return P(BASE + (i << 20) + off)


OK, EINVAL, EUNSUPPORTED, EALIGN, EWORKSPACE = 0, -1, -2, -3, -5
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    kvbuild.build()
    return kv.lib()


def lay8(**more):
    x = kv.q8_layout(128, 8, 100)
    for k, v in more.items():
        setattr(x, k, v)
    return x


def test_page_bytes(L):
    assert kv.q8_page_bytes(kv.q8_layout(128, 8, 1)) == 4128 == b8.page_bytes(128)
    assert kv.q8_page_bytes(kv.q8_layout(256, 8, 1)) == 8224 == b8.page_bytes(256)
    for bad in (dict(head_dim=64), dict(tile_tokens=32), dict(page_tokens=8), dict(k_bits=4), dict(v_bits=4), dict(rope_dim=64),
                dict(kv_dtype=2), dict(num_kv_heads=0), dict(num_pages=-1)):
        with pytest.raises(kv.KvarnError):
            kv.q8_page_bytes(lay8(**bad))


def test_the_page_format_by_hand():
    """Bytes of a page at places worked out by hand."""
    kb, vb = np.zeros((16, 128), np.uint8), np.zeros((16, 128), np.uint8)
    kb[2, 3], kb[3, 3], kb[3, 70] = 11, 12, 13
    vb[0, 0], vb[1, 0], vb[8, 0], vb[9, 9], vb[6, 33] = 21, 22, 23, 24, 25
    page = b8.pack_page(kb, 0.5, vb, 2.0)
    assert page[2 * 128 + 3] == 11  # an even token's units lie in order
    assert page[3 * 128 + 64 + 3] == 12 and page[3 * 128 + 6] == 13  # an odd token's halves are exchanged
    assert list(page[2048:2051]) == [21, 22, 23]  # lane 0's first word: tokens 0, 1, 8 of channel 0
    assert page[2048 + 16 * 4 + 4 + 3] == 24  # channel 9: block 1, lane 4; token 9: byte 3
    assert page[2048 + 16 * (32 + 4 + 3) + 0] == 25  # channel 33: block 4, lane 4 + 3; token 6: byte 0
    assert page[4096:4104].view(np.float32).tolist() == [0.5, 2.0] and not page[4104:].any()
    k, v = b8.values_of_cache(page[None, None], 128, b8.INT8)
    assert k[0, 0, 2, 3] == 0.5 * (11 - 128) and v[0, 0, 6, 33] == 2.0 * (25 - 128)


def test_codes_by_hand():
    x = np.zeros((16, 128), np.float32)
    x[0, :8] = [254, -254, 1, 3, 5, -1, 2, 0.9]  # int8: steps of 2
    c, s = b8.code_bytes(x, b8.INT8)
    assert s == np.float32(254) * (np.float32(1) / np.float32(127))
    assert c[0, :2].tolist() == [255, 1] and c[0, 6] == 129 and c[1, 0] == 128
    x[0, :8] = [448, -448, 0.0009765625, 0.00098, 17, 19, 18, -17]  # e4m3: scale 1; half the least step is a tie to 0
    c, s = b8.code_bytes(x, b8.E4M3)
    v = b8.byte_values(c, b8.E4M3)[0, :8]
    assert s == np.float32(448) * (np.float32(1) / np.float32(448)) and v.tolist() == [448, -448, 0, 2.0 ** -9, 16, 20, 18, -16]


def blocks(L, call="kvarn_q8_encode_blocks", lay=None, code=0, k=at(1), v=at(2), ss=8192, hs=1024, ts=128, B=1, C=32, start=at(3),
           bt=at(4), bts=4, cache=at(5), err=at(6)):
    lay = lay or lay8()
    return getattr(L, call)(k, v, ss, hs, ts, B, C, start, bt, bts, ctypes.byref(lay), code, cache, err, None)


@pytest.mark.parametrize("call", ["kvarn_q8_encode_blocks", "kvarn_q8_read_blocks"])
@pytest.mark.parametrize("code,kw", [
    (EUNSUPPORTED, dict(code=2)), (EUNSUPPORTED, dict(code=-1)), (EUNSUPPORTED, dict(lay=lay8(head_dim=512))), (EINVAL, dict(C=17)),
    (EINVAL, dict(C=-16)), (EINVAL, dict(B=-1)), (OK, dict(B=0)), (OK, dict(C=0)), (EINVAL, dict(k=None)), (EINVAL, dict(v=None)),
    (EINVAL, dict(start=None)), (EINVAL, dict(bt=None)), (EINVAL, dict(cache=None)), (EINVAL, dict(err=None)), (EINVAL, dict(ss=-8)),
    (EINVAL, dict(hs=-8)), (EINVAL, dict(ts=-8)), (EINVAL, dict(bts=0)), (EALIGN, dict(k=at(1, 8))), (EALIGN, dict(ts=132)),
    (EALIGN, dict(ss=4)), (EALIGN, dict(cache=at(5, 64))), (EALIGN, dict(start=at(3, 2))), (EUNSUPPORTED, dict(B=1 << 30, C=1 << 20)),
])
def test_block_refusals(L, call, code, kw):
    assert blocks(L, call, **kw) == code


def test_read_refuses_one_buffer_for_both(L):
    assert blocks(L, "kvarn_q8_read_blocks", v=at(1)) == EINVAL


def append(L, lay=None, code=0, k=at(1), v=at(2), lens=at(3), n=64, tk=at(4), tv=at(5), cap=16, B=1, bt=at(6), bts=4, cache=at(7), err=at(8)):
    return L.kvarn_q8_append(k, v, lens, n, tk, tv, cap, B, bt, bts, ctypes.byref(lay or lay8()), code, cache, err, None)


@pytest.mark.parametrize("code,kw", [
    (EUNSUPPORTED, dict(code=2)), (EUNSUPPORTED, dict(lay=lay8(tile_tokens=128))), (EINVAL, dict(cap=14)), (EINVAL, dict(bts=3)),
    (EINVAL, dict(n=-1)), (EINVAL, dict(B=-1)), (OK, dict(B=0)), (EINVAL, dict(tk=None)), (EINVAL, dict(tv=at(4))), (EINVAL, dict(lens=None)),
    (EALIGN, dict(tk=at(4, 8))), (EALIGN, dict(cache=at(7, 16))), (EALIGN, dict(lens=at(3, 1))), (EINVAL, dict(err=None)),
])
def test_append_refusals(L, code, kw):
    assert append(L, **kw) == code


def decode(L, lay=None, code=0, q=at(1), Hq=64, Q=1, cache=at(2), bt=at(3), bts=64, lens=at(4), n=1024, tk=at(5), tv=at(6), cap=16,
           W=0, S=0, B=1, out=at(7), lse=at(8), ws=at(9), size=BIG, err=at(10)):
    return L.kvarn_q8_decode(q, Hq, Q, 0.1, cache, ctypes.byref(lay or lay8()), code, bt, bts, lens, n, tk, tv, cap, W, S, B, out, lse, ws,
                             size, err, None)


@pytest.mark.parametrize("code,kw", [
    (EUNSUPPORTED, dict(code=3)), (EUNSUPPORTED, dict(lay=lay8(k_bits=6))), (EINVAL, dict(Hq=63)), (EINVAL, dict(Hq=0)), (EUNSUPPORTED, dict(Hq=72)),
    (EINVAL, dict(Q=0)), (EINVAL, dict(Q=9)), (EINVAL, dict(W=-1)), (EINVAL, dict(S=-1)), (EINVAL, dict(n=-1)), (EINVAL, dict(B=-1)),
    (OK, dict(B=0)), (EINVAL, dict(bts=63)), (EINVAL, dict(cap=14)), (EINVAL, dict(Q=4, cap=17)), (EINVAL, dict(q=None)),
    (EINVAL, dict(cache=None)), (EINVAL, dict(out=None)), (EINVAL, dict(ws=None)), (EINVAL, dict(err=None)), (EINVAL, dict(lens=None)),
    (EALIGN, dict(q=at(1, 8))), (EALIGN, dict(tk=at(5, 4))), (EALIGN, dict(cache=at(2, 32))), (EALIGN, dict(lse=at(8, 2))),
    (EALIGN, dict(ws=at(9, 8))), (EWORKSPACE, dict(size=1000)), (EINVAL, dict(lay=lay8(num_pages=0))), (EUNSUPPORTED, dict(B=1 << 25)),
])
def test_decode_refusals(L, code, kw):
    assert decode(L, **kw) == code


def test_decode_workspace(L):
    lay = lay8()
    assert kv.q8_decode_workspace_bytes(lay, 4, 64, 1, 1000) > 0
    for bad in ((4, 63, 1, 1000), (-1, 64, 1, 1000), (4, 64, 9, 1000), (4, 64, 1, -1), (4, 64, 1, 10, -1), (4, 64, 1, 10, 1, -1)):
        with pytest.raises(kv.KvarnError):
            kv.q8_decode_workspace_bytes(lay, *bad)


def norm(L, n=1, D=128, dtype=0, wdtype=2, B=2, S=3, pos=at(20), inv=at(21), R=64, off=0, inter=0, eps=1e-6, back=False, ws=at(22), size=BIG,
         tensors=True, second=None, **t):
    one = dict(x=BASE + (1 << 20), dy=BASE + (2 << 20), out=BASE + (3 << 20), weight=BASE + (4 << 20), dweight=BASE + (5 << 20),
               num_heads=1, **{f"{s}_{a}_stride": d for s in ("x", "dy", "out") for a, d in (("seq", 384), ("token", 128), ("head", 128))})
    one.update(t)
    two = {**one, "x": BASE + (6 << 20), "dy": BASE + (7 << 20), "out": BASE + (8 << 20), "dweight": BASE + (9 << 20), **(second or {})}
    arr = (kv.NormRopeTensor * 8)(kv.NormRopeTensor(**one), *[kv.NormRopeTensor(**two) for _ in range(7)]) if tensors else None
    head = (arr, n, D, dtype, wdtype, B, S, pos, 3, inv, R, off, inter, 1.0, eps, 0.0)
    return L.kvarn_norm_rope_backward(*head, ws, size, None) if back else L.kvarn_norm_rope(*head, None)


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("code,kw", [
    (EINVAL, dict(tensors=False)), (EINVAL, dict(n=0)), (EINVAL, dict(n=5)), (EINVAL, dict(D=0)), (EUNSUPPORTED, dict(D=1026)),
    (EUNSUPPORTED, dict(dtype=3)), (EUNSUPPORTED, dict(wdtype=-1)), (EINVAL, dict(R=63)), (EINVAL, dict(R=-2)), (EINVAL, dict(R=130)),
    (EINVAL, dict(off=65)), (EINVAL, dict(off=-1)), (EINVAL, dict(inter=2)), (EINVAL, dict(eps=-1.0)), (EINVAL, dict(eps=float("nan"))),
    (EINVAL, dict(B=-1)), (EINVAL, dict(pos=None)), (EINVAL, dict(inv=None)), (EALIGN, dict(pos=at(20, 2))), (EALIGN, dict(inv=at(21, 4))),
    (EINVAL, dict(x=None)), (EINVAL, dict(out=None)), (EALIGN, dict(x=BASE + 1)), (EALIGN, dict(weight=BASE + 2)), (EINVAL, dict(num_heads=-1)),
    (EUNSUPPORTED, dict(num_heads=(1 << 20) + 1)), (EUNSUPPORTED, dict(B=1 << 20, S=1 << 20)),
    (EINVAL, dict(out=BASE + (1 << 20), out_token_stride=64)), (EINVAL, dict(out=BASE + (4 << 20))),
    (EINVAL, dict(n=2, second=dict(out=BASE + (3 << 20)))), (EINVAL, dict(n=2, second=dict(out=BASE + (1 << 20)))),
    (EINVAL, dict(n=2, second=dict(x=BASE + (3 << 20)))),
])
def test_norm_refusals(L, code, kw, back):
    assert norm(L, back=back, **kw) == code


@pytest.mark.parametrize("code,kw", [
    (EINVAL, dict(dy=None)), (EINVAL, dict(ws=None)), (EALIGN, dict(ws=at(22, 8))), (EWORKSPACE, dict(size=3)), (EALIGN, dict(dweight=BASE + 2)),
    (EINVAL, dict(out=BASE + (2 << 20), out_head_stride=256, num_heads=2)), (EINVAL, dict(dweight=BASE + (4 << 20))),
    (EINVAL, dict(n=2, second=dict(dweight=BASE + (5 << 20)))), (EINVAL, dict(n=2, second=dict(dy=BASE + (3 << 20)))),
    (EINVAL, dict(n=2, second=dict(weight=BASE + (5 << 20)))), (EINVAL, dict(dweight=BASE + (1 << 20))), (EINVAL, dict(dweight=BASE + (2 << 20))),
    (EINVAL, dict(n=2, second=dict(dweight=BASE + (3 << 20)))), (EINVAL, dict(n=2, second=dict(x=BASE + (5 << 20)))),
    (EINVAL, dict(n=2, second=dict(weight=BASE + (3 << 20)))),
])
def test_norm_backward_refusals(L, code, kw):
    assert norm(L, back=True, **kw) == code


def test_norm_of_nothing(L):
    assert norm(L, B=0) == OK and norm(L, S=0) == OK and norm(L, num_heads=0) == OK
    assert norm(L, B=0, back=True, dweight=None) == OK


def test_norm_workspace(L):
    x = torch.empty((2, 3, 4, 128))
    assert kv.norm_rope_backward_workspace_bytes([x, x]) >= 2 * 128 * 4 and kv.norm_rope_backward_workspace_bytes(x[:0]) == 0
    for bad in ([x] * 5, torch.empty((2, 3, 4)), torch.empty((1, 1, 1, 2000))):
        with pytest.raises(kv.KvarnError):
            kv.norm_rope_backward_workspace_bytes(bad)


def fork(L, parents=at(1), n_in=2, n_out=2, lens=at(2), lens_out=at(3), n=64, bt=at(4), bt_out=at(5), bts=4, refs=at(6), refs_out=at(7),
         freed=at(8), count=at(9), tails=1, lay=None, recent=0, W=0, S=0, err=at(10), **t):
    one = dict(in_=BASE + (11 << 20), out=BASE + (12 << 20), row_bytes=256, num_heads=2, capacity=16, whole=0)
    one.update(t)
    arr = (kv.ForkTail * 5)(*[kv.ForkTail(**{**one, "out": one["out"] and one["out"] + (k << 21), "in_": one["in_"] and one["in_"] + (k << 21)})
                              for k in range(5)])
    return L.kvarn_fork_sequences(parents, n_in, n_out, lens, lens_out, n, bt, bt_out, bts, refs, refs_out, freed, count, arr, tails,
                                  ctypes.byref(lay or lay8()), recent, W, S, err, None)


@pytest.mark.parametrize("code,kw", [
    (EUNSUPPORTED, dict(lay=lay8(page_tokens=32))), (EUNSUPPORTED, dict(lay=lay8(tile_tokens=24))), (EUNSUPPORTED, dict(lay=lay8(tile_tokens=8))),
    (EINVAL, dict(lay=lay8(num_pages=-1))), (EUNSUPPORTED, dict(lay=lay8(num_pages=(1 << 23) + 1))), (EINVAL, dict(n_in=-1)),
    (EINVAL, dict(n_out=-1)), (EUNSUPPORTED, dict(n_in=32769)), (EUNSUPPORTED, dict(n_out=32769)), (EINVAL, dict(n=-1)),
    (EINVAL, dict(recent=-1)), (EINVAL, dict(W=-1)), (EINVAL, dict(S=-1)), (EINVAL, dict(bts=3)), (EINVAL, dict(parents=None)),
    (EINVAL, dict(lens=None)), (EINVAL, dict(lens_out=None)), (EINVAL, dict(bt=None)), (EINVAL, dict(bt_out=None)), (EINVAL, dict(refs=None)),
    (EINVAL, dict(refs_out=None)), (EINVAL, dict(freed=None)), (EINVAL, dict(count=None)), (EINVAL, dict(err=None)),
    (EALIGN, dict(parents=at(1, 2))), (EALIGN, dict(freed=at(8, 1))), (EINVAL, dict(bt_out=at(4))), (EINVAL, dict(lens_out=at(2))),
    (EINVAL, dict(freed=at(6))), (EINVAL, dict(freed=at(7))), (EINVAL, dict(count=at(8))), (EINVAL, dict(refs_out=at(2))),
    (EUNSUPPORTED, dict(tails=5)), (EINVAL, dict(tails=-1)), (EINVAL, dict(in_=None)), (EINVAL, dict(out=None)), (EALIGN, dict(row_bytes=24)),
    (EINVAL, dict(row_bytes=-16)), (EINVAL, dict(whole=2)), (EINVAL, dict(out=BASE + (11 << 20))), (EALIGN, dict(out=BASE + 8)),
    (EINVAL, dict(tails=2, out=BASE + (13 << 20))),  # the first tail's new rows are the second's old ones
    (EUNSUPPORTED, dict(num_heads=(1 << 20) + 1)),
])
def test_fork_refusals(L, code, kw):
    assert fork(L, **kw) == code


def compact(L, cache=at(1), stride=4128, pages=100, refs=at(2), refs_out=at(3), bt=at(4), bt_out=at(5), rows=2, entries=4, bts=4, remap=at(6),
            live=at(7), ws=at(8), size=BIG, err=at(9)):
    return L.kvarn_compact_pages(cache, stride, pages, refs, refs_out, bt, bt_out, rows, entries, bts, remap, live, ws, size, err, None)


@pytest.mark.parametrize("code,kw", [
    (EINVAL, dict(cache=None)), (EINVAL, dict(stride=0)), (EALIGN, dict(stride=24)), (EINVAL, dict(pages=-1)), (EUNSUPPORTED, dict(pages=(1 << 30) + 1)),
    (EINVAL, dict(refs=None)), (EINVAL, dict(refs_out=None)), (EINVAL, dict(bt=None)), (EINVAL, dict(bt_out=None)), (EINVAL, dict(rows=-1)),
    (EINVAL, dict(entries=-1)), (EINVAL, dict(bts=3)), (EINVAL, dict(remap=None)), (EINVAL, dict(live=None)), (EINVAL, dict(ws=None)),
    (EINVAL, dict(err=None)), (EALIGN, dict(cache=at(1, 8))), (EALIGN, dict(refs=at(2, 2))), (EALIGN, dict(ws=at(8, 8))), (EINVAL, dict(remap=at(2))),
    (EINVAL, dict(remap=at(5))), (EINVAL, dict(live=at(9))), (EINVAL, dict(bt_out=at(2))), (EINVAL, dict(refs_out=at(4))), (EWORKSPACE, dict(size=100)),
])
def test_compact_refusals(L, code, kw):
    assert compact(L, **kw) == code


# ------------------------------------------------------------------ the binding
@pytest.fixture
def calls(monkeypatch):
    """Names of the C entries that the binding has called, the library and the GPU replaced by fakes."""
    kvbuild.build()
    real, made = kv.lib(), []

    def entry(name):
        def call(*args):
            made.append(name)
            return 0
        return call

    names = ("kvarn_q8_encode_blocks", "kvarn_q8_read_blocks", "kvarn_q8_append", "kvarn_q8_decode", "kvarn_norm_rope",
             "kvarn_norm_rope_backward", "kvarn_fork_sequences", "kvarn_compact_pages")
    fake = types.SimpleNamespace(**{n: entry(n) for n in names}, kvarn_q8_page_bytes=real.kvarn_q8_page_bytes,
                                 kvarn_status_string=real.kvarn_status_string)
    monkeypatch.setattr(kv, "lib", lambda: fake)
    monkeypatch.setattr(kv, "_device_of", lambda what, *tensors: 0)
    monkeypatch.setattr(kv, "_raw_stream", lambda what, stream, dev: 0)
    return made


H16, I32 = torch.float16, torch.int32


def refused(made, call, *args, **more):
    before = len(made)
    with pytest.raises(kv.KvarnError):
        call(*args, **more)
    assert len(made) == before


def test_binding_of_blocks(calls):
    lay, err = kv.q8_layout(128, 2, 4), torch.zeros(1, dtype=I32)
    cache, start, table = torch.zeros(4 * 2 * 4128, dtype=torch.uint8), torch.zeros(3, dtype=I32), torch.zeros((3, 5), dtype=I32)
    k, v = torch.zeros((3, 2, 32, 128), dtype=H16), torch.zeros((3, 2, 32, 128), dtype=H16)
    for f in (kv.q8_encode_blocks, kv.q8_read_blocks):
        f(k, v, lay, 0, start, table, cache, err)
        f(k.transpose(1, 2).contiguous().transpose(1, 2), v.transpose(1, 2).contiguous().transpose(1, 2), lay, 0, start, table, cache, err)
        for bad in ((k.float(), v.float()), (k[:, :1], v[:, :1]), (k[..., :64], v[..., :64]), (k, v.transpose(1, 2).contiguous().transpose(1, 2)),
                    (k[0], v[0]), (k, v[:2])):
            refused(calls, f, *bad, lay, 0, start, table, cache, err)
        refused(calls, f, k, v, lay, 0, start.long(), table, cache, err)
        refused(calls, f, k, v, lay, 0, start, table[:, :3], cache, err)  # entries between the rows are nobody's
        refused(calls, f, k, v, lay, 0, start, table[:2], cache, err)
        refused(calls, f, k, v, lay, 0, start, table, cache[:-1], err)
        refused(calls, f, k, v, lay, 0, start, table, cache, torch.zeros(2, dtype=I32))
    one = torch.zeros((1, 2, 32, 128), dtype=H16)
    kv.q8_encode_blocks(one.expand(3, -1, -1, -1), one.expand(3, -1, -1, -1), lay, 0, start, table, cache, err)
    refused(calls, kv.q8_read_blocks, one.expand(3, -1, -1, -1), one.expand(3, -1, -1, -1), lay, 0, start, table, cache, err)
    assert calls == ["kvarn_q8_encode_blocks"] * 2 + ["kvarn_q8_read_blocks"] * 2 + ["kvarn_q8_encode_blocks"]


def test_binding_of_append_and_decode(calls):
    lay, err, cache = kv.q8_layout(128, 2, 4), torch.zeros(1, dtype=I32), torch.zeros(4 * 2 * 4128, dtype=torch.uint8)
    k, tail, lens, table = (torch.zeros((3, 2, 128), dtype=H16), torch.zeros((3, 2, 16, 128), dtype=H16), torch.zeros(3, dtype=I32),
                            torch.zeros((3, 5), dtype=I32))
    kv.q8_append(k, k, lay, 0, lens, 80, tail, tail.clone(), table, cache, err)
    refused(calls, kv.q8_append, k, k, lay, 0, lens, 96, tail, tail, table, cache, err)
    refused(calls, kv.q8_append, k, k.bfloat16(), lay, 0, lens, 80, tail, tail, table, cache, err)
    refused(calls, kv.q8_append, k, k, lay, 0, lens, 80, tail, tail[:, :, :15], table, cache, err)
    refused(calls, kv.q8_append, k[:2], k, lay, 0, lens, 80, tail, tail, table, cache, err)
    q, out, lse, ws = torch.zeros((3, 1, 8, 128), dtype=H16), torch.zeros((3, 1, 8, 128)), torch.zeros((3, 1, 8)), torch.zeros(8)
    kv.q8_decode(q, lay, 0, cache, table, lens, 80, out, ws, err, 0.1, tail, tail, lse, window=5)
    kv.q8_decode(q, lay, 0, cache, table, lens, 80, out, ws, err, 0.1)
    for change in (dict(q=q[:, 0]), dict(q=q.float()), dict(out=out[:, :, :4]), dict(lse=lse[:2]), dict(n=96), dict(tk=None), dict(tv=tail[:2]),
                   dict(table=table.long()), dict(lens=lens[:2]), dict(cache=cache[1:])):
        a = dict(q=q, cache=cache, table=table, lens=lens, n=80, out=out, tk=tail, tv=tail, lse=lse)
        a.update(change)
        refused(calls, kv.q8_decode, a["q"], lay, 0, a["cache"], a["table"], a["lens"], a["n"], a["out"], ws, err, 0.1, a["tk"], a["tv"], a["lse"])
    assert calls == ["kvarn_q8_append", "kvarn_q8_decode", "kvarn_q8_decode"]


def test_binding_of_norms(calls):
    x, w, pos, inv = torch.zeros((2, 3, 4, 128), dtype=H16), torch.zeros(128), torch.zeros((2, 3), dtype=I32), torch.zeros(64, dtype=torch.float64)
    kv.norm_rope(x, x.clone(), w, pos, inv)
    kv.norm_rope([x, x[:, :, :1]], [x.clone(), x[:, :, :1].clone()], [w, None], pos[:1], inv)
    kv.norm_rope(x, x.clone(), None, None, None)
    dw, ws = torch.zeros(128), torch.zeros(64)
    kv.norm_rope_backward(x, x.clone(), x.clone(), w, dw, pos, inv, ws)
    for change in (dict(x=x.double()), dict(x=x[0]), dict(y=x[:1].clone()), dict(y=x.float()), dict(y=x[:1].expand(2, -1, -1, -1)), dict(w=w[:64]),
                   dict(w=w.double()), dict(pos=pos.long()), dict(pos=pos[:, :2]), dict(inv=inv.float()), dict(x=x.transpose(2, 3)),
                   dict(x=[x] * 5, y=[x] * 5, w=[w] * 5)):
        a = dict(x=x, y=x.clone(), w=w, pos=pos, inv=inv)
        a.update(change)
        refused(calls, kv.norm_rope, a["x"], a["y"], a["w"], a["pos"], a["inv"])
    for change in (dict(dy=x[:1]), dict(dy=x.float()), dict(dw=dw[:64]), dict(dw=dw.half()), dict(dy=None), dict(ws=torch.zeros(64)[::2])):
        a = dict(dy=x.clone(), dw=dw, ws=ws)
        a.update(change)
        refused(calls, kv.norm_rope_backward, x, a["dy"], x.clone(), w, a["dw"], pos, inv, a["ws"])
    refused(calls, kv.norm_rope, [x, x], [x.clone(), x.clone()], [w, w.half()], pos, inv)
    assert calls == ["kvarn_norm_rope"] * 3 + ["kvarn_norm_rope_backward"]


def test_binding_of_pages(calls):
    lay, err = kv.q8_layout(128, 2, 10), torch.zeros(1, dtype=I32)
    i = lambda *s: torch.zeros(s, dtype=I32)  # noqa: E731
    good = dict(parents=i(3), lens=i(2), table=i(2, 4), refs=i(10), n=64, lens_out=i(3), table_out=i(3, 4), refs_out=i(10), freed=i(10), count=i(1),
                tails=((torch.zeros((2, 2, 16, 128), dtype=H16), torch.zeros((3, 2, 16, 128), dtype=H16)),))

    def call(**change):
        a = {**good, **change}
        kv.fork_sequences(a["parents"], a["lens"], a["table"], a["refs"], lay, a["n"], a["lens_out"], a["table_out"], a["refs_out"], a["freed"],
                          a["count"], err, tails=a["tails"])

    call()
    t = good["tails"][0]
    for change in (dict(n=80), dict(parents=i(3).long()), dict(lens_out=i(2)), dict(table_out=i(2, 4)), dict(table_out=i(3, 5)), dict(refs=i(9)),
                   dict(freed=i(11)), dict(count=i(2)), dict(tails=((t[0], t[1][:2]),)), dict(tails=((t[0], t[1].float()),)),
                   dict(tails=((t[0], t[1][:, :, :8]),)), dict(tails=(t,) * 5), dict(tails=((t[0][0], t[1][0]),))):
        refused(calls, call, **change)
    cache, ws = torch.zeros((10, 2, 64), dtype=torch.uint8), torch.zeros(64)
    kv.compact_pages(cache, i(10), i(2, 3), i(10), i(2, 3), i(10), i(1), ws, err)
    kv.compact_pages(cache, i(10), None, i(10), None, i(10), i(1), ws, err)
    for args in ((cache.int(), i(10), i(2, 3), i(10), i(2, 3), i(10), i(1)), (cache[:, :1], i(10), i(2, 3), i(10), i(2, 3), i(10), i(1)),
                 (cache, i(9), i(2, 3), i(10), i(2, 3), i(10), i(1)), (cache, i(10), i(2, 3), i(10), None, i(10), i(1)),
                 (cache, i(10), i(2, 3), i(10), i(2, 4), i(10), i(1)), (cache, i(10), i(2, 3), i(10), i(2, 3), i(9), i(1)),
                 (cache, i(10), i(2, 3), i(10), i(2, 3), i(10), i(2))):
        refused(calls, kv.compact_pages, *args, ws, err)
    assert calls == ["kvarn_fork_sequences", "kvarn_compact_pages", "kvarn_compact_pages"]


def test_norm_gradient_of_more_heads_than_a_grid_holds(L):
    """The weights' gradient adds up at most 128 heads of a group in a row, so that tokens times heads are limited."""
    most = dict(B=1 << 20, S=1 << 10, D=8, R=0, num_heads=1 << 20)
    assert norm(L, back=True, **most) == EUNSUPPORTED
    heads = (ctypes.c_int32 * 1)(1 << 20)
    assert L.kvarn_norm_rope_backward_workspace_bytes(heads, 1, 8, 1 << 20, 1 << 10) == -1
    assert L.kvarn_norm_rope_backward_workspace_bytes(heads, 1, 8, 1, 64) > 0
