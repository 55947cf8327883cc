"""Refusals of the serving calls (rotary positions, shared prefix, tile masses,
eviction), before any launch: by the C ABI on fake addresses, and by the
binding on what the C ABI can not see. No compute call is made here."""
import ctypes

import pytest
import torch

import quantized_kv_cache_kvarn_gb300 as kv
from quantized_kv_cache_kvarn_gb300 import build as kvbuild

P = ctypes.c_void_p
A16, BAD = P(1 << 20), P((1 << 20) + 2)
OK, EINVAL, EUNSUPPORTED, EALIGN, EWORKSPACE = 0, -1, -2, -3, -5
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    kvbuild.build()
    return kv.lib()


def rope(L, n=1, dtype=0, B=2, S=3, pos=A16, inv=A16, R=64, off=0, inter=0, inverse=0, tensors=True, **t):
    one = dict(in_=1 << 20, out=1 << 21, in_seq_stride=384, in_token_stride=128, in_head_stride=128, out_seq_stride=384,
               out_token_stride=128, out_head_stride=128, num_heads=1, head_dim=128)
    one.update(t)
    arr = (kv.RopeTensor * 8)(*[kv.RopeTensor(**one) for _ in range(8)])
    return L.kvarn_rope(arr if tensors else None, n, dtype, B, S, pos, 3, inv, R, off, inter, 1.0, inverse, None)


@pytest.mark.parametrize("code,kw", [
    (EINVAL, dict(tensors=False)), (EINVAL, dict(n=0)), (EINVAL, dict(n=5)), (EUNSUPPORTED, dict(dtype=3)),
    (EUNSUPPORTED, dict(dtype=-1)), (EINVAL, dict(R=63)), (EINVAL, dict(R=0)), (EINVAL, dict(R=130)),
    (EINVAL, dict(R=64, off=65)), (EINVAL, dict(off=-1)), (EINVAL, dict(B=-1)), (EINVAL, dict(S=-1)),
    (EINVAL, dict(pos=None)), (EINVAL, dict(inv=None)), (EALIGN, dict(pos=BAD)), (EALIGN, dict(inv=BAD)),
    (EINVAL, dict(inter=2)), (EINVAL, dict(inverse=-1)), (EINVAL, dict(in_=None)), (EINVAL, dict(out=None)),
    (EALIGN, dict(in_=(1 << 20) + 1)), (EALIGN, dict(dtype=2, out=(1 << 20) + 2)),
    (EINVAL, dict(out=1 << 20, out_token_stride=64)),  # in place with other strides
    (EINVAL, dict(num_heads=-1)), (EINVAL, dict(head_dim=0)), (EUNSUPPORTED, dict(head_dim=1026)),
    (EUNSUPPORTED, dict(num_heads=(1 << 20) + 1)), (EUNSUPPORTED, dict(B=1 << 20, S=1 << 20)),
    (OK, dict(B=0)), (OK, dict(S=0)), (OK, dict(num_heads=0)),
])
def test_rope_refusals(L, code, kw):
    assert rope(L, **kw) == code


def mass(L, lay=None, q=A16, Hq=64, cache=A16, bts=1024, lens=A16, n=16384, B=1, out=A16, mi=A16, mo=A16, ms=128, decay=1.0,
         ws=A16, size=BIG, err=A16):
    lay = lay or kv.dense_layout(128, 128, 8, 10)
    return L.kvarn_decode_mass(q, Hq, 0.1, cache, ctypes.byref(lay), A16, bts, lens, n, None, None, B, out, None, mi, mo, ms,
                               decay, ws, size, err, None)


@pytest.mark.parametrize("code,kw", [
    (EINVAL, dict(q=None)), (EINVAL, dict(Hq=12)), (EUNSUPPORTED, dict(Hq=72)), (EINVAL, dict(cache=None)),
    (EINVAL, dict(bts=1023)), (EINVAL, dict(mi=None)), (EINVAL, dict(mo=None)), (EINVAL, dict(ms=127)),
    (EINVAL, dict(decay=1.5)), (EINVAL, dict(decay=-0.1)), (EINVAL, dict(decay=float("nan"))), (EALIGN, dict(mi=BAD)),
    (EALIGN, dict(mo=BAD)), (EWORKSPACE, dict(size=1024)), (EINVAL, dict(err=None)), (EINVAL, dict(n=-1)),
    (EUNSUPPORTED, dict(B=65536)), (OK, dict(B=0)), (EALIGN, dict(q=BAD)),
])
def test_mass_refusals(L, code, kw):
    assert mass(L, **kw) == code


def test_mass_workspace_is_the_decodes_and_the_pairs(L):
    lay = kv.dense_layout(128, 128, 8, 10)
    n = kv.decode_mass_workspace_bytes(lay, 3, 64, 16384)
    assert n >= kv.lib().kvarn_decode_verify_workspace_bytes(ctypes.byref(lay), 3, 64, 1, 16384) + 3 * 64 * 128 * 8
    assert mass(L, B=3, bts=1024, size=n - 1) == EWORKSPACE
    with pytest.raises(kv.KvarnError):
        kv.decode_mass_workspace_bytes(kv.latent_layout(4), 1, 64, 100)
    with pytest.raises(kv.KvarnError):
        kv.decode_mass_workspace_bytes(lay, 1, 12, 100)
    for kb, vb, s16, ok in ((4, 2, True, 1), (6, 6, True, 1), (8, 8, True, 1), (4, 4, True, 1), (6, 6, False, 0),
                            (6, 3, True, 0), (3, 3, True, 0)):
        wide = kv.dense_layout(128, 128, 8, 10, k_bits=kb, v_bits=vb, fp16_scales=s16)
        assert (mass(L, lay=wide, size=1024) == EWORKSPACE) == bool(ok)
        assert (mass(L, lay=wide) == EUNSUPPORTED) == (not ok) if not ok else True


def shared(L, lay=None, q=A16, Hq=64, Q=1, cache=A16, pt=A16, S=1024, bt=A16, bts=1024, lens=A16, n=16384, cap=128, B=4, out=A16,
           ws=A16, size=BIG, err=A16, tail=None):
    lay = lay or kv.dense_layout(128, 128, 8, 10)
    return L.kvarn_decode_shared(q, Hq, Q, 0.1, cache, ctypes.byref(lay), pt, S, bt, bts, lens, n, tail, tail, cap, B, out, None,
                                 ws, size, err, None)


@pytest.mark.parametrize("code,kw", [
    (EINVAL, dict(q=None)), (EINVAL, dict(cache=None)), (EINVAL, dict(pt=None)), (EINVAL, dict(bt=None)),
    (EINVAL, dict(S=0)), (EINVAL, dict(S=1000)), (EINVAL, dict(S=-128)), (EUNSUPPORTED, dict(Q=0)),
    (EUNSUPPORTED, dict(Q=9)), (EINVAL, dict(Hq=12)), (EUNSUPPORTED, dict(Hq=72)), (EINVAL, dict(bts=1023)),
    (EINVAL, dict(cap=126)), (EINVAL, dict(Q=3, cap=128)), (EALIGN, dict(q=BAD)), (EALIGN, dict(tail=BAD)),
    (EALIGN, dict(cache=P((1 << 20) + 64))), (EWORKSPACE, dict(size=4096)), (EINVAL, dict(B=-1)), (EINVAL, dict(n=-1)),
    (EINVAL, dict(B=1 << 25)), (OK, dict(B=0)), (EINVAL, dict(out=None)), (EINVAL, dict(err=None)),
    (EINVAL, dict(lay=kv.dense_layout(128, 128, 8, 0))),
])
def test_shared_refusals(L, code, kw):
    assert shared(L, **kw) == code


def test_shared_takes_dense_layouts_only(L):
    assert shared(L, lay=kv.latent_layout(10)) == EUNSUPPORTED
    assert shared(L, lay=kv.dense_layout(64, 128, 8, 10)) == EUNSUPPORTED
    lay = kv.dense_layout(128, 128, 8, 10)
    n = kv.decode_shared_workspace_bytes(lay, 4, 64, 1, 16384, 1024)
    assert shared(L, size=n - 1) == EWORKSPACE
    for bad in ((4, 64, 0, 16384, 1024), (4, 64, 1, 16384, 0), (4, 64, 1, 16384, 100), (4, 12, 1, 16384, 1024), (-1, 64, 1, 1, 128)):
        with pytest.raises(kv.KvarnError):
            kv.decode_shared_workspace_bytes(lay, *bad)


def evict(L, lay=None, mi=A16, mo=A16, ms=8, bt=A16, bo=A16, fr=P(1 << 22), bts=64, lens=A16, lo=A16, fc=A16, n=1024, B=2, keep=4,
          sink=1, recent=1, err=A16):
    lay = lay or kv.dense_layout(128, 128, 8, 10)
    return L.kvarn_evict_tiles(mi, mo, ms, bt, bo, fr, bts, lens, lo, fc, n, B, ctypes.byref(lay), keep, sink, recent, err, None)


@pytest.mark.parametrize("code,kw", [
    (EINVAL, dict(mi=None)), (EINVAL, dict(mo=None)), (EINVAL, dict(ms=7)), (EINVAL, dict(bt=None)), (EINVAL, dict(bo=None)),
    (EINVAL, dict(fr=None)), (EINVAL, dict(bts=63)), (EINVAL, dict(lens=None)), (EINVAL, dict(lo=None)),
    (EINVAL, dict(fc=None)), (EINVAL, dict(err=None)), (EINVAL, dict(keep=1)), (EINVAL, dict(sink=-1)),
    (EINVAL, dict(recent=-1)), (EINVAL, dict(keep=-1, sink=0, recent=0)), (EINVAL, dict(fr=A16)), (EINVAL, dict(n=-1)),
    (EINVAL, dict(B=-1)), (OK, dict(B=0)), (EALIGN, dict(mi=BAD)), (EALIGN, dict(fr=BAD)),
    (EUNSUPPORTED, dict(lay=kv.latent_layout(4))), (EINVAL, dict(keep=2 ** 31 - 1, sink=2 ** 31 - 1, recent=1)),
])
def test_evict_refusals(L, code, kw):
    assert evict(L, **kw) == code


def test_frequencies():
    inv, scale = kv.rope_frequencies(64, 10000.0, device="cpu")
    assert inv.dtype == torch.float64 and inv.shape == (32,) and scale == 1.0
    assert float(inv[0]) == 1.0 and abs(float(inv[16]) - 0.01) < 1e-15
    lin, _ = kv.rope_frequencies(64, 10000.0, linear=4.0, device="cpu")
    assert torch.equal(lin, inv / 4)
    ntk, _ = kv.rope_frequencies(64, 10000.0, ntk=4.0, device="cpu")
    assert float(ntk[0]) == 1.0 and abs(float(ntk[-1] / inv[-1]) - 0.25) < 1e-12
    y, s = kv.rope_frequencies(64, 10000.0, yarn=(8.0, 4096), device="cpu")
    turns = 4096 * inv / (2 * torch.pi)
    assert torch.equal(y[turns > 64], inv[turns > 64]) and torch.allclose(y[turns < 0.5], inv[turns < 0.5] / 8, rtol=1e-12)
    assert ((y <= inv) & (y >= inv / 8 * (1 - 1e-12))).all() and abs(s - (0.1 * 2.0794415416798357 + 1)) < 1e-12
    for bad in (dict(rope_dim=63), dict(rope_dim=0), dict(rope_dim=64, linear=2.0, ntk=2.0), dict(rope_dim=64, base=-1.0),
                dict(rope_dim=2, ntk=2.0), dict(rope_dim=64, yarn=(0.5, 4096)), dict(rope_dim=64, yarn=(2.0, 4096, 1.0, 32.0))):
        with pytest.raises(kv.KvarnError):
            kv.rope_frequencies(device="cpu", **bad)


def test_the_binding_refuses_host_tensors(L):
    """There is no CPU path: every call refuses tensors that are not on the GPU."""
    x = torch.zeros(2, 1, 4, 128, dtype=torch.float16)
    i = torch.zeros(2, dtype=torch.int32)
    lay = kv.dense_layout(128, 128, 1, 8)
    cache, t, f = torch.zeros(8 * 1920, dtype=torch.uint8), torch.zeros(2, 8, dtype=torch.int32), torch.zeros(2, 1)
    out, ws = torch.zeros(2, 1, 4, 128), torch.zeros(1 << 20, dtype=torch.uint8)
    with pytest.raises(kv.KvarnError):
        kv.rope(x, x, i[:, None], torch.ones(64, dtype=torch.float64))
    with pytest.raises(kv.KvarnError):
        kv.decode_shared(x, lay, cache, t[0], 128, t, i, 128, out, ws, i[:1], 0.1)
    with pytest.raises(kv.KvarnError):
        kv.decode_mass(x[:, 0], lay, cache, t, i, 128, out[:, 0], f, f, ws, i[:1], 0.1)
    with pytest.raises(kv.KvarnError):
        kv.evict_tiles(f, t, i, lay, 128, 1, f, t, i, t.clone(), i, i[:1])
