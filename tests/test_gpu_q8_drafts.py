"""Verification of drafted tokens over the 8-bit block cache as a decoding loop makes it: the sampled token appended, the
drafts written behind it in the raw tail, all of them attended over, and those that were accepted appended."""
import numpy as np
import pytest
import torch

import quantized_kv_cache_kvarn_gb300 as kv
from tests import blocks8 as b8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_kv_cache_kvarn_gb300 import build
    build.build()
    kv.lib()


@pytest.mark.parametrize("Q,D,code,bf16,window,sinks", [(2, 128, b8.E4M3, False, 0, 0), (4, 128, b8.INT8, True, 40, 4), (8, 256, b8.E4M3, False, 0, 0),
                                                        (8, 128, b8.INT8, False, 50, 3)])
def test_drafted_tokens(Q, D, code, bf16, window, sinks):
    B, Hq, Hkv, T, steps = 5, 4, 2, 16, 24
    dt, rng = torch.bfloat16 if bf16 else torch.float16, np.random.default_rng(Q)
    lay = kv.q8_layout(D, Hkv, B * T, kv.BF16 if bf16 else kv.FP16)
    table = torch.from_numpy(rng.permutation(B * T).astype(np.int32).reshape(B, T)).cuda()
    cache, err, most = kv.alloc_q8_cache(lay), kv.new_error_word(), T * 16
    tails = [torch.zeros((B, Hkv, Q + 14, D), dtype=dt, device="cuda") for _ in range(2)]
    space = torch.empty(kv.q8_decode_workspace_bytes(lay, B, Hq, Q, most, window, sinks), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty((B, Q, Hq, D), device="cuda"), torch.empty((B, Q, Hq), device="cuda")
    n = torch.tensor([0, 3, 14, 15, 16], dtype=torch.int32, device="cuda")  # accepted tokens
    rows = torch.arange(B, device="cuda")
    seen = [[np.zeros((Hkv, 0, D), np.float32) for _ in range(2)] for _ in range(B)]

    def tokens():
        return torch.from_numpy(rng.standard_normal((B, Hkv, D)).astype(np.float32)).to(dt).cuda()

    def remember(kvs, which):
        for b in which:
            seen[b] = [np.concatenate([s, x[b, :, None].float().cpu().numpy()], 1) for s, x in zip(seen[b], kvs)]

    for i in range(16):  # prompts, a token at a time
        kvs, on = [tokens(), tokens()], i < n
        kv.q8_append(*kvs, lay, code, torch.where(on, i + 1, 0).int(), most, *tails, table, cache, err)
        remember(kvs, torch.nonzero(on).flatten().tolist())
    crossed = 0
    for step in range(steps):
        drafts = [[tokens(), tokens()] for _ in range(Q)]  # the sampled token and Q - 1 behind it
        n += 1
        kv.q8_append(*drafts[0], lay, code, n, most, *tails, table, cache, err)
        for j in range(1, Q):  # drafted token j is row n % 16 + j - 1: no block is completed before it is accepted
            for tail, x in zip(tails, drafts[j]):
                tail[rows, :, (n % 16 + j - 1).long()] = x
        lens = n + Q - 1
        q = torch.from_numpy(rng.standard_normal((B, Q, Hq, D)).astype(np.float32)).to(dt).cuda()
        kv.q8_decode(q, lay, code, cache, table, lens, most, out, space, err, D ** -0.5, *tails, lse, window=window, sink_tokens=sinks)
        accepted = rng.integers(0, Q, B)  # of the Q - 1 drafts
        for b in range(B):
            L = int(lens[b])
            kvs = []
            for side in (0, 1):
                x = np.concatenate([seen[b][side]] + [d[side][b, :, None].float().cpu().numpy() for d in drafts], 1)
                assert x.shape[1] == L
                whole = (L - Q + 1) // 16 * 16
                codes, scale = b8.code_bytes(x[:, :whole].reshape(Hkv, -1, 16, D), code)
                values = b8.byte_values(codes, code) * scale.astype(np.float64)[..., None, None]
                kvs.append(np.concatenate([values.reshape(Hkv, whole, D), x[:, whole:].astype(np.float64)], 1))
            want, want_lse, off, off_lse = b8.attend(q[b].double().cpu().numpy(), *kvs, D ** -0.5, L, window, sinks)
            assert (np.abs(out[b].double().cpu().numpy() - want) <= off).all(), (step, b)
            assert (np.abs(lse[b].double().cpu().numpy() - want_lse) <= off_lse).all(), (step, b)
        remember(drafts[0], range(B))
        crossed += sum(int(a) // 16 != (int(a) + int(m)) // 16 for a, m in zip(n.tolist(), accepted))
        for j in range(1, Q):  # the accepted ones: each to its row, or completing a block; length 0 passes a sequence by
            on = torch.from_numpy(accepted >= j).cuda()
            n += on
            kv.q8_append(*drafts[j], lay, code, torch.where(on, n, 0).int(), most, *tails, table, cache, err)
            remember(drafts[j], np.flatnonzero(accepted >= j).tolist())
        assert kv.read_error_flags(err) == 0
        if int(n.max()) + Q > most:
            break
    assert crossed > 2
