"""The calls around the 8-bit block cache as a serving loop makes them: norms and positions of the new tokens, append,
attention behind a window with sinks, beams that fork and end, pages given back and the cache compacted; every step's
output against its definition over what every beam has seen, once eagerly and once with the step replayed from graphs."""
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


class Loop:
    """Two requests of two beams; `self.seen` holds every row's keys and values as they went into the cache."""

    def __init__(self, code, bf16, Hq=4, Hkv=2, D=128, window=40, sinks=4, prompts=(37, 64), pages=60, T=12):
        self.code, self.Hq, self.Hkv, self.D, self.W, self.S, self.T = code, Hq, Hkv, D, window, sinks, T
        self.dt = torch.bfloat16 if bf16 else torch.float16
        self.g = torch.Generator(device="cuda").manual_seed(3)
        self.B = B = 2 * len(prompts)
        self.lay = kv.q8_layout(D, Hkv, pages, kv.BF16 if bf16 else kv.FP16)
        i32 = dict(dtype=torch.int32, device="cuda")
        self.cache, self.err, self.max_len = kv.alloc_q8_cache(self.lay), kv.new_error_word(), T * 16 + 15
        self.inv, _ = kv.rope_frequencies(D)
        self.weights = [1 + 0.2 * torch.randn(D, generator=self.g, device="cuda") for _ in range(2)]
        # two of everything that a step's fork writes; self.now says which is current
        self.table = [torch.full((B, T), -1, **i32) for _ in range(2)]
        self.lens = [torch.zeros(B, **i32) for _ in range(2)]
        self.tail = [[torch.zeros((B, Hkv, 16, D), dtype=self.dt, device="cuda") for _ in range(2)] for _ in range(2)]
        self.refs, self.freed, self.count = torch.zeros(pages, **i32), torch.zeros(pages, **i32), torch.zeros(1, **i32)
        self.remap, self.live, self.parents = torch.zeros(pages, **i32), torch.zeros(1, **i32), torch.zeros(B, **i32)
        self.now, self.free = 0, list(range(pages))
        self.x = [torch.zeros((B, 1, h, D), dtype=self.dt, device="cuda") for h in (Hq, Hkv, Hkv)]  # q, k, v of the step
        self.pos = torch.zeros((B, 1), **i32)
        self.out, self.lse = torch.zeros((B, 1, Hq, D), device="cuda"), torch.zeros((B, 1, Hq), device="cuda")
        n = kv.q8_decode_workspace_bytes(self.lay, B, Hq, 1, self.max_len, window, sinks)
        self.space = torch.empty(n, dtype=torch.uint8, device="cuda")
        self.cspace = torch.empty(kv.compact_pages_workspace_bytes(pages), dtype=torch.uint8, device="cuda")
        self.seen = [None] * B
        for r, L in enumerate(prompts):
            self.prompt(r, L)

    def prompt(self, r, L):
        """A request's prompt, shared by its two rows: whole blocks to pages, the rest to the tails."""
        k, v = (torch.randn((1, L, self.Hkv, self.D), generator=self.g, device="cuda").to(self.dt) for _ in range(2))
        kv.norm_rope(k, k, self.weights[1], torch.arange(L, dtype=torch.int32, device="cuda")[None], self.inv)
        n = L // 16
        ids = [self.free.pop(0) for _ in range(n)]
        table = torch.tensor([ids], dtype=torch.int32).cuda()
        kv.q8_encode_blocks(k[:, :16 * n].transpose(1, 2), v[:, :16 * n].transpose(1, 2), self.lay, self.code,
                            torch.zeros(1, dtype=torch.int32, device="cuda"), table, self.cache, self.err)
        for b in (2 * r, 2 * r + 1):
            self.table[0][b, :n] = table[0]
            self.lens[0][b] = L
            for t, x in zip(self.tail[0], (k, v)):
                t[b, :, :L - 16 * n] = x[0, 16 * n:].transpose(0, 1)
            self.seen[b] = [x[0].transpose(0, 1).float().cpu().numpy() for x in (k, v)]
        self.refs[ids] = 2

    def inputs(self):
        for x in self.x:
            x.copy_(torch.randn(x.shape, generator=self.g, device="cuda").to(self.dt))
        lens = self.lens[self.now]
        self.pos.copy_(lens[:, None])
        lens += 1
        for b, L in enumerate(lens.tolist()):
            if L % 16 == 0:
                page = self.free.pop(0)
                self.table[self.now][b, L // 16 - 1] = page
                self.refs[page] = 1

    def step(self):
        c = self.now
        kv.norm_rope(self.x[:2], self.x[:2], self.weights, self.pos, self.inv)
        kv.q8_append(self.x[1][:, 0], self.x[2][:, 0], self.lay, self.code, self.lens[c], self.max_len, *self.tail[c],
                     self.table[c], self.cache, self.err)
        kv.q8_decode(self.x[0], self.lay, self.code, self.cache, self.table[c], self.lens[c], self.max_len, self.out, self.space,
                     self.err, self.D ** -0.5, *self.tail[c], self.lse, window=self.W, sink_tokens=self.S)
        kv.fork_sequences(self.parents, self.lens[c], self.table[c], self.refs, self.lay, self.max_len, self.lens[1 - c],
                          self.table[1 - c], self.refs, self.freed, self.count, self.err,
                          tails=tuple(zip(self.tail[c], self.tail[1 - c])), window=self.W, sink_tokens=self.S)

    def check(self, parents):
        """The step's outputs, then the rows that go on."""
        for b in range(self.B):
            self.seen[b] = [np.concatenate([old, x[b].transpose(0, 1).float().cpu().numpy()], 1) for old, x in zip(self.seen[b], self.x[1:])]
            L = self.seen[b][0].shape[1]
            n = L // 16 * 16
            kvs = []
            for x in self.seen[b]:
                codes, scale = b8.code_bytes(x[:, :n].reshape(self.Hkv, -1, 16, self.D), self.code)
                whole = b8.byte_values(codes, self.code) * scale.astype(np.float64)[..., None, None]
                kvs.append(np.concatenate([whole.reshape(self.Hkv, n, self.D), x[:, n:].astype(np.float64)], 1))
            want, lse, off, off_lse = b8.attend(self.x[0][b].double().cpu().numpy(), *kvs, self.D ** -0.5, L, self.W, self.S)
            assert (np.abs(self.out[b].double().cpu().numpy() - want) <= off).all()
            assert (np.abs(self.lse[b].double().cpu().numpy() - lse) <= off_lse).all()
        self.seen = [self.seen[p] for p in parents]
        self.now = 1 - self.now
        assert kv.read_error_flags(self.err) == 0
        gone = self.freed[:int(self.count)].tolist()
        assert gone == sorted(gone) and not set(gone) & set(self.free)
        self.free += gone
        # the counts are those of the rows
        held = self.table[self.now].flatten()
        assert torch.equal(self.refs, torch.bincount(held[held >= 0], minlength=self.refs.numel()).int())
        assert sorted(self.free) == torch.nonzero(self.refs == 0).flatten().tolist()

    def compact(self):
        t = self.table[self.now]
        kv.compact_pages(self.cache, self.refs, t, self.refs, t, self.remap, self.live, self.cspace, self.err)
        assert kv.read_error_flags(self.err) == 0
        self.free = list(range(int(self.live), self.refs.numel()))
        assert (self.refs[:int(self.live)] > 0).all() and not self.refs[int(self.live):].any()


@pytest.mark.parametrize("code,bf16,D,graphs", [(b8.E4M3, False, 128, False), (b8.INT8, True, 256, False), (b8.INT8, False, 128, True)])
def test_loop(code, bf16, D, graphs):
    x = Loop(code, bf16, D=D)
    rng = np.random.default_rng(1)
    captured = []
    if graphs:
        x.inputs()
        x.parents.copy_(torch.arange(4))
        state = [t.clone() for t in (x.refs, x.cache, *x.lens, *x.table, *(y for z in x.tail for y in z), *x.x)]
        x.step()  # before a capture, so that the kernels' attributes are set
        for t, s in zip((x.refs, x.cache, *x.lens, *x.table, *(y for z in x.tail for y in z), *x.x), state):
            t.copy_(s)
        for x.now in (0, 1):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                x.step()
            captured.append(g)
        x.now = 0
    for i in range(75):
        if i or not graphs:
            x.inputs()
        parents = [2 * r + int(rng.integers(2)) for r in range(2) for _ in range(2)]
        x.parents.copy_(torch.tensor(parents))
        if graphs:
            captured[x.now].replay()
        else:
            x.step()
        x.check(parents)
        if i % 11 == 10:
            x.compact()
