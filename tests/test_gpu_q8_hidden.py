"""Blocks of the 8-bit cache that read as NaN and that some queries of a verification see and others do not: the rows
that see nothing of them keep their bits."""
import numpy as np
import pytest
import torch

import quantized_kv_cache_kvarn_gb300 as kv
from tests import blocks8 as b8
from tests.test_gpu_q8 import check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_kv_cache_kvarn_gb300 import build
    build.build()
    kv.lib()


def block_of_the_first_queries(x, b):
    """The block of sequence b that query 0 sees the end of and the last query nothing, and the first query that does not
    see it; None where there is none. (Every block that the table names is seen by some query: a block of which none sees
    anything is not read.)"""
    L, Q, W, S = x.lens[b], x.Q, x.window, x.sinks
    for u in range(x.done[b]):
        sees = [any(i < S or i > L - Q + j - W for i in range(16 * u, 16 * u + 16)) for j in range(Q)]
        if sees[0] and not sees[-1]:
            return u, sees.index(False)
    return None


@pytest.mark.parametrize("scales", [(0, 1), (0,), (1,)])
@pytest.mark.parametrize("code", [b8.E4M3, b8.INT8])
@pytest.mark.parametrize("Hq,Hkv,D", [(4, 2, 128), (8, 2, 128), (2, 1, 256), (8, 2, 256)])
def test_blocks_of_nan_that_leave_the_window(Hq, Hkv, D, code, scales):
    Q, W, S = 4, 20, 5
    x = b8.Batch([84, 85, 86, 200, 36 + 160, 30], Hq, Hkv, D, Q=Q, window=W, sinks=S, code=code, seed=D + Hq).gpu(kv)
    first, first_lse = (t.clone() for t in x.decode(kv))
    check(x, first, first_lse)
    poisoned = []
    for b in range(len(x.lens)):
        found = block_of_the_first_queries(x, b)
        if found:
            poisoned.append((b, *found))
            for side in scales:
                at = 32 * D + 4 * side
                x.t["cache"][int(x.table[b, found[0]]), :, at:at + 4] = 255
    assert len(poisoned) >= 4 and {p[2] for p in poisoned} == {1, 2, 3}
    out, lse = x.decode(kv)
    assert kv.read_error_flags(x.t["err"]) == 0
    for b in range(len(x.lens)):
        until = next((p[2] for p in poisoned if p[0] == b), 0)
        assert out[b, :until].isnan().all()
        assert lse[b, :until].isnan().all() if 0 in scales else torch.equal(lse[b, :until], first_lse[b, :until])
        assert torch.equal(out[b, until:], first[b, until:]) and torch.equal(lse[b, until:], first_lse[b, until:])


@pytest.mark.parametrize("Hq,Hkv,D,Q", [(4, 2, 128, 1), (8, 2, 128, 4), (2, 1, 256, 1), (8, 2, 256, 4)])
def test_pages_that_nobody_sees_are_not_read(Hq, Hkv, D, Q):
    """Blocks outside every query's window whose table entries name pages of NaN: the same bits as with entries that name
    no page at all."""
    W, S = 40, 18
    x = b8.Batch([500, 130, 77], Hq, Hkv, D, Q=Q, window=W, sinks=S, seed=Q).gpu(kv)
    first, first_lse = (t.clone() for t in x.decode(kv))
    check(x, first, first_lse)
    hidden = (x.table == 0x7fffffff) & (np.arange(x.table.shape[1]) < np.array(x.done)[:, None])
    assert hidden.sum() > 20
    used = set(x.table[x.table != 0x7fffffff].tolist())
    spare = next(p for p in range(x.cache.shape[0]) if p not in used)
    x.t["cache"][spare] = 255
    table = torch.from_numpy(np.where(hidden, spare, x.table).astype(np.int32)).cuda()
    out, lse = x.decode(kv, table=table)
    assert kv.read_error_flags(x.t["err"]) == 0 and torch.equal(out, first) and torch.equal(lse, first_lse)
