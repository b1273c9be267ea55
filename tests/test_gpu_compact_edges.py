"""pa_compact_tokens and its 8-bit form at the ends of their arguments' range."""
import numpy as np
import pytest
import torch

from paged_kv_cache_299_gb300 import binding as pa
from _gpu import i32
from test_gpu_compact import POOLS, Cache

pytestmark = pytest.mark.gpu
LAST = (1 << 31) - 1


@pytest.mark.parametrize("pool", POOLS)
@pytest.mark.parametrize("first", [LAST, LAST - 2, LAST - 3, LAST - 4, LAST - 16, LAST - 40])
@pytest.mark.parametrize("entries", [4, 40])
def test_destinations_past_the_end_of_the_ints(pool, first, entries):
    """A wrong `first` whose list would end past 2^31 - 1 is reported and its sequence left alone."""
    c = Cache(pool, [20, 33, 0], [[1, 3, 9], list(range(1, 2 * entries, 2)), [4, 5]], 2, seed=8)
    c.run(first=i32([20, first, 0]))
    assert int(c.status.item()) == pa.DEVFLAG_BAD_CONTEXT
    c.check(skip=[1])


def raw(c):
    return [x.cpu().view(torch.uint8) for x in c.dev]


def test_tokens_that_stay_are_not_written():
    """bf16: sequences that share blocks may keep all they have there, whichever runs first."""
    c = Cache("bf16", [0, 0, 5], [list(range(40)), list(range(33)), list(range(30))], 2, seed=1)
    shared = c.bt.clone()
    shared[1:, :3] = shared[0, :3]
    before = raw(c)
    c.run(bt=shared)
    assert int(c.status.item()) == 0
    assert all(torch.equal(x, y) for x, y in zip(raw(c), before))


@pytest.mark.parametrize("kept", [list(range(23)), list(range(3, 26)), [0, 1, 2, 20]])
@pytest.mark.parametrize("first", [0, 20])
def test_forks_own_the_blocks_that_their_list_covers(kept, first):
    """8 bits: after a copy of these blocks the other owner of the context keeps every byte; the blocks before
    the list may stay shared."""
    c = Cache("q8", [first], [list(range(60))], 2, seed=2, slack=2.0)
    tables = np.zeros((2, c.bt.shape[1]), dtype=np.int32)
    tables[0] = c.w.block_tables[0]
    tables[1] = tables[0]
    used = [int(b) for b in tables[0][:-(-(first + 60) // 16)]]
    free = [b for b in range(c.w.num_blocks) if b not in used]
    covered = range(first // 16, (first + len(kept) - 1) // 16 + 1)
    pairs = []
    for i, lb in enumerate(covered):
        tables[1, lb] = free[i]
        pairs.append((used[lb], free[i]))
    assert len(free) >= len(pairs)
    before = raw(c)
    pa.pa_copy_blocks_q8(*c.dev, torch.tensor(pairs, dtype=torch.int64, device="cuda"))
    c.run(kept=i32(kept), starts=i32([0, len(kept)]), first=i32([first]), most=len(kept), bt=i32(tables[1:]))
    assert pa.pa_check_device_status(c.status) == pa.PA_OK
    for x, y in zip(raw(c), before):
        assert torch.equal(x[used], y[used])
    for which, value in ((0, c.k64), (1, c.v64)):
        have = c.dev[which].cpu().float().double() * c.dev[2 + which].cpu().double()[..., None, None]
        for i, k in enumerate(kept):
            d, s = first + i, first + k
            got, want = have[tables[1, d // 16], :, d % 16], value[used[s // 16], :, s % 16]
            step = c.dev[2 + which].cpu().double()[tables[1, d // 16]][:, None]
            assert ((got - want).abs() <= torch.maximum(2.0 ** -4 * want.abs(), 2.0 ** -10 * step)).all()
