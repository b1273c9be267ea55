"""pa_compact_tokens and its 8-bit form.  bf16 rows move bit for bit.  8-bit values go to their new
blocks as an append of them would store them: scales must be equal, codes off by half a step of
e4m3 (the values code * scale are exact in fp32 when scales are powers of two, and so is their
quotient by the new scale)."""
import numpy as np
import pytest
import torch

from paged_kv_cache_299_gb300 import binding as pa
from paged_kv_cache_299_gb300 import graphs
from paged_kv_cache_299_gb300 import workloads as wl
from _gpu import i32
from _q8 import E4M3_HALF_STEP, E4M3_SUB_HALF_STEP, needed_scale
from _tree import random_pools

pytestmark = pytest.mark.gpu
POOLS = ["bf16", "q8"]


class Cache:
    def __init__(self, pool, first, kept, hkv=2, seed=0, scales="powers", slack=0.3):
        self.pool, self.hkv, self.first, self.kept = pool, hkv, list(first), [sorted(k) for k in kept]
        lens = [f + (max(k) + 1 if k else 0) for f, k in zip(self.first, self.kept)]
        self.w = wl.make_workload("kept", lens, np.zeros(len(lens), int), num_prefill=0, seed=seed, pool_slack=slack)
        tensors, self.k64, self.v64 = random_pools(pool, self.w.num_blocks, hkv, seed + 1, scales=scales)
        self.host = tensors
        self.dev = [x.cuda() for x in tensors]
        self.bt = i32(self.w.block_tables)
        self.lists = i32(np.array([x for k in self.kept for x in k], dtype=np.int32))
        self.starts = i32(np.concatenate([[0], np.cumsum([len(k) for k in self.kept])]))
        self.first_dev = i32(self.first)
        self.most = max([len(k) for k in self.kept] + [1])
        self.status = pa.new_device_status()

    def run(self, **kw):
        a = dict(kept=self.lists, starts=self.starts, first=self.first_dev, most=self.most, bt=self.bt)
        a.update({k: kw.pop(k) for k in list(kw) if k in a})
        f = pa.pa_compact_tokens_q8 if self.pool == "q8" else pa.pa_compact_tokens
        f(a["kept"], a["starts"], a["first"], a["most"], *self.dev, a["bt"], device_status=self.status, **kw)

    def place(self, s, p):
        return int(self.w.block_tables[s, p // 16]), p % 16

    def check(self, skip=()):
        assert pa.pa_check_device_status(self.status) == pa.PA_OK or skip
        got = [x.cpu() for x in self.dev]
        for which, value in ((0, self.k64), (1, self.v64)):
            if self.pool == "bf16":
                want = self.host[which].clone()
                for s, ks in enumerate(self.kept):
                    for i, k in enumerate(ks if s not in skip else []):
                        b, o = self.place(s, self.first[s] + i)
                        fb, fo = self.place(s, self.first[s] + k)
                        want[b, :, o] = self.host[which][fb, :, fo]
                assert torch.equal(got[which].view(torch.int16), want.view(torch.int16))
                continue
            codes, scales = self.host[which].float().double(), self.host[2 + which].double().clone()
            have = got[which].float().double()
            for s, ks in enumerate(self.kept):
                if not ks or s in skip:
                    continue
                f = self.first[s]
                for lb in range(f // 16, (f + len(ks) - 1) // 16 + 1):
                    b = int(self.w.block_tables[s, lb])
                    take = [i for i in range(len(ks)) if (f + i) // 16 == lb]
                    at = [(f + i) % 16 for i in take]
                    src = [self.place(s, f + ks[i]) for i in take]
                    x = torch.stack([value[fb, :, fo] for fb, fo in src], dim=1)  # [H, n, 64]
                    for h in range(self.hkv):
                        scale = needed_scale(float(x[h].abs().max()))
                        if at[0] > 0:
                            old = float(scales[b, h])
                            scale = max(scale, old)
                            if scale > old:
                                was = codes[b, h, :at[0]] * (old / scale)
                                codes[b, h, :at[0]] = was.float().to(torch.float8_e4m3fn).double()
                        scales[b, h] = scale
                        codes[b, h, at] = x[h] / scale
            # what no step is lost on must be equal, what is rounded off by half a step at most
            tol = (E4M3_HALF_STEP * codes.abs()).clamp(min=E4M3_SUB_HALF_STEP) * (1 + 2.0 ** -20)
            exact = codes == codes.float().to(torch.float8_e4m3fn).double()
            assert torch.equal(got[2 + which].double(), scales)
            assert torch.equal(torch.where(exact, have, codes), codes)
            assert ((have - codes).abs() <= tol).all()


def lists(rng, seqs, span, low, high):
    return [sorted(rng.choice(span, size=int(rng.integers(low, high + 1)), replace=False).tolist()) for _ in range(seqs)]


@pytest.mark.parametrize("pool", POOLS)
@pytest.mark.parametrize("hkv", [1, 2, 3, 8])
def test_accepted_nodes(pool, hkv):
    rng = np.random.default_rng(hkv)
    Run = Cache(pool, rng.integers(0, 200, 20), lists(rng, 20, 26, 0, 6), hkv, seed=hkv)
    Run.run()
    Run.check()


@pytest.mark.parametrize("pool", POOLS)
def test_every_start_in_a_block(pool):
    rng = np.random.default_rng(1)
    c = Cache(pool, list(range(64)), lists(rng, 64, 40, 1, 20), 2, seed=2)
    c.run()
    c.check()


@pytest.mark.parametrize("pool", POOLS)
@pytest.mark.parametrize("n,span", [(1, 1), (15, 15), (16, 17), (17, 300), (31, 40), (32, 64), (33, 64), (100, 101),
                                    (128, 400), (129, 130), (500, 1000), (1500, 4000)])
def test_list_lengths(pool, n, span):
    rng = np.random.default_rng(n)
    c = Cache(pool, [5, 0, 77], [sorted(rng.choice(span, size=n, replace=False).tolist()) for _ in range(3)], 2, seed=n)
    c.run()
    c.check()


@pytest.mark.parametrize("pool", POOLS)
def test_keeping_all_and_keeping_none(pool):
    c = Cache(pool, [0, 9, 33, 4], [list(range(40)), [], list(range(3)), list(range(200))], 2, seed=3)
    c.run()
    c.check()


@pytest.mark.parametrize("pool", POOLS)
def test_shift_by_one_over_many_rounds(pool):
    """Every slot is the source of its neighbour: what a round writes the round before has read."""
    c = Cache(pool, [3, 0], [list(range(1, 2000)), list(range(1, 700))], 2, seed=4)
    c.run()
    c.check()


@pytest.mark.parametrize("pool", POOLS)
def test_many_long_lists(pool):
    rng = np.random.default_rng(6)
    kept = lists(rng, 20, 900, 1, 600) + [list(range(1, n)) for n in (2, 256, 257, 258, 513, 700)]
    c = Cache(pool, rng.integers(0, 40, len(kept)), kept, 8, seed=6)
    c.run()
    c.check()


@pytest.mark.parametrize("pool", POOLS)
def test_a_large_bound_changes_nothing(pool):
    rng = np.random.default_rng(5)
    first, kept = rng.integers(0, 100, 12), lists(rng, 12, 50, 0, 30)
    results = []
    for most in (30, 33, 200, 100000):
        c = Cache(pool, first, kept, 3, seed=5)
        c.run(most=most)
        c.check()
        results.append([x.cpu().view(torch.uint8) for x in c.dev])
    assert all(torch.equal(a, b) for r in results[1:] for a, b in zip(results[0], r))


def test_scales_that_are_no_powers_of_two():
    """A value code * scale and its quotient are then rounded to fp32 on the way (twice 2^-24)."""
    rng = np.random.default_rng(6)
    c = Cache("q8", rng.integers(0, 60, 10), lists(rng, 10, 40, 1, 30), 2, seed=6, scales="any")
    kept_first = [b for f in c.first for b in [f % 16]]
    assert any(kept_first)
    c.run()
    got, scales = c.dev[0].cpu().float().double(), c.dev[2].cpu().double()
    for s, ks in enumerate(c.kept):
        for i, k in enumerate(ks):
            b, o = c.place(s, c.first[s] + i)
            fb, fo = c.place(s, c.first[s] + k)
            ref = c.k64[fb, :, fo]
            step = scales[b][:, None]
            tol = torch.maximum(E4M3_HALF_STEP * ref.abs(), E4M3_SUB_HALF_STEP * step) * (1 + 2.0 ** -20)
            assert ((got[b, :, o] * step - ref).abs() <= tol).all()


@pytest.mark.parametrize("pool", POOLS)
def test_repeat_graph_and_stream(pool):
    rng = np.random.default_rng(7)
    first, kept = rng.integers(0, 100, 30), lists(rng, 30, 60, 0, 40)
    a = Cache(pool, first, kept, 4, seed=7)
    a.run()
    a.check()
    b = Cache(pool, first, kept, 4, seed=7)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    b.run(stream=side)
    torch.cuda.synchronize()
    c = Cache(pool, first, kept, 4, seed=7)
    graph = graphs.StepGraph(c.run)
    for x, h in zip(c.dev, c.host):
        x.copy_(h)  # undo the warm-up
    graph.replay()
    for other in (b, c):
        assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a.dev, other.dev))


@pytest.mark.parametrize("pool", POOLS)
def test_bad_entries_are_reported(pool):
    def fresh():
        return Cache(pool, [20, 33, 0], [[1, 3, 9], [0, 2, 5, 30], [4, 5]], 2, seed=8)

    def word(c):
        return int(c.status.item())

    c = fresh()
    c.run(most=3)  # a longer list than the bound
    assert word(c) == pa.DEVFLAG_BAD_CONTEXT
    c.check(skip=[1])
    c = fresh()
    c.run(starts=i32([0, 3, 7, 10]))  # entries outside the list
    assert word(c) == pa.DEVFLAG_BAD_CONTEXT
    c.check(skip=[2])
    c = fresh()
    c.run(first=i32([20, -1, 0]))
    assert word(c) == pa.DEVFLAG_BAD_CONTEXT
    c.check(skip=[1])
    c = fresh()
    bt = c.bt.clone()
    bt[1] = c.w.num_blocks
    c.run(bt=bt)
    assert word(c) == pa.DEVFLAG_BAD_BLOCK
    c.check(skip=[1])
    for far in (16 * c.bt.shape[1], 1 << 28, (1 << 31) - 20):  # destinations past the block-table row
        c = fresh()
        c.run(first=i32([20, far, 0]))
        assert word(c) == pa.DEVFLAG_BAD_CONTEXT
        c.check(skip=[1])
    for entries in ([1, 3, 9, 7, 7, 7, 7, 4, 5], [1, 3, 9, 0, 1 << 30, (1 << 30) + 1, (1 << 31) - 1, 4, 5],
                    [1, 3, 9, -1, -5, -(1 << 31), 0, 4, 5]):
        c = fresh()
        c.run(kept=i32(entries))
        assert word(c) & pa.DEVFLAG_BAD_CONTEXT
        got = [x.cpu() for x in c.dev]
        # the other sequences moved as they should, and this one touched no block but its own
        own = set(int(b) for b in c.w.block_tables[1][:4])
        d = fresh()
        d.run()
        for x, y in zip(got, d.dev):
            rest = [b for b in range(c.w.num_blocks) if b not in own]
            assert torch.equal(x.view(torch.uint8)[rest], y.cpu().view(torch.uint8)[rest])


def test_bad_scales_leave_the_block():
    c = Cache("q8", [4], [[2, 5]], 1, seed=9)
    c.dev[2][int(c.w.block_tables[0, 0])] = float("nan")
    c.run()
    assert int(c.status.item()) == pa.DEVFLAG_BAD_SCALE
    assert torch.equal(c.dev[0].cpu().view(torch.uint8), c.host[0].view(torch.uint8))
    assert not torch.equal(c.dev[1].cpu().view(torch.uint8), c.host[1].view(torch.uint8))


def test_blocks_far_into_large_pools():
    blocks, hkv = 300000, 8  # 4.9 GB a pool
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("not enough device memory")
    kc = torch.zeros(blocks, hkv, 16, 64, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    far = [blocks - 1, blocks - 20]
    x = torch.randn(2, hkv, 16, 64).to(torch.bfloat16).cuda()
    kc[far] = x
    vc[far] = -x
    pa.pa_compact_tokens(i32([3, 17]), i32([0, 2]), i32([2]), 2, kc, vc, i32([far]))
    assert torch.equal(kc[far[0], :, 2], x[0, :, 5]) and torch.equal(kc[far[0], :, 3], x[1, :, 3])
    assert torch.equal(vc[far[0], :, 2], -x[0, :, 5]) and torch.equal(vc[far[0], :, 3], -x[1, :, 3])
