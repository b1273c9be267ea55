"""pa_tree_attention and pa_tree_attention_q8 against attention in 64 bits under the same masks
(tolerance: _tree.attend_tree)."""
import random

import numpy as np
import pytest
import torch

from paged_kv_cache_299_gb300 import binding as pa
from paged_kv_cache_299_gb300 import graphs
from paged_kv_cache_299_gb300 import workloads as wl
from _gpu import i32
from _tree import KINDS, attend_tree, batch_bits, live_slots, mask_words, random_pools

pytestmark = pytest.mark.gpu
POOLS = ["bf16", "q8"]


class Trees:
    """A batch of drafted trees over pools whose every slot that is not in use is poison."""

    def __init__(self, pool, hist, nodes, hq=32, hkv=8, kind="tree", seed=0, pad=0, words=None, junk=True, bits=None,
                 slack=0.3, **kw):
        self.pool, self.hq, self.hkv = pool, hq, hkv
        self.nodes = [int(n) for n in nodes]
        w = self.w = wl.make_workload("trees", hist, nodes, num_prefill=len(self.nodes), seed=seed, pool_slack=slack)
        self.lens = [int(n) for n in w.context_lens]
        live = live_slots(w.num_blocks, w.block_tables, self.lens)
        tensors, self.k64, self.v64 = random_pools(pool, w.num_blocks, hkv, seed + 1, live, **kw)
        self.dev = [x.cuda() for x in tensors]
        self.rows = sum(self.nodes)
        g = torch.Generator().manual_seed(seed + 2)
        self.q = (1.5 * torch.randn(self.rows + pad, hq, 64, generator=g)).to(torch.bfloat16)
        self.pad = pad
        self.bits = bits or batch_bits(kind, self.nodes, seed)
        self.mask = mask_words(self.bits, self.nodes, words, pad, junk).cuda()
        self.bt, self.ctx = i32(w.block_tables), i32(self.lens)
        self.starts = i32(np.concatenate([[0], np.cumsum(self.nodes)]))
        self.most = max(self.nodes)
        self.status = pa.new_device_status()

    def run(self, **kw):
        f = pa.pa_tree_attention_q8 if self.pool == "q8" else pa.pa_tree_attention
        out = torch.full(self.q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        a = dict(q=self.q.cuda(), mask=self.mask, starts=self.starts, most=self.most, dev=self.dev, bt=self.bt, ctx=self.ctx,
                 device_status=self.status)
        a.update(kw)
        f(out, a.pop("q"), a.pop("mask"), a.pop("starts"), a.pop("most"), *a.pop("dev"), a.pop("bt"), a.pop("ctx"), 0.125, **a)
        return out

    def ok(self):
        return pa.pa_check_device_status(self.status) == pa.PA_OK

    def expected(self):
        return attend_tree(self.q[:self.rows], self.k64.cuda(), self.v64.cuda(), self.w.block_tables, self.lens,
                           self.nodes, self.bits, 0.125)

    def check(self, got=None, floor=0.0):
        got = (self.run() if got is None else got).cpu().double()
        assert self.ok()
        ref, tol = self.expected()
        if self.pad:
            assert (got[self.rows:] == 7.0).all()
        close(got[:self.rows], ref, tol + floor)
        return got


def close(got, ref, tol):
    assert torch.isfinite(got).all(), "non-finite output (poison was read)"
    bad = (got - ref).abs() > tol
    worst = float(((got - ref).abs() / tol.clamp(min=1e-30)).max())
    assert not bad.any(), f"{int(bad.sum())} values out of tolerance, worst {worst:.3g} of it, rows {bad.flatten(1).any(dim=1).nonzero().flatten().tolist()[:20]}"


@pytest.mark.parametrize("pool", POOLS)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("hq,hkv", [(32, 8), (1, 1), (6, 3), (8, 8), (4, 1)])
def test_head_layouts(pool, kind, hq, hkv):
    Trees(pool, [0, 5, 33, 200, 700], [17, 1, 40, 3, 64], hq, hkv, kind, seed=hq).check()


@pytest.mark.parametrize("pool", POOLS)
@pytest.mark.parametrize("hq,hkv", [(4, 1), (2, 1), (1, 1)])
def test_every_number_of_nodes(pool, hq, hkv):
    nodes = list(range(1, 70)) + [95, 96, 97, 127, 128, 129, 191, 192, 193, 255, 256, 257]
    Trees(pool, [(37 * n) % 150 for n in nodes], nodes, hq, hkv, "mask", seed=3).check()


@pytest.mark.parametrize("pool", POOLS)
@pytest.mark.parametrize("n", [1, 7, 33])
def test_every_prefix_length(pool, n):
    """Where the drafted tokens begin and end within a block and within a tile of keys."""
    Trees(pool, list(range(0, 146)), [n] * 146, 4, 1, "mask", seed=n).check()


@pytest.mark.parametrize("pool", POOLS)
@pytest.mark.parametrize("L", [0, 1, 300, 2000, 9000, 40000])
@pytest.mark.parametrize("n", [1, 12, 60])
def test_one_sequence(pool, L, n):
    Trees(pool, [L], [n], 8, 2, "tree", seed=L + n, slack=0.5).check()


@pytest.mark.parametrize("L", [300, 4000, 32000, 60000])
@pytest.mark.parametrize("seqs,hq,hkv,n", [(1, 8, 2, 8), (3, 4, 1, 3), (1, 2, 1, 16), (1, 1, 1, 32)])
def test_few_rows_over_8_bits(L, seqs, hq, hkv, n):
    """At most 32 rows per K/V head: contexts on both sides of where another kernel takes over."""
    Trees("q8", [L - 7 * i for i in range(seqs)], [n] + [max(1, n - 2)] * (seqs - 1), hq, hkv, "mask", seed=L + n).check()


@pytest.mark.parametrize("seqs,hq,hkv", [(40, 32, 8), (14, 16, 8), (9, 32, 8), (24, 3, 3)])
def test_small_trees_of_uneven_batches(seqs, hq, hkv):
    """Under block tables as wide as the contexts, and as wide as a cache for much longer ones (entries that are not
    in use name no block): what serves the call depends on it."""
    r = np.random.default_rng(seqs)
    t = Trees("q8", r.integers(0, 1900, seqs), r.integers(1, 9, seqs), hq, hkv, "tree", seed=seqs)
    t.check()
    t.check(t.run(bt=torch.nn.functional.pad(t.bt, (0, 1100), value=-1)))


@pytest.mark.parametrize("pool", POOLS)
@pytest.mark.parametrize("hist,nodes", [
    ([20000] + [30] * 40, [20] + [5] * 40),
    ([30, 0, 0, 9000, 17, 0, 700], [1, 3, 0, 64, 0, 9, 130]),
    (list(range(0, 300)), [1 + i % 4 for i in range(300)]),
    ([600, 0, 1, 90] + [16] * 9, [4] * 13),
    ([5000] * 3, [100, 1, 32])])
def test_uneven_batches(pool, hist, nodes):
    Trees(pool, hist, nodes, 8, 2, "tree", seed=len(hist)).check()


@pytest.mark.parametrize("pool", POOLS)
def test_serving_batch(pool):
    r = np.random.default_rng(4)
    Trees(pool, r.integers(100, 1500, 32), r.integers(8, 33, 32), seed=4).check()


@pytest.mark.parametrize("pool", POOLS)
@pytest.mark.parametrize("hist,seqs", [(100, 70), (1500, 40), (1500, 70), (4000, 30)])
def test_large_and_small_trees_together(pool, hist, seqs):
    """More segments than CTAs, and of the two halves of a CTA's rows now one, now both in use."""
    r = np.random.default_rng(seqs)
    Trees(pool, r.integers(0, hist, seqs), r.integers(1, 70, seqs), 32, 8, "tree", seed=seqs).check()


@pytest.mark.parametrize("pool", POOLS)
def test_many_short_sequences(pool):
    r = np.random.default_rng(5)
    Trees(pool, r.integers(0, 40, 3000), r.integers(0, 3, 3000), 4, 1, "tree", seed=5).check()


@pytest.mark.parametrize("pool", POOLS)
def test_largest_tree(pool):
    Trees(pool, [100], [1024], 4, 1, "mask", seed=6).check()


@pytest.mark.parametrize("pool", POOLS)
def test_rows_that_see_nothing_are_zero(pool):
    t = Trees(pool, [0, 0, 40], [5, 33, 4], 8, 2, bits=[[0] * 5, [0, 1] * 16 + [0], [0] * 4], seed=7)
    got = t.check()
    assert (got[:5] == 0).all() and (got[5:38:2] == 0).all()


@pytest.mark.parametrize("pool", POOLS)
def test_padding_rows_and_empty_sequences(pool):
    Trees(pool, [4, 9, 0, 50], [0, 12, 0, 2], 8, 8, seed=8, pad=9).check()


@pytest.mark.parametrize("pool", POOLS)
def test_wider_masks_than_needed(pool):
    """Words past the drafted tokens, their bits set, change nothing."""
    t = Trees(pool, [70, 10], [31, 33], 4, 1, "mask", seed=9)
    u = Trees(pool, [70, 10], [31, 33], 4, 1, "mask", seed=9, words=7)
    assert torch.equal(t.check(), u.check())


def test_chain_is_the_causal_chunk():
    t = Trees("bf16", [0, 100, 1000], [30, 64, 9], kind="chain", seed=10)
    got = t.check()
    out = torch.empty_like(t.q, device="cuda")
    pa.pa_prefill_chunk(out, t.q.cuda(), t.starts, t.most, *t.dev, t.bt, t.ctx, 0.125)
    ref, tol = t.expected()
    assert ((out.cpu().double() - got).abs() <= 2 * tol).all()


@pytest.mark.parametrize("what", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("hist,n,hq,hkv", [(0, 20, 4, 1), (50, 20, 8, 2), (60, 70, 2, 2), (3000, 33, 4, 1)])
def test_what_a_row_does_not_see_never_reaches_it(what, hist, n, hq, hkv):
    """A drafted token whose key or value is no number reaches the rows that see it, and no other."""
    for which in (0, 1):
        t = Trees("bf16", [hist, 10], [n, 5], hq, hkv, "tree", seed=11)
        j = n // 2
        pos = hist + j
        block, off = int(t.w.block_tables[0, pos // 16]), pos % 16
        clean = t.run().cpu()
        t.dev[which][block, :, off, 5:40] = what
        got = t.run().cpu()
        assert t.ok()
        sees = [i for i, b in enumerate(t.bits[0]) if b >> j & 1]
        blind = [i for i in range(t.rows) if i not in sees]
        assert torch.equal(got[blind], clean[blind])
        assert sees
        if which == 1:
            assert not torch.isfinite(got[sees][..., 5:40].float()).any()
            if what == what:
                assert (got[sees][..., 5:40].float() == what).all()
            assert torch.equal(got[sees][..., :5], clean[sees][..., :5])
            assert torch.equal(got[sees][..., 40:], clean[sees][..., 40:])
        elif what != what:
            assert torch.isnan(got[sees].float()).all()


def test_non_finite_prefix_reaches_every_row():
    t = Trees("bf16", [100, 100], [4, 4], 4, 1, seed=12)
    t.dev[1][int(t.w.block_tables[0, 2]), :, 3, 7] = float("inf")
    got = t.run().cpu().float()
    assert (got[:4, :, 7] == float("inf")).all() and torch.isfinite(got[4:]).all()


@pytest.mark.parametrize("pool", POOLS)
def test_large_scores(pool):
    """Scores far apart: the running maximum moves and rows rescale."""
    t = Trees(pool, [500, 3000], [9, 40], 4, 1, "tree", seed=13, spread=2.0)
    t.q *= 8
    t.check()


@pytest.mark.parametrize("q_size", [2.0 ** -60, 2.0 ** 30])
def test_query_sizes(q_size):
    for pool in POOLS:
        t = Trees(pool, [90], [20], 4, 1, "tree", seed=14)
        t.q *= q_size
        t.check()


def test_scales_that_are_no_powers_of_two():
    Trees("q8", [5, 100, 2000], [20, 1, 64], 8, 2, "mask", seed=15, scales="any").check()


@pytest.mark.parametrize("key_exp,value_exp", [(-120, -100), (90, 100), (0, 0), (-149, -140), (-160, -160)])
def test_extreme_scales(key_exp, value_exp):
    """Block scales over the whole range of floats, zero and the subnormal ones included."""
    t = Trees("q8", [120, 700], [16, 33], 4, 1, "mask", seed=16)
    for pool, e in ((0, key_exp), (1, value_exp)):
        codes = t.dev[pool].cpu()
        scale = torch.full((t.w.num_blocks, 1), 2.0 ** e if e > -150 else 0.0)
        t.dev[2 + pool] = scale.cuda()
        x = codes.float().nan_to_num(0).double() * scale.double()[..., None, None]
        if pool == 0:
            t.k64 = x
        else:
            t.v64 = x
    if key_exp > 0:
        t.q = (t.q.float() * 2.0 ** (-key_exp - 8)).to(torch.bfloat16)
    t.check(floor=2.0 ** -126)  # (what falls below the normal floats may vanish)


@pytest.mark.parametrize("pool", POOLS)
def test_one_workspace_serves_batches_of_every_size(pool):
    ws = torch.zeros(pa.pa_tree_workspace_size(), dtype=torch.uint8, device="cuda")
    batches = [([40000], [9], 8, 2), ([10, 2000, 0], [3, 40, 7], 32, 8), ([9000] * 5, [70] * 5, 4, 1),
               ([100] * 200, [2] * 200, 2, 1)]
    for turn in range(2):
        for i, (hist, nodes, hq, hkv) in enumerate(batches):
            t = Trees(pool, hist, nodes, hq, hkv, seed=20 + i)
            first = t.run(workspace=ws)
            t.check(first)
            assert torch.equal(first, t.run(workspace=ws))  # and the results repeat, bit for bit


@pytest.mark.parametrize("pool", POOLS)
def test_replays_and_streams(pool):
    t = Trees(pool, [3000, 17, 800], [20, 5, 64], seed=30)
    ws = torch.zeros(pa.pa_tree_workspace_size(), dtype=torch.uint8, device="cuda")
    q, out = t.q.cuda(), torch.empty_like(t.q, device="cuda")
    f = pa.pa_tree_attention_q8 if pool == "q8" else pa.pa_tree_attention

    def step():
        f(out, q, t.mask, t.starts, t.most, *t.dev, t.bt, t.ctx, 0.125, workspace=ws, device_status=t.status)

    want = t.check()
    one, two = graphs.StepGraph(step), graphs.StepGraph(step)  # two graphs, one after the other, on one workspace
    for graph in (one, two, one):
        out.zero_()
        graph.replay()
        assert torch.equal(out.cpu().double(), want)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = t.run(stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got.cpu().double(), want)
    # a replayed graph follows lengths that change in place
    t.ctx.copy_(i32([2999 + 20, 10 + 5, 64 + 64]))
    t.lens = [3019, 15, 128]
    one.replay()
    t.check(out)


@pytest.mark.parametrize("n", [4, 40])
@pytest.mark.parametrize("pool", POOLS)
def test_contexts_longer_than_the_pool_are_reported(pool, n):
    t = Trees(pool, [100, 20], [n, 3], 4, 1, seed=33)
    wide = t.bt.repeat(1, 40).contiguous().clamp(min=0)
    got = t.run(bt=wide, ctx=i32([16 * t.w.num_blocks + 1, 23]))
    assert int(t.status.item()) == pa.DEVFLAG_BAD_CONTEXT and (got[:n] == 7.0).all()


@pytest.mark.parametrize("n", [6, 70])
@pytest.mark.parametrize("pool", POOLS)
def test_bad_entries_are_reported(pool, n):
    def flag(t, **kw):
        t.status.zero_()
        got = t.run(**kw)
        return int(t.status.item()), got.cpu().double()

    def fresh():
        return Trees(pool, [100, 40, 7], [9, n, 3], 8, 2, seed=31)

    t = fresh()
    ref, tol = t.expected()
    others = list(range(9)) + [9 + n, 10 + n, 11 + n]
    past = 40 + n
    bt = t.bt.clone()
    bt[1, 1] = t.w.num_blocks
    word, got = flag(t, bt=bt)
    assert word == pa.DEVFLAG_BAD_BLOCK
    close(got[others], ref[others], tol[others])
    bt[1, 1] = -1
    assert flag(t, bt=bt)[0] == pa.DEVFLAG_BAD_BLOCK
    for ctx in ([109, 5, 10], [109, -3, 10], [109, 1 << 30, 10]):  # shorter than its rows; past its table row
        word, got = flag(t, ctx=i32(ctx))
        assert word == pa.DEVFLAG_BAD_CONTEXT
        assert (got[9:9 + n] == 7.0).all()
        close(got[others], ref[others], tol[others])
    most = max(9, n) - 1  # a tree larger than max_query_len
    word, got = flag(t, most=most)
    lost = list(range(9)) if n < 9 else list(range(9, 9 + n))
    kept = [i for i in range(t.rows) if i not in lost]
    assert word == pa.DEVFLAG_BAD_CONTEXT and (got[lost] == 7.0).all()
    close(got[kept], ref[kept], tol[kept])
    word, got = flag(t, starts=i32([0, 9, 9 + n, 13 + n]), ctx=i32([109, past, 11]))  # rows past the buffer
    assert word == pa.DEVFLAG_BAD_CONTEXT and (got[9 + n:] == 7.0).all()
    close(got[:9 + n], ref[:9 + n], tol[:9 + n])
    word, got = flag(t, starts=i32([0, 9, 4, 7]), ctx=i32([109, past, 10]))  # fewer than no rows: none
    assert word in (0, pa.DEVFLAG_BAD_CONTEXT)
    t = fresh()
    t.check()  # and the call after is as ever


def test_blocks_far_into_large_pools():
    """Tiles past 2^31 elements and 2^32 bytes of a pool."""
    blocks, hkv = 300000, 8  # 4.9 GB a pool
    free, _ = torch.cuda.mem_get_info()
    if free < 16 << 30:
        pytest.skip("not enough device memory")
    kc = torch.zeros(blocks, hkv, 16, 64, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    t = Trees("bf16", [200], [20], 32, 8, seed=40)
    ids = torch.tensor([blocks - 1 - 17 * i for i in range(t.w.block_tables.shape[1])])
    old = torch.tensor(t.w.block_tables[0].astype(np.int64))
    kc[ids.cuda()] = t.dev[0][old.cuda()]
    vc[ids.cuda()] = t.dev[1][old.cuda()]
    t.check(t.run(dev=[kc, vc], bt=ids.to(torch.int32)[None].cuda()))
