"""A run of the operators together, as a serving loop uses them: a tree of drafted tokens is appended at
the positions of its depths, attended under its mask, and the accepted path kept; the conversation that
results agrees with one in which the accepted tokens had been appended one after the other."""
import random

import numpy as np
import pytest
import torch

from paged_kv_cache_299_gb300 import binding as pa
from _gpu import i32
from _q8 import angles, attend
from _tree import attend_tree

pytestmark = pytest.mark.gpu
HQ, HKV = 8, 2


class Loop:
    """Sequences that grow by speculation over pools of one kind, on device blocks of the block manager."""

    def __init__(self, pool, seqs, blocks=400, seed=0):
        self.pool, self.n = pool, seqs
        self.rng = random.Random(seed)
        self.g = torch.Generator().manual_seed(seed)
        self.bm = pa.BlockManager(blocks)
        if pool == "q8":
            self.dev = list(pa.new_q8_cache(blocks, HKV))
        else:
            self.dev = [torch.full((blocks, HKV, 16, 64), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        self.table = angles(600).cuda()
        self.len = [0] * seqs
        self.largest = 0.0
        self.status = pa.new_device_status()
        self.ws = torch.zeros(pa.pa_tree_workspace_size(), dtype=torch.uint8, device="cuda")
        self.log = [[] for _ in range(seqs)]  # (key row, value row, position) of every token kept
        for s in range(seqs):
            self.bm.add_sequence(s)

    def tables(self, lens):
        """Block tables with room for `lens` tokens of every sequence."""
        for s, n in enumerate(lens):
            have = self.bm.num_tokens(s)
            if n > have:
                assert self.bm.append_tokens(s, n - have) == []
        width = max(1, max(-(-self.bm.num_tokens(s) // 16) for s in range(self.n)))
        return i32([self.bm.block_table(s, width)[0] for s in range(self.n)])

    def rows(self, n, heads):
        x = torch.randn(n, heads, 64, generator=self.g).to(torch.bfloat16)
        self.largest = max(self.largest, float(x.abs().max())) if n else self.largest
        return x

    def append(self, counts, positions):
        """New tokens of every sequence; their (q rotated, q, k, v)."""
        n = sum(counts)
        q, k, v = self.rows(n, HQ), self.rows(n, HKV), self.rows(n, HKV)
        ctx = [a + b for a, b in zip(self.len, counts)]
        bt = self.tables(ctx)
        f = pa.pa_rope_append_at_q8 if self.pool == "q8" else pa.pa_rope_append_at
        starts = i32(np.concatenate([[0], np.cumsum(counts)]))
        out = f(q.cuda(), k.cuda(), v.cuda(), self.table, i32([positions]), *self.dev, bt, i32(ctx), starts,
                device_status=self.status)
        return out, k, v, bt, ctx, starts

    def values(self):
        """The pools as float64."""
        if self.pool == "q8":
            return [c.cpu().float().double() * s.cpu().double()[..., None, None]
                    for c, s in zip(self.dev[:2], self.dev[2:])]
        return [x.cpu().double() for x in self.dev]


@pytest.mark.parametrize("pool", ["bf16", "q8"])
def test_a_conversation_by_speculation(pool):
    loop = Loop(pool, 5, seed=3)
    # prompts, at the positions of their slots
    counts = [0, 1, 15, 40, 130]
    _, k, v, *_ = loop.append(counts, [i for n in counts for i in range(n)])
    row = 0
    for s, n in enumerate(counts):
        loop.log[s] = [(k[row + i], v[row + i], i) for i in range(n)]
        row += n
    loop.len = list(counts)
    for step in range(6):
        # a tree per sequence: parents, depths, ancestors
        counts = [loop.rng.randint(1, 40) for _ in range(loop.n)]
        seen = torch.zeros(sum(counts), max(counts), dtype=torch.bool)
        positions, parents, row = [], [], 0
        for s, n in enumerate(counts):
            depth = []
            parents.append([loop.rng.randint(max(-1, i - 4), i - 1) for i in range(n)])
            for i, p in enumerate(parents[s]):
                depth.append(depth[p] + 1 if p >= 0 else 0)
                if p >= 0:
                    seen[row + i] |= seen[row + p]
                seen[row + i, i] = True
            positions += [loop.len[s] + d for d in depth]
            row += n
        q, k, v, bt, ctx, starts = loop.append(counts, positions)
        out = torch.empty_like(q)
        f = pa.pa_tree_attention_q8 if pool == "q8" else pa.pa_tree_attention
        f(out, q, pa.pack_tree_mask(seen).cuda(), starts, max(counts), *loop.dev, bt, i32(ctx), 0.125, workspace=loop.ws,
          device_status=loop.status)
        k64, v64 = loop.values()
        bits = [[sum(1 << j for j in range(n) if seen[at + i, j]) for i in range(n)]
                for at, n in zip(np.cumsum([0] + counts[:-1]).tolist(), counts)]
        ref, tol = attend_tree(q.cpu(), k64.nan_to_num(0), v64.nan_to_num(0), bt.cpu().numpy(), ctx, counts, bits, 0.125)
        assert ((out.cpu().double() - ref).abs() <= tol).all()
        # the path to a node of every sequence is accepted
        kept, row = [], 0
        for s, n in enumerate(counts):
            path, i = [], loop.rng.randint(-1, n - 1)
            while i >= 0:
                path.append(i)
                i = parents[s][i]
            path.reverse()
            kept.append(path)
            loop.log[s] += [(k[row + i], v[row + i], loop.len[s] + d) for d, i in enumerate(path)]
            row += n
        f = pa.pa_compact_tokens_q8 if pool == "q8" else pa.pa_compact_tokens
        f(i32([i for path in kept for i in path]), i32(np.concatenate([[0], np.cumsum([len(p) for p in kept])])),
          i32(loop.len), max(len(p) for p in kept), *loop.dev, bt, device_status=loop.status)
        loop.len = [a + len(p) for a, p in zip(loop.len, kept)]
    assert pa.pa_check_device_status(loop.status) == pa.PA_OK

    # the same tokens, appended without detours
    plain = Loop(pool, 5, seed=4)
    bt = plain.tables(loop.len)
    for s in range(loop.n):
        if loop.len[s] == 0:
            continue
        pos = [p for _, _, p in loop.log[s]]
        assert pos == list(range(loop.len[s]))
        f = pa.pa_rope_append_q8 if pool == "q8" else pa.pa_rope_append
        f(None, torch.stack([x for x, _, _ in loop.log[s]]).cuda(), torch.stack([x for _, x, _ in loop.log[s]]).cuda(),
          plain.table, *plain.dev, bt[s:s + 1].contiguous(), i32([loop.len[s]]), i32([0, loop.len[s]]))
    mine, theirs = loop.values(), plain.values()
    old = loop.tables(loop.len)
    for s, n in enumerate(loop.len):
        for p in range(n):
            a = [x[int(old[s, p // 16]), :, p % 16] for x in mine]
            b = [x[int(bt[s, p // 16]), :, p % 16] for x in theirs]
            for x, y in zip(a, b):
                if pool == "bf16":
                    assert torch.equal(x, y)
                else:
                    # Both are roundings of one value, each by at most 2^-4 of it: changes of scale by powers
                    # of two are exact down to the subnormal codes.  There a rounding is off by 2^-10 of the
                    # scale, once when drafted, once when moved, once in the other cache, and at each growth of
                    # the scale (which doubles: twice the last).  No scale exceeds 2 / 448 of the largest
                    # value, and a rotation grows none beyond sqrt(2).
                    scale = 2 / 448 * 1.5 * loop.largest
                    assert ((x - y).abs() <= 2.3 * 2.0 ** -4 * y.abs() + 5 * 2.0 ** -10 * scale).all()

    # and the next token attends alike over both
    q = loop.rows(loop.n, HQ).cuda()
    most = max(loop.len)
    outs = []
    for x, tables in ((loop, old), (plain, bt)):
        out = torch.empty_like(q)
        if pool == "q8":
            pa.pa_decode_q8(out, q, *x.dev, tables, i32(loop.len), 0.125, most)
        else:
            pa.pa_decode(out, q, *x.dev, tables, i32(loop.len), 0.125, most)
        outs.append(out.cpu().float())
    if pool == "bf16":
        assert torch.equal(*outs)
    else:
        for out, values, tables in ((outs[0], mine, old), (outs[1], theirs, bt)):
            ref, tol = attend(q.cpu(), *(x.nan_to_num(0) for x in values), tables.cpu().numpy(), loop.len, 0.125)
            assert ((out.double() - ref).abs() <= tol).all()
