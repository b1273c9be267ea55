"""pa_rope_append_q8 and pa_copy_blocks_q8 against the cache's definition in 64 bits.

Tolerances: scales are equal (the largest magnitudes here are kept away from the powers' edges
where the fp32 rotation could cross them, or are not rotated); rescaled codes are equal; a new
code is within half an e4m3 step of value / scale, plus the fp32 rotation's error bound."""
import numpy as np
import pytest
import torch

from paged_kv_cache_299_gb300 import binding as pa
from paged_kv_cache_299_gb300 import graphs
from paged_kv_cache_299_gb300 import workloads as wl
from _gpu import i32
from _q8 import (E4M3_HALF_STEP, E4M3_SUB_HALF_STEP, angles, needed_scale, quantise, rotate, rotation_error,
                 store_q8, tokens_of)

pytestmark = pytest.mark.gpu


def rows(n, heads, seed, spread=1.0):
    """Rows of unlike size, so that scales grow within a block."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, heads, 64, generator=g)
    x = x * torch.exp(spread * torch.randn(n, heads, 1, generator=g))
    return x.to(torch.bfloat16)


class Cache:
    """An 8-bit cache with random content, on the CPU (float64 codes) and on the GPU."""

    def __init__(self, w, hkv, seed=5):
        g = torch.Generator().manual_seed(seed)
        self.raw = []
        for i in range(2):
            codes, scales = quantise(0.3 * torch.randn(w.num_blocks, hkv, 16, 64, generator=g))
            self.raw.append((codes, scales))
        self.codes = [c.float().double() for c, _ in self.raw]
        self.scales = [s.double() for _, s in self.raw]
        self.kc, self.vc = (c.cuda() for c, _ in self.raw)
        self.ks, self.vs = (s.cuda() for _, s in self.raw)


def check_pool(got_codes, got_scales, codes, scales, where, err):
    """codes: the definition's (new ones unrounded); err [T, H, 64]: bound of the values' error."""
    assert torch.equal(got_scales.cpu().double(), scales)
    got = got_codes.cpu().float().double()
    blk = torch.tensor([b for b, _ in where])
    off = torch.tensor([o for _, o in where])
    new, ref = got[blk, :, off], codes[blk, :, off]
    tol = torch.maximum(ref.abs() * E4M3_HALF_STEP, torch.full_like(ref, E4M3_SUB_HALF_STEP))
    tol = tol + (1 + E4M3_HALF_STEP) * err / scales[blk][..., None]
    bad = (new - ref).abs() > tol
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} new codes out of tolerance"
    got[blk, :, off] = 0
    rest = codes.clone()
    rest[blk, :, off] = 0
    assert torch.equal(got, rest)  # rescaled and untouched codes


def run_case(w, hq, hkv, interleaved=False, rotated=True, one_each=False, extra_rows=0, spread=1.0, strided=False):
    n = int(w.new_lens.sum())
    total = n + extra_rows
    table = angles(int(w.context_lens.max()))
    q, k, v = rows(total, hq, 1), rows(total, hkv, 2, spread), rows(total, hkv, 3, spread)
    c = Cache(w, hkv)
    status = pa.new_device_status()
    pos = torch.tensor([p for _, p in tokens_of(w)])
    qo = torch.full((total, hq, 64), 7.0, dtype=torch.bfloat16, device="cuda") if rotated else None
    if strided:
        fused = torch.cat([q, k, v], dim=1).cuda()
        dq, dk, dv = fused[:, :hq], fused[:, hq:hq + hkv], fused[:, hq + hkv:]
    else:
        dq, dk, dv = q.cuda(), k.cuda(), v.cuda()
    pa.pa_rope_append_q8(dq if rotated else None, dk, dv, table.cuda() if rotated else None, c.kc, c.vc,
                         c.ks, c.vs, i32(w.block_tables), i32(w.context_lens),
                         None if one_each else i32(w.new_start_loc), q_out=qo, interleaved=interleaved,
                         device_status=status)
    assert pa.pa_check_device_status(status) == pa.PA_OK
    kk = rotate(k[:n], table[pos], interleaved) if rotated else k[:n].double()
    err = rotation_error(k[:n], interleaved) if rotated else torch.zeros(n, hkv, 64, dtype=torch.float64)
    where = store_q8(kk, c.codes[0], c.scales[0], w)
    store_q8(v[:n].double(), c.codes[1], c.scales[1], w)
    check_pool(c.kc, c.ks, c.codes[0], c.scales[0], where, err)
    check_pool(c.vc, c.vs, c.codes[1], c.scales[1], where, torch.zeros_like(err))
    if rotated:
        plain_k = torch.zeros(w.num_blocks, hkv, 16, 64, dtype=torch.bfloat16, device="cuda")
        out = pa.pa_rope_append(dq[:n], dk[:n], dv[:n], table.cuda(), plain_k, torch.zeros_like(plain_k),
                                i32(w.block_tables), i32(w.context_lens), i32(w.new_start_loc),
                                interleaved=interleaved)
        assert torch.equal(qo[:n], out) and bool((qo[n:] == 7.0).all())


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("hq,hkv", [(32, 8), (1, 1), (6, 3)])
def test_ragged_chunks(hq, hkv, interleaved):
    w = wl.make_workload("ragged", [0, 5, 31, 200, 16, 15], [17, 1, 40, 3, 16, 2], seed=hq, pool_slack=0.4)
    run_case(w, hq, hkv, interleaved)


@pytest.mark.parametrize("hist", range(16))
def test_every_start_in_a_block_and_every_length(hist):
    new = np.arange(1, 36)
    w = wl.make_workload("starts", np.full(35, hist), new, seed=hist, pool_slack=0.2)
    run_case(w, 2, 2, rotated=hist % 2 == 0)


@pytest.mark.parametrize("seqs", [1, 5, 300])
def test_one_token_per_sequence(seqs):
    hist = np.random.default_rng(seqs).integers(0, 100, size=seqs)
    w = wl.make_workload("steps", hist, np.ones(seqs, np.int32), seed=seqs, pool_slack=0.2)
    run_case(w, 8, 2, one_each=True)
    run_case(w, 8, 2, strided=True)
    run_case(w, 0, 2, rotated=False, one_each=True)


def test_empty_sequences_and_padding_rows():
    w = wl.make_workload("empty", [4, 9, 0, 50, 3], [0, 12, 0, 2, 0], seed=8, pool_slack=0.5)
    run_case(w, 8, 8, extra_rows=5)
    run_case(w, 8, 8, extra_rows=40, strided=True)


@pytest.mark.parametrize("spread", [0.0, 8.0])
def test_scales_over_a_wide_range(spread):
    """spread 8: magnitudes over e^+-24; rescaled tokens fall to subnormal codes and to zero."""
    w = wl.make_workload("wide", [0, 3, 14], [64, 20, 30], seed=9, pool_slack=0.5)
    run_case(w, 4, 4, rotated=False, spread=spread)


def one_block(values, status=None, table=None):
    """Append [n, 64] values as n tokens of one head, token by token; returns codes and scale."""
    c = pa.new_q8_cache(2, 1)
    bt = i32(np.array([[1]]))
    for t in range(len(values)):
        pa.pa_rope_append_q8(None, values[t].view(1, 1, 64).cuda(), values[t].view(1, 1, 64).cuda(), table, *c, bt,
                             i32([t + 1]), None, device_status=status)
    if table is None:  # keys and values are stored alike
        assert torch.equal(c[0].view(torch.uint8), c[1].view(torch.uint8)) and torch.equal(c[2], c[3])
    return c[0][1, 0].cpu().float(), float(c[2][1, 0])


def test_scale_edges():
    """The largest magnitude at, just below and just above 448 * 2^k; zeros; the extremes of
    bf16; a growing block."""
    def row(x):
        r = torch.zeros(64, dtype=torch.bfloat16)
        r[7] = x
        return r

    for k in (-20, -3, 0, 5, 100):
        for mul in (448.0, 446.0, 450.0, 256.0, 255.0, 512.0):
            x = float(torch.tensor(mul * 2.0 ** k, dtype=torch.bfloat16))
            codes, scale = one_block([row(-x)])
            assert scale == needed_scale(x)
            assert abs(float(codes[0, 7]) * scale + x) <= E4M3_HALF_STEP * x
    assert one_block([row(0.0)])[1] == 2.0 ** -126
    tiny = float(torch.finfo(torch.bfloat16).smallest_normal)
    assert one_block([row(tiny)])[1] == 2.0 ** -126
    codes, scale = one_block([row(torch.finfo(torch.bfloat16).max)])
    assert scale == 2.0 ** 120 and float(codes[0, 7]) == 256.0  # 255 * 2^120, to three bits
    codes, scale = one_block([row(1.0), row(1000.0), row(3.0)])
    assert scale == 4.0 and [float(codes[i, 7]) for i in range(3)] == [0.25, 256.0, 0.75]
    # token 0 again starts the block anew, whatever it held
    c = pa.new_q8_cache(1, 1)
    bt = i32(np.array([[0]]))
    for x, t in ((1000.0, 0), (1.0, 1), (1.0, 0)):
        r = row(x).view(1, 1, 64).cuda()
        pa.pa_rope_append_q8(None, r, r, None, *c, bt, i32([t + 1]))
    assert float(c[2]) == 2.0 ** -8


def test_non_finite_values():
    status = pa.new_device_status()
    r = torch.ones(64, dtype=torch.bfloat16)
    r[3], r[4], r[5] = float("nan"), float("inf"), float("-inf")
    codes, scale = one_block([r], status)
    assert scale == 2.0 ** -8 and codes[0, 3] == 0 and codes[0, 4] == 448 and codes[0, 5] == -448
    assert bool((codes[0, 6:] == 256).all())
    assert int(status.item()) == pa.DEVFLAG_NONFINITE
    assert pa.pa_check_device_status(status) == pa.PA_ERR_DEVICE_VALUE
    # rotated: infinities meet and make NaN; nothing but codes comes out
    status.zero_()
    codes, _ = one_block([r], status, angles(4).cuda())
    assert torch.isfinite(codes).all() and int(status.item()) == pa.DEVFLAG_NONFINITE


def test_bad_entries_are_reported_and_skipped():
    w = wl.make_workload("bad", [10, 20], [3, 4], seed=11, pool_slack=0.5)
    k = rows(7, 2, 1).cuda()

    def go(bt, ctx, table=None, scales=None):
        status, c = pa.new_device_status(), pa.new_q8_cache(w.num_blocks, 2)
        if scales is not None:
            c[2].fill_(scales)
        pa.pa_rope_append_q8(None, k, k, table, *c, i32(bt), i32(ctx), i32([0, 3, 7]), device_status=status)
        return int(status.item()), int((c[0].float() != 0).any(dim=3).sum())

    bt = w.block_tables.copy()
    bt[0, 0] = -1
    assert go(bt, w.context_lens) == (pa.DEVFLAG_BAD_BLOCK, 4 * 2)
    assert go(w.block_tables, [2, 24]) == (pa.DEVFLAG_BAD_CONTEXT, 4 * 2)
    assert go(w.block_tables, [13, 5000]) == (pa.DEVFLAG_BAD_CONTEXT, 3 * 2)
    assert go(w.block_tables, w.context_lens, angles(23).cuda()) == (pa.DEVFLAG_BAD_CONTEXT, 3 * 2)
    for bad in (0.0, -1.0, float("nan"), float("inf")):  # both blocks hold earlier tokens
        assert go(w.block_tables, w.context_lens, None, bad) == (pa.DEVFLAG_BAD_SCALE, 0)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("hq,hkv", [(2, 1), (6, 3), (16, 8), (9, 9), (20, 20)])
def test_one_token_form_equals_chunks_of_one(hq, hkv, interleaved):
    """Without query_start_loc, against the checked definition and bit for bit against chunks of
    one token, with blocks that start, grow, hold a bad scale and receive non-finite rows."""
    n = 70
    w = wl.make_workload("ones", np.arange(n) % 37, np.ones(n, int), seed=hkv, pool_slack=0.3)
    run_case(w, hq, hkv, interleaved, one_each=True, spread=2.5)
    table = angles(40).cuda()
    c = Cache(w, hkv)
    k, v = rows(n, hkv, 2, 2.5), rows(n, hkv, 3, 2.5)
    k[5, 0, 3], v[6, -1, 60], v[7, 0, 0] = float("nan"), float("inf"), float("-inf")
    c.ks[int(w.block_tables[20, 1]), -1] = -1.0  # position 20
    c.vs[int(w.block_tables[16, 1]), 0] = float("nan")  # position 16 starts its block
    c.vs[int(w.block_tables[40, 0]), 0] = 0.0  # position 3
    bt = w.block_tables.copy()
    bt[9, 0] = w.num_blocks
    ctx = w.context_lens.copy()
    ctx[30], ctx[31], ctx[32] = 41, -1, 5000  # beyond the angles, negative, beyond the table row
    got = []
    for qsl in (None, i32(np.arange(n + 1))):
        cache = [x.clone() for x in (c.kc, c.vc, c.ks, c.vs)]
        status = pa.new_device_status()
        pa.pa_rope_append_q8(None, k.cuda(), v.cuda(), table, *cache, i32(bt), i32(ctx), qsl,
                             interleaved=interleaved, device_status=status)
        got.append(([x.cpu() for x in cache], int(status.item())))
    assert got[0][1] == got[1][1] == (pa.DEVFLAG_NONFINITE | pa.DEVFLAG_BAD_SCALE | pa.DEVFLAG_BAD_BLOCK
                                      | pa.DEVFLAG_BAD_CONTEXT)
    for a, b in zip(got[0][0], got[1][0]):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("starts", [[0, 3, 9], [0, 7, 9], [0, 9, 12]])
def test_rows_past_the_buffer_are_reported(starts):
    """Seven rows, and sequences that claim more: what lies past the buffer is reported and skipped."""
    w = wl.make_workload("past", [10, 20], [9, 9], seed=11, pool_slack=0.5)
    k = rows(7, 2, 1).cuda()
    ctx = [10 + starts[1], 20 + starts[2] - starts[1]]
    for table in (None, angles(64).cuda()):
        status, c = pa.new_device_status(), pa.new_q8_cache(w.num_blocks, 2)
        pa.pa_rope_append_q8(None, k, k, table, *c, i32(w.block_tables), i32(ctx), i32(starts), device_status=status)
        assert int(status.item()) == pa.DEVFLAG_BAD_CONTEXT
        stored = 0 if starts[1] > 7 else starts[1]  # the first sequence, where it ends within the rows
        assert int((c[0].float() != 0).any(dim=3).sum()) == 2 * stored


def test_repeat_graph_and_stream_are_bit_identical():
    w = wl.make_workload("side", [11, 300], [100, 257], seed=13, pool_slack=0.2)
    n = int(w.new_lens.sum())
    q, k, v = rows(n, 32, 1).cuda(), rows(n, 8, 2).cuda(), rows(n, 8, 3).cuda()
    table, bt, ctx, qsl = angles(600).cuda(), i32(w.block_tables), i32(w.context_lens), i32(w.new_start_loc)
    results = []
    for how in ("call", "twice", "stream", "graph"):
        c, out = Cache(w, 8), torch.empty_like(q)
        first = [x.clone() for x in (c.kc, c.vc, c.ks, c.vs)]

        def step(stream=None):
            pa.pa_rope_append_q8(q, k, v, table, c.kc, c.vc, c.ks, c.vs, bt, ctx, qsl, q_out=out, stream=stream)

        torch.cuda.synchronize()
        if how == "graph":
            graph = graphs.StepGraph(step)
            for x, y in zip((c.kc, c.vc, c.ks, c.vs), first):
                x.copy_(y)
            graph.replay()
        else:
            step(torch.cuda.Stream() if how == "stream" else None)
            if how == "twice":  # the same tokens again change nothing
                step()
        torch.cuda.synchronize()
        results.append([x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x
                        for x in (out, c.kc, c.vc, c.ks, c.vs)])
    for other in results[1:]:
        assert all(torch.equal(x, y) for x, y in zip(results[0], other))


@pytest.mark.parametrize("hkv", [1, 3, 8])
def test_copy_blocks_is_bit_exact(hkv):
    g = torch.Generator().manual_seed(hkv)
    nb = 40
    pools = [torch.randint(0, 256, (nb, hkv, 16, 64), generator=g, dtype=torch.uint8) for _ in range(2)]
    scales = [torch.randn(nb, hkv, generator=g) for _ in range(2)]
    perm = torch.randperm(nb, generator=g)
    pairs = torch.stack([perm[:12], perm[12:24]], dim=1).contiguous()
    pairs = torch.cat([pairs, torch.tensor([[0, nb], [-1, 3], [nb, 2]])])  # the last three are bad
    dev = [p.cuda().view(torch.float8_e4m3fn) for p in pools] + [s.cuda() for s in scales]
    status = pa.new_device_status()
    pa.pa_copy_blocks_q8(*dev, pairs.cuda(), device_status=status)
    assert pa.pa_check_device_status(status) == pa.PA_ERR_DEVICE_INDEX
    for got, ref in zip(dev, pools + scales):
        ref = ref.clone()
        for s, d in pairs[:12].tolist():
            ref[d] = ref[s]
        got = got.cpu().view(torch.uint8) if got.dtype == torch.float8_e4m3fn else got.cpu()
        assert torch.equal(got, ref)
    pa.pa_copy_blocks_q8(*dev, pairs[:0].cuda())  # nothing to copy
