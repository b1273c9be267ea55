"""pa_rope_append: the rotated queries and the bf16 pools against the rotation in 64 bits.

Tolerance: half a bf16 step of the rotated value (values are stored as they are and must be
equal) plus the bound of the fp32 rotation's own error."""
import numpy as np
import pytest
import torch

from paged_kv_cache_299_gb300 import binding as pa
from paged_kv_cache_299_gb300 import graphs
from paged_kv_cache_299_gb300 import workloads as wl
from _gpu import GpuStep, bits, i32, oracle_step, host_vals
from _q8 import BF16_HALF_STEP, angles, rotate, rotation_error, tokens_of
from _util import ATOL_MAX, ATOL_MEAN, errors

pytestmark = pytest.mark.gpu


def rows(n, heads, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(n, heads, 64, generator=g).to(torch.bfloat16)


def check_rotated(got, x, table, positions, interleaved):
    ref = rotate(x, table[positions], interleaved)
    tol = BF16_HALF_STEP * ref.abs() + rotation_error(x, interleaved) * (1 + BF16_HALF_STEP)
    bad = (got.double() - ref).abs() > tol
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} values out of tolerance"


def run_case(w, hq, hkv, interleaved, strided=False, in_place=False, one_each=False, extra_rows=0):
    """One append over a random pool; checks queries, pools, and that nothing else changed."""
    n = int(w.new_lens.sum())
    table = angles(int(w.context_lens.max()))
    q, k, v = rows(n + extra_rows, hq, 1), rows(n + extra_rows, hkv, 2), rows(n + extra_rows, hkv, 3)
    if strided:
        fused = torch.cat([q, k, v], dim=1).cuda()
        dq, dk, dv = fused[:, :hq], fused[:, hq:hq + hkv], fused[:, hq + hkv:]
    else:
        fused = None
        dq, dk, dv = q.cuda(), k.cuda(), v.cuda()
    pool = rows(w.num_blocks * 16, hkv, 4).view(w.num_blocks, 16, hkv, 64).transpose(1, 2).contiguous()
    kc, vc = pool.cuda(), pool.cuda()
    status = pa.new_device_status()
    sentinel = torch.full((n + extra_rows, hq, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    out = pa.pa_rope_append(dq, dk, dv, table.cuda(), kc, vc, i32(w.block_tables), i32(w.context_lens),
                            None if one_each else i32(w.new_start_loc),
                            q_out=dq if in_place else sentinel, interleaved=interleaved,
                            device_status=status)
    assert pa.pa_check_device_status(status) == pa.PA_OK
    where = tokens_of(w)
    pos = torch.tensor([p for _, p in where], dtype=torch.int64)
    got = out.cpu()
    check_rotated(got[:n], q[:n], table, pos, interleaved)
    if extra_rows:  # padding rows are left alone
        assert torch.equal(got[n:], q[n:] if in_place else sentinel.cpu()[n:])
    gk, gv = kc.cpu(), vc.cpu()
    blk = torch.tensor([int(w.block_tables[s, p // 16]) for s, p in where], dtype=torch.int64)
    off = pos % 16
    check_rotated(gk[blk, :, off], k[:n], table, pos, interleaved)
    assert torch.equal(gv[blk, :, off], v[:n])
    gk[blk, :, off] = pool[blk, :, off]
    gv[blk, :, off] = pool[blk, :, off]
    assert torch.equal(gk, pool) and torch.equal(gv, pool)  # every other slot untouched
    if fused is not None:
        assert torch.equal(fused[:, hq:].cpu(), torch.cat([k, v], dim=1))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("hq,hkv", [(32, 8), (1, 1), (6, 3), (5, 2)])
def test_ragged_chunks(hq, hkv, interleaved):
    w = wl.make_workload("ragged", [0, 5, 31, 200, 16], [17, 1, 40, 3, 16], seed=hq, pool_slack=0.4)
    run_case(w, hq, hkv, interleaved)


@pytest.mark.parametrize("interleaved", [False, True])
def test_strided_rows_of_a_fused_projection(interleaved):
    w = wl.make_workload("strided", [3, 0, 77], [30, 1, 9], seed=3, pool_slack=0.4)
    run_case(w, 8, 2, interleaved, strided=True)
    run_case(w, 8, 2, interleaved, strided=True, in_place=True)
    run_case(w, 8, 2, interleaved, in_place=True)


@pytest.mark.parametrize("seqs", [1, 2, 33, 700])
def test_one_token_per_sequence(seqs):
    hist = np.random.default_rng(seqs).integers(0, 300, size=seqs)
    w = wl.make_workload("steps", hist, np.ones(seqs, np.int32), seed=seqs, pool_slack=0.2)
    run_case(w, 32, 8, False, one_each=True)
    run_case(w, 4, 4, True)


def test_empty_sequences_and_padding_rows():
    w = wl.make_workload("empty", [4, 9, 0, 50], [0, 12, 0, 2], seed=8, pool_slack=0.5)
    run_case(w, 8, 8, False, extra_rows=5)
    run_case(w, 8, 8, True, extra_rows=1, in_place=True)


def test_far_positions():
    w = wl.make_workload("far", [131000, 70000], [72, 1], seed=9, pool_slack=0.1)
    run_case(w, 4, 1, False)


def test_keys_and_values_only():
    w = wl.make_workload("kv", [7, 0], [20, 1], seed=10, pool_slack=0.5)
    n = int(w.new_lens.sum())
    k, v, table = rows(n, 8, 1), rows(n, 8, 2), angles(64)
    kc = torch.zeros(w.num_blocks, 8, 16, 64, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    assert pa.pa_rope_append(None, k.cuda(), v.cuda(), table.cuda(), kc, vc, i32(w.block_tables),
                             i32(w.context_lens), i32(w.new_start_loc)) is None
    pos = torch.tensor([p for _, p in tokens_of(w)])
    blk = torch.tensor([int(w.block_tables[s, p // 16]) for s, p in tokens_of(w)])
    check_rotated(kc.cpu()[blk, :, pos % 16], k, table, pos, False)


def test_bad_entries_are_reported_and_skipped():
    w = wl.make_workload("bad", [10, 20], [3, 4], seed=11, pool_slack=0.5)
    k = rows(7, 2, 1).cuda()
    table = angles(64).cuda()
    zero = torch.zeros(w.num_blocks, 2, 16, 64, dtype=torch.bfloat16, device="cuda")

    def go(bt, ctx, tab=table):
        status, kc, vc = pa.new_device_status(), zero.clone(), zero.clone()
        pa.pa_rope_append(None, k, k, tab, kc, vc, i32(bt), i32(ctx), i32([0, 3, 7]), device_status=status)
        return int(status.item()), kc

    bt = w.block_tables.copy()
    bt[0, 0] = w.num_blocks  # positions 10..12 of sequence 0
    flag, kc = go(bt, w.context_lens)
    assert flag == pa.DEVFLAG_BAD_BLOCK
    assert int((kc != 0).any(dim=3).sum()) == 4 * 2  # the other sequence's four tokens
    flag, kc = go(w.block_tables, [2, 24])  # a context shorter than its rows
    assert flag == pa.DEVFLAG_BAD_CONTEXT
    flag, _ = go(w.block_tables, [13, 5000])  # beyond the block-table row
    assert flag == pa.DEVFLAG_BAD_CONTEXT
    flag, kc = go(w.block_tables, w.context_lens, table[:22].contiguous())  # beyond the angles
    assert flag == pa.DEVFLAG_BAD_CONTEXT
    assert int((kc != 0).any(dim=3).sum()) == (3 + 2) * 2


@pytest.mark.parametrize("starts", [[0, 3, 9], [0, 7, 9], [0, 9, 12]])
def test_rows_past_the_buffer_are_reported(starts):
    """Seven rows, and sequences that claim more: what lies past the buffer is reported and skipped."""
    w = wl.make_workload("past", [10, 20], [9, 9], seed=11, pool_slack=0.5)
    k, table = rows(7, 2, 1).cuda(), angles(64).cuda()
    status = pa.new_device_status()
    kc = torch.zeros(w.num_blocks, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    ctx = [10 + starts[1], 20 + starts[2] - starts[1]]
    pa.pa_rope_append(None, k, k, table, kc, vc, i32(w.block_tables), i32(ctx), i32(starts), device_status=status)
    assert int(status.item()) == pa.DEVFLAG_BAD_CONTEXT
    stored = 0 if starts[1] > 7 else starts[1]  # the first sequence, where it ends within the rows
    assert int((kc != 0).any(dim=3).sum()) == 2 * stored


def test_non_finite_rows_pass_through():
    """bf16 pools hold what the arithmetic gives: a NaN stays in its pair, the rest is exact."""
    w = wl.make_workload("nan", [0], [4], seed=12, pool_slack=1.0)
    k = rows(4, 1, 1)
    k[1, 0, 3] = float("nan")
    k[2, 0, 5] = float("inf")
    kc = torch.zeros(w.num_blocks, 1, 16, 64, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    pa.pa_rope_append(None, k.cuda(), k.cuda(), angles(8).cuda(), kc, vc, i32(w.block_tables), i32([4]), i32([0, 4]))
    b = int(w.block_tables[0, 0])
    nan = torch.isnan(kc.cpu()[b, 0, 1])
    assert nan.nonzero().flatten().tolist() == [3, 35]
    assert not torch.isfinite(kc.cpu()[b, 0, 2])[[5, 37]].any()
    assert torch.isfinite(kc.cpu()[b, 0, 2]).sum() == 62
    assert torch.equal(vc.cpu()[b, 0, :4].view(torch.int16), k[:, 0].view(torch.int16))


def test_same_pools_as_store_and_decode_on_unrotated_rows():
    """With all angles zero the append stores what slot mapping and store do, bit for bit, and
    decode over its pools agrees with the oracle; captured and replayed, it gives the same."""
    w = wl.random_small(77, num_seqs=6, max_ctx=300)
    a = GpuStep(w)
    b = GpuStep(w, store_new=False)
    flat = torch.zeros(300, 64, device="cuda")
    flat[:, :32] = 1.0
    q = b.vals["q_decode"]
    q_out = torch.empty_like(q)

    def step():
        pa.pa_rope_append(q, b.vals["new_k"], b.vals["new_v"], flat, b.kc, b.vc, b.bt, b.ctx, None, q_out=q_out,
                          device_status=b.status)

    graph = graphs.StepGraph(step)
    b.kc.copy_(GpuStep(w, store_new=False).kc)  # undo the warm-up's store
    q_out.zero_()
    graph.replay()
    assert torch.equal(q_out, q)
    assert np.array_equal(bits(a.kc), bits(b.kc)) and np.array_equal(bits(a.vc), bits(b.vc))
    ref = oracle_step(w, host_vals(b.vals))
    mx, mean = errors(b.decode().float().cpu().numpy(), ref["decode"])
    assert mx <= ATOL_MAX and mean <= ATOL_MEAN
    assert b.check_status() == pa.PA_OK


def test_side_stream_and_repeat_are_bit_identical():
    w = wl.make_workload("side", [11, 300], [100, 257], seed=13, pool_slack=0.2)
    n = int(w.new_lens.sum())
    q, k, v = rows(n, 32, 1).cuda(), rows(n, 8, 2).cuda(), rows(n, 8, 3).cuda()
    table = angles(600).cuda()
    results = []
    for stream in (None, torch.cuda.Stream(), torch.cuda.Stream()):
        kc = torch.zeros(w.num_blocks, 8, 16, 64, dtype=torch.bfloat16, device="cuda")
        vc = torch.zeros_like(kc)
        bt, ctx, qsl = i32(w.block_tables), i32(w.context_lens), i32(w.new_start_loc)
        torch.cuda.synchronize()
        out = pa.pa_rope_append(q, k, v, table, kc, vc, bt, ctx, qsl, stream=stream)
        torch.cuda.synchronize()
        results.append((out, kc, vc))
    for other in results[1:]:
        assert all(torch.equal(x, y) for x, y in zip(results[0], other))
