"""pa_rope_append_at and its 8-bit form: rotation by positions of the tokens' own, on up to four axes,
against the rotation in 64 bits (tolerances as for the appends that rotate by the slots' positions)."""
import numpy as np
import pytest
import torch

from paged_kv_cache_299_gb300 import binding as pa
from paged_kv_cache_299_gb300 import graphs
from paged_kv_cache_299_gb300 import workloads as wl
from _gpu import i32
from _q8 import (BF16_HALF_STEP, E4M3_HALF_STEP, E4M3_SUB_HALF_STEP, angles, rotate, rotation_error, store_q8,
                 tokens_of)

pytestmark = pytest.mark.gpu
TABLE = 500
AXES = {"one": None, "sections": [0] * 8 + [1] * 12 + [2] * 12, "odd sections": [0] * 5 + [1] * 13 + [2] * 14,
        "cycled": [i % 3 for i in range(32)], "four": [3 - i % 4 for i in range(32)], "last": [2] * 32}


def rows(n, heads, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(n, heads, 64, generator=g).to(torch.bfloat16)


def positions_for(n, axes, seed):
    return torch.from_numpy(np.random.default_rng(seed).integers(0, TABLE, (axes, n)).astype(np.int32))


def table_rows(pos, pair_axes):
    """[T, 64] of the angles each pair of a token turns by."""
    table = angles(TABLE)
    axis = torch.tensor(pair_axes or [0] * 32)
    at = pos.long()[axis].t()  # [T, 32]
    pair = torch.arange(32)
    return torch.cat([table[at, pair], table[at, 32 + pair]], dim=1)


def run_case(w, hq, hkv, q8, name, interleaved=False, strided=False, in_place=False, one_each=False, extra=0):
    n = int(w.new_lens.sum())
    pair_axes = AXES[name]
    axes = 1 if pair_axes is None else 4 if name == "four" else 3
    pos = positions_for(n + extra, axes, 5)
    q, k, v = rows(n + extra, hq, 1), rows(n + extra, hkv, 2), rows(n + extra, hkv, 3)
    if strided:
        fused = torch.cat([q, k, v], dim=1).cuda()
        dq, dk, dv = fused[:, :hq], fused[:, hq:hq + hkv], fused[:, hq + hkv:]
    else:
        dq, dk, dv = q.cuda(), k.cuda(), v.cuda()
    sentinel = torch.full((n + extra, hq, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    status = pa.new_device_status()
    tail = (i32(w.block_tables), i32(w.context_lens), None if one_each else i32(w.new_start_loc))
    kw = dict(pair_axes=pair_axes, q_out=dq if in_place else sentinel, interleaved=interleaved, device_status=status)
    turn = table_rows(pos[:, :n], pair_axes)
    where = tokens_of(w)
    if q8:
        g = torch.Generator().manual_seed(4)
        codes = (100 * torch.randn(w.num_blocks, hkv, 16, 64, generator=g)).to(torch.float8_e4m3fn)
        scales = torch.exp2(torch.randint(-9, 3, (w.num_blocks, hkv), generator=g).float())
        dev = [codes.cuda(), codes.cuda(), scales.cuda(), scales.cuda()]
        out = pa.pa_rope_append_at_q8(dq, dk, dv, angles(TABLE).cuda(), pos.cuda(), *dev, *tail, **kw)
    else:
        pool = rows(w.num_blocks * 16, hkv, 4).view(w.num_blocks, 16, hkv, 64).transpose(1, 2).contiguous()
        dev = [pool.cuda(), pool.cuda()]
        out = pa.pa_rope_append_at(dq, dk, dv, angles(TABLE).cuda(), pos.cuda(), *dev, *tail, **kw)
    assert pa.pa_check_device_status(status) == pa.PA_OK
    got = out.cpu()
    if extra:
        assert torch.equal(got[n:], q[n:] if in_place else sentinel.cpu()[n:])

    def rotated(got, x, factor=BF16_HALF_STEP):
        ref = rotate(x, turn, interleaved)
        tol = factor * ref.abs() + rotation_error(x, interleaved) * (1 + factor)
        assert not ((got.double() - ref).abs() > tol).any()

    rotated(got[:n], q[:n])
    if q8:
        for i, x in enumerate((rotate(k[:n], turn, interleaved), v[:n].double())):
            err = rotation_error(k[:n], interleaved) if i == 0 else torch.zeros_like(x)
            want, sc = codes.float().double(), scales.double().clone()
            places = store_q8(x, want, sc, w)
            now = dev[2 + i].cpu().double()
            assert torch.equal(now, sc)  # (random values: none stands at a border of scales)
            have = dev[i].cpu().float().double()
            for t, (b, o) in enumerate(places):
                ref = want[b, :, o]
                tol = (E4M3_HALF_STEP * ref.abs()).clamp(min=E4M3_SUB_HALF_STEP) + 1.25 * err[t] / now[b][:, None]
                assert ((have[b, :, o] - ref).abs() <= tol).all()
                have[b, :, o] = want[b, :, o] = 0
            # (a few of the pool's random codes are no numbers, and stay that)
            assert torch.equal(have.nan_to_num(1e9), want.nan_to_num(1e9))
        return
    blk = torch.tensor([int(w.block_tables[s, p // 16]) for s, p in where], dtype=torch.int64)
    off = torch.tensor([p % 16 for _, p in where], dtype=torch.int64)
    gk, gv = dev[0].cpu(), dev[1].cpu()
    rotated(gk[blk, :, off], k[:n])
    assert torch.equal(gv[blk, :, off], v[:n])
    gk[blk, :, off] = pool[blk, :, off]
    gv[blk, :, off] = pool[blk, :, off]
    assert torch.equal(gk, pool) and torch.equal(gv, pool)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("name", list(AXES))
def test_axes(q8, interleaved, name):
    w = wl.make_workload("ragged", [0, 5, 31, 200, 16], [17, 1, 40, 3, 16], seed=2, pool_slack=0.4)
    run_case(w, 8, 2, q8, name, interleaved)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("hq,hkv", [(32, 8), (1, 1), (6, 3), (5, 2)])
def test_head_layouts(q8, hq, hkv):
    w = wl.make_workload("heads", [7, 0, 90], [33, 2, 12], seed=hq, pool_slack=0.4)
    run_case(w, hq, hkv, q8, "sections")
    run_case(w, hq, hkv, q8, "cycled", True, strided=True)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("seqs", [1, 33, 300])
def test_one_token_per_sequence(q8, seqs):
    hist = np.random.default_rng(seqs).integers(0, 300, size=seqs)
    w = wl.make_workload("steps", hist, np.ones(seqs, np.int32), seed=seqs, pool_slack=0.2)
    run_case(w, 8, 4, q8, "sections", one_each=True)
    run_case(w, 8, 4, q8, "odd sections", True)


@pytest.mark.parametrize("q8", [False, True])
def test_strides_in_place_and_padding(q8):
    w = wl.make_workload("pad", [4, 9, 0, 50], [0, 12, 0, 2], seed=8, pool_slack=0.5)
    run_case(w, 8, 8, q8, "sections", strided=True, in_place=True, extra=3)
    run_case(w, 8, 8, q8, "four", extra=5)


def test_long_prompts():
    w = wl.make_workload("long", [3, 0], [3001, 5000], seed=9, pool_slack=0.1)
    run_case(w, 32, 8, False, "sections")
    run_case(w, 32, 8, True, "cycled")


@pytest.mark.parametrize("q8", [False, True])
def test_slot_positions_give_the_plain_append(q8):
    """With the slots' positions on every axis the two calls agree bit for bit, whatever the axes."""
    w = wl.make_workload("same", [3, 40, 0], [30, 1, 9], seed=10, pool_slack=0.4)
    n = int(w.new_lens.sum())
    q, k, v, table = rows(n, 8, 1).cuda(), rows(n, 2, 2).cuda(), rows(n, 2, 3).cuda(), angles(TABLE).cuda()
    pos = torch.tensor([[p for _, p in tokens_of(w)]] * 3, dtype=torch.int32).cuda()
    tail = (i32(w.block_tables), i32(w.context_lens), i32(w.new_start_loc))

    def pools():
        return pa.new_q8_cache(w.num_blocks, 2) if q8 else [
            torch.zeros(w.num_blocks, 2, 16, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)]

    plain, at = (pa.pa_rope_append_q8, pa.pa_rope_append_at_q8) if q8 else (pa.pa_rope_append, pa.pa_rope_append_at)
    a = pools()
    q_a = plain(q, k, v, table, *a, *tail)
    for name in ("sections", "cycled"):
        b = pools()
        q_b = at(q, k, v, table, pos, *b, *tail, pair_axes=AXES[name])
        assert torch.equal(q_a, q_b)
        assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("one_each", [False, True])
@pytest.mark.parametrize("bad", [-1, TABLE, 1 << 30, -(1 << 31)])
def test_positions_outside_the_table(q8, one_each, bad):
    """The token is reported and skipped; the 8-bit pools leave its whole block as it was."""
    lens = [1, 1, 1] if one_each else [5, 1, 20]
    w = wl.make_workload("bad", [20, 40, 14], lens, seed=11, pool_slack=0.5)
    n = sum(lens)
    q, k, v = rows(n, 4, 1).cuda(), rows(n, 2, 2).cuda(), rows(n, 2, 3).cuda()
    pos = positions_for(n, 3, 1)
    victim = 2 if one_each else 8  # of the last sequence: its third token, in its second block
    pos[1, victim] = bad
    status = pa.new_device_status()
    shape = (w.num_blocks, 2, 16, 64)
    tail = (i32(w.block_tables), i32(w.context_lens), None if one_each else i32(w.new_start_loc))
    out = torch.full_like(q, 7.0)
    kw = dict(pair_axes=AXES["sections"], q_out=out, device_status=status)
    if q8:
        dev = pa.new_q8_cache(w.num_blocks, 2)
        pa.pa_rope_append_at_q8(q, k, v, angles(TABLE).cuda(), pos.cuda(), *dev, *tail, **kw)
    else:
        dev = [torch.zeros(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        pa.pa_rope_append_at(q, k, v, angles(TABLE).cuda(), pos.cuda(), *dev, *tail, **kw)
    assert int(status.item()) == pa.DEVFLAG_BAD_CONTEXT
    assert (out[victim] == 7.0).all() and not (out[[i for i in range(n) if i != victim]] == 7.0).all(dim=2).any()
    for pool in dev[:2]:
        stored = (pool.float() != 0).any(dim=3).cpu()  # [N, H, 16]
        for t, (s, p) in enumerate(tokens_of(w)):
            there = bool(stored[int(w.block_tables[s, p // 16]), :, p % 16].any())
            vs, vp = tokens_of(w)[victim]
            lost = t == victim or (q8 and s == vs and p // 16 == vp // 16)
            assert there != lost, (t, s, p)


def test_captured_positions_that_change():
    w = wl.make_workload("graph", [10, 20], [12, 7], seed=12, pool_slack=0.5)
    n = 19
    q, k, v, table = rows(n, 8, 1).cuda(), rows(n, 2, 2).cuda(), rows(n, 2, 3).cuda(), angles(TABLE).cuda()
    kc = torch.zeros(w.num_blocks, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    pos, out = positions_for(n, 3, 1).cuda(), torch.empty_like(q)
    tail = (i32(w.block_tables), i32(w.context_lens), i32(w.new_start_loc))
    graph = graphs.StepGraph(lambda: pa.pa_rope_append_at(q, k, v, table, pos, kc, vc, *tail, pair_axes=AXES["cycled"],
                                                          q_out=out))
    for seed in (2, 3):
        pos.copy_(positions_for(n, 3, seed))
        graph.replay()
        kept = (out.clone(), kc.clone(), vc.clone())
        pa.pa_rope_append_at(q, k, v, table, pos, kc, vc, *tail, pair_axes=AXES["cycled"], q_out=out)
        assert all(torch.equal(a, b) for a, b in zip(kept, (out, kc, vc)))
