"""Ends of the 8-bit calls' contracts: scales of zero and below the normal floats, bounds that the
caller states too small, one workspace under batches of every size."""
import numpy as np
import pytest
import torch

from paged_kv_cache_299_gb300 import binding as pa
from paged_kv_cache_299_gb300 import graphs
from paged_kv_cache_299_gb300 import workloads as wl
from _q8 import attend, dequantise
from test_gpu_q8_attention import State, close

pytestmark = pytest.mark.gpu


# ---- scales ---------------------------------------------------------------------------------
@pytest.mark.parametrize("hq", [8, 4, 2])
@pytest.mark.parametrize("q_exp,key_scales,value_scales", [
    (118, [0.0], [1.0]),                                              # every score is zero
    (112, [0.0, 2.0 ** -126, 1.37 * 2.0 ** -127, 2.0 ** -121], [1.0, 0.7]),
    (116, [2.0 ** -140, 2.0 ** -149, 0.0, 1.6 * 2.0 ** -131], [0.3]),
    (0, [0.05], [1.37 * 2.0 ** -127, 2.0 ** -128, 0.0, 1.9 * 2.0 ** -129]),
    (0, [0.05], [2.0 ** -126, 1.6 * 2.0 ** -126, 1.99 * 2.0 ** -127])])
def test_scales_of_zero_and_below_the_normal_floats(hq, q_exp, key_scales, value_scales):
    """Any non-negative finite scale stands for itself, in long chunks, chunks of few rows and
    decode rows alike; block b of the pool has the b-th of the listed scales, in turn."""
    w = wl.make_workload("far", [0, 40, 300, 7], [1, 130, 33, 16], num_prefill=4, seed=17, pool_slack=0.5)
    st = State(w, 2, hq, rows=180, spread=0.0)
    st.q = (st.q.double() * 2.0 ** q_exp).to(torch.bfloat16)
    k, v, ks, vs = (x.cpu() for x in st.dev)
    for scales, values in ((ks, key_scales), (vs, value_scales)):
        live = ~torch.isnan(scales)
        turn = torch.tensor(values).float()[torch.arange(len(scales)) % len(values)]
        scales[:] = torch.where(live, turn[:, None].expand_as(scales), scales)
    st.dev = [x.cuda() for x in (k, v, ks, vs)]
    st.k64, st.v64 = dequantise(k, ks), dequantise(v, vs)
    ref, tol = attend(st.q, st.k64, st.v64, w.block_tables, w.context_lens, st.scale, w.new_lens)
    tol = tol + 2.0 ** -126  # (what falls below the normal floats may vanish)
    got = st.chunk()
    assert st.ok()
    close(got, ref, tol, "chunk")
    last = torch.tensor(np.cumsum(w.new_lens) - 1)
    st.q = st.q[last]
    close(st.decode(), ref[last], tol[last], "decode")
    st.w = wl.Workload("rows", w.context_lens - 1, np.ones(4, np.int32), 4, w.num_blocks, w.block_tables, 0)
    close(st.chunk(), ref[last], tol[last], "few rows")
    assert st.ok()


# ---- bounds that the caller states ----------------------------------------------------------
def test_decode_reports_a_context_above_its_bound():
    """One context above max_context_len among many far below it, in the same block as the
    bound or far past it; every row is right all the same."""
    lens = [20] * 20 + [500] + [100] * 3 + [0]
    w = wl.make_workload("bound", lens, np.zeros(len(lens), int), seed=2, pool_slack=0.3)
    st = State(w, 2, 8)
    ref, tol = attend(st.q, st.k64, st.v64, w.block_tables, w.context_lens, st.scale)
    for bound, told in ((100, True), (499, True), (500, False), (10 ** 6, False)):
        st.max_ctx = bound
        st.status.zero_()
        close(st.decode(), ref, tol, f"bound {bound}")
        assert int(st.status.item()) == (pa.DEVFLAG_BAD_CONTEXT if told else 0), bound
    short = wl.make_workload("short", [300, 0], [0, 0], seed=3, pool_slack=0.3)
    st = State(short, 8, 32)
    st.max_ctx = 299  # the same number of blocks
    st.decode()
    assert int(st.status.item()) == pa.DEVFLAG_BAD_CONTEXT


@pytest.mark.parametrize("hq,hkv,bound,lens", [
    (8, 2, 20, [40, 20, 13]),                             # listed units
    (2, 2, 64, [65, 64, 1]),
    (4, 1, 64, [70] + [3] * 2100),                        # units in grid order: rows past the bound
    (4, 1, 11, [12, 11, 64] + [3] * 2100)])
def test_chunk_reports_more_rows_than_its_bound(hq, hkv, bound, lens):
    """A chunk longer than max_query_len is reported and left alone, whatever form the call takes."""
    lens = np.array(lens)
    w = wl.make_workload("longer", np.full(len(lens), 5), lens, num_prefill=len(lens), seed=4, pool_slack=0.1)
    st = State(w, hkv, hq, rows=int(lens.sum()))
    ref, tol = attend(st.q, st.k64, st.v64, w.block_tables, w.context_lens, st.scale, w.new_lens)
    got = st.chunk(bound)
    assert int(st.status.item()) == pa.DEVFLAG_BAD_CONTEXT
    over = torch.from_numpy(np.repeat(lens > bound, lens))
    assert bool(torch.isnan(got[over.cuda()]).all())  # left as they were
    close(got[~over.cuda()], ref[~over], tol[~over], "the others")
    st.status.zero_()
    close(st.chunk(), ref, tol, "all")
    assert st.ok()


# ---- one workspace --------------------------------------------------------------------------
def test_one_workspace_serves_batches_of_every_size():
    """A program's one buffer, zeroed once, under batches that come and go: the counters of one call
    never lie where another leaves its partials."""
    ws = torch.zeros(16 << 20, dtype=torch.uint8, device="cuda")
    states = []
    for i, (hq, hkv, lens) in enumerate([(32, 8, [3000] * 5), (4, 1, [9000, 20]), (8, 8, [700] * 60), (32, 8, [40000]),
                                         (2, 1, [500] * 300), (32, 8, [2000, 1, 0] * 40), (16, 8, [6000] * 9)]):
        w = wl.make_workload("batch", lens, np.zeros(len(lens), int), seed=i, pool_slack=0.1)
        st = State(w, hkv, hq, seed=i)
        st.max_ctx = 65536
        states.append((st, st.decode()))
        need = pa.pa_decode_q8_workspace_size(len(lens), hkv, hq, 65536)
        assert need <= ws.numel()
        assert need == pa.pa_decode_q8_workspace_size(1, 1, hq // hkv, 1)  # nor does its size
    order = np.random.default_rng(5).integers(0, len(states), size=40)
    for i in order:
        st, want = states[i]
        assert torch.equal(st.decode(workspace=ws), want), f"batch {i}"
    st, want = states[0]
    q, out = st.q.cuda(), torch.empty_like(want)
    graph = graphs.StepGraph(lambda: pa.pa_decode_q8(out, q, *st.dev, st.bt, st.ctx, st.scale, st.max_ctx, workspace=ws))
    for i in order[:10]:
        assert torch.equal(states[i][0].decode(workspace=ws), states[i][1])
        out.zero_()
        graph.replay()
        assert torch.equal(out, want)
    assert all(st.ok() for st, _ in states)
