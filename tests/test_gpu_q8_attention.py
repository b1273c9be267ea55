"""pa_decode_q8 and pa_prefill_chunk_q8 against softmax attention over the dequantised cache in
64 bits (tolerances: _q8.attend), and the operators together: append, fork, copy, attend."""
import numpy as np
import pytest
import torch

from paged_kv_cache_299_gb300 import binding as pa
from paged_kv_cache_299_gb300 import graphs
from paged_kv_cache_299_gb300 import workloads as wl
from _gpu import i32
from _q8 import angles, attend, dequantise, quantise, rotate, store_q8, tokens_of

pytestmark = pytest.mark.gpu


class State:
    """A cache whose live slots hold random values and whose every other byte is poison: codes
    0x7f (NaN) and NaN scales."""

    def __init__(self, w, hkv, hq, seed=0, q_size=1.0, spread=0.5, scales="powers", rows=None):
        g = torch.Generator().manual_seed(seed)
        nb = w.num_blocks
        self.w, self.hq, self.hkv = w, hq, hkv
        live = torch.zeros(nb, 16, dtype=torch.bool)
        for s, n in enumerate(w.context_lens):
            for b in range(-(-int(n) // 16)):
                live[int(w.block_tables[s, b]), :min(16, int(n) - 16 * b)] = True
        self.pools = []
        for _ in range(2):
            x = torch.randn(nb, hkv, 16, 64, generator=g)
            x *= torch.exp(spread * torch.randn(nb, hkv, 1, 1, generator=g))
            codes, sc = quantise(x)
            if scales == "any":  # written by someone else: no powers of two
                sc = sc * (0.6 + torch.rand(sc.shape, generator=g))
            raw = codes.view(torch.uint8).clone()
            raw[~live[:, None, :].expand(-1, hkv, -1)] = 0x7f
            sc = sc.clone()
            sc[~live.any(dim=1)] = float("nan")
            self.pools.append((raw.view(torch.float8_e4m3fn), sc))
        (k, ks), (v, vs) = self.pools
        self.k64, self.v64 = dequantise(k, ks), dequantise(v, vs)
        rows = w.num_seqs if rows is None else rows
        self.q = (q_size * torch.randn(rows, hq, 64, generator=g)).to(torch.bfloat16)
        self.dev = [x.cuda() for x in (k, v, ks, vs)]
        self.bt, self.ctx = i32(w.block_tables), i32(w.context_lens)
        self.status = pa.new_device_status()
        self.scale = 0.125
        self.max_ctx = int(w.context_lens.max())

    def decode(self, **kw):
        out = torch.full(self.q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
        pa.pa_decode_q8(out, self.q.cuda(), *self.dev, self.bt, self.ctx, self.scale, self.max_ctx,
                        device_status=self.status, **kw)
        return out

    def chunk(self, max_query_len=None):
        out = torch.full(self.q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
        pa.pa_prefill_chunk_q8(out, self.q.cuda(), i32(self.w.new_start_loc),
                               max_query_len or int(self.w.new_lens.max()), *self.dev, self.bt, self.ctx,
                               self.scale, device_status=self.status)
        return out

    def ok(self):
        return pa.pa_check_device_status(self.status) == pa.PA_OK


def close(got, ref, tol, what=""):
    got = got.cpu().double()
    assert torch.isfinite(got).all(), f"{what}: non-finite output (poison was read)"
    bad = (got - ref).abs() > tol
    worst = float(((got - ref).abs() / tol.clamp(min=1e-30)).max())
    assert not bad.any(), f"{what}: {int(bad.sum())} values out of tolerance, worst {worst:.3g} of it"


def check_decode(w, hkv=8, hq=32, **kw):
    st = State(w, hkv, hq, **kw)
    got = st.decode()
    assert st.ok()
    ref, tol = attend(st.q, st.k64, st.v64, w.block_tables, w.context_lens, st.scale)
    close(got, ref, tol, w.name)
    return st, got


def check_chunk(w, hkv=8, hq=32, **kw):
    st = State(w, hkv, hq, rows=int(w.new_lens.sum()), **kw)
    got = st.chunk()
    assert st.ok()
    ref, tol = attend(st.q, st.k64, st.v64, w.block_tables, w.context_lens, st.scale, w.new_lens)
    close(got, ref, tol, w.name)
    return st, got


# ---- decode ---------------------------------------------------------------------------------
@pytest.mark.parametrize("hq,hkv", [(32, 8), (8, 8), (2, 1), (12, 3), (4, 1)])
def test_decode_head_layouts(hq, hkv):
    check_decode(wl.make_workload("heads", [0, 14, 15, 16, 99, 700], np.ones(6, int), seed=hq, pool_slack=0.3),
                 hkv, hq)


def test_decode_every_tail_length():
    ctx = np.arange(1, 97)
    check_decode(wl.make_workload("tails", ctx - 1, np.ones_like(ctx), seed=5, pool_slack=0.25))


@pytest.mark.parametrize("L", [1, 2, 16, 17, 300, 768, 769, 2000, 9000, 40000])
def test_decode_one_sequence(L):
    check_decode(wl.make_workload(f"one{L}", [L - 1], [1], seed=L, pool_slack=0.5))


def test_decode_batches():
    check_decode(wl.decode_batch64_uniform())
    rng = np.random.default_rng(1)
    ctx = np.clip(np.exp(rng.normal(5, 1.5, size=300)).astype(int), 1, 4000)
    check_decode(wl.make_workload("b300", ctx - 1, np.ones_like(ctx), seed=6), 2, 8)


@pytest.mark.parametrize("hq,hkv,lens", [
    (4, 1, [40000]),                          # one segment over more than 32 CTAs
    (2, 1, [33000, 1, 0, 500]),
    (8, 2, [20000] + [30] * 40),              # one long among short ones
    (8, 2, [30, 0, 0, 9000, 17, 0, 700]),
    (32, 8, [600, 0, 1, 90] + [16] * 9),      # a CTA per segment, some with fewer tiles than warps
    (4, 1, list(range(0, 150))),
    (2, 2, [190] * 76),                       # as many segments as a 152-SM device has CTAs
    (2, 2, [190] * 77)])
def test_decode_uneven_batches(hq, hkv, lens):
    """Every way pieces meet: whole segments, within a CTA, over many, and a CTA per segment."""
    w = wl.make_workload("uneven", lens, np.zeros(len(lens), int), num_prefill=0, seed=len(lens), pool_slack=0.2)
    st, got = check_decode(w, hkv, hq)
    ws = torch.zeros(pa.pa_decode_q8_workspace_size(len(lens), hkv, hq, 131072), dtype=torch.uint8, device="cuda")
    st.max_ctx = 131072  # planned for longer contexts than there are
    for _ in range(2):
        ref, tol = attend(st.q, st.k64, st.v64, w.block_tables, w.context_lens, st.scale)
        close(st.decode(workspace=ws), ref, tol, "planned longer")


def test_decode_most_sequences():
    lens = np.random.default_rng(9).integers(0, 50, size=4096)
    check_decode(wl.make_workload("most", lens, np.zeros(4096, int), seed=9), 1, 4)


def test_decode_long_contexts():
    check_decode(wl.make_workload("long", [20000, 3, 33333, 8191], [1, 1, 1, 1], seed=7), 4, 16)


@pytest.mark.parametrize("kw", [dict(q_size=12.0), dict(q_size=1e-3), dict(spread=6.0), dict(scales="any"),
                                dict(q_size=4e4, spread=0.0), dict(q_size=0.0)])
def test_decode_values(kw):
    """Peaked and flat weights, scales that differ by orders of magnitude between blocks, scales
    that are no powers of two, scores far outside an exponential's range, zero queries."""
    w = wl.make_workload("values", [500, 100, 37], [1, 1, 1], seed=8, pool_slack=0.3)
    check_decode(w, 2, 8, **kw)
    check_chunk(wl.make_workload("values", [460, 60, 0], [40, 40, 37], seed=8, pool_slack=0.3), 2, 8, **kw)


def test_decode_empty_context_gives_zero_rows():
    w = wl.make_workload("empty", [30, -1, 5], [1, 1, 1], seed=9, pool_slack=0.5)
    st, got = check_decode(w)
    assert bool((got[1] == 0).all())
    many = wl.make_workload("empty2", [9000, -1], [1, 1], seed=9, pool_slack=0.5)
    _, got = check_decode(many)
    assert bool((got[1] == 0).all())


def test_decode_workspace_is_reusable_and_results_repeat():
    w = wl.random_small(31, num_seqs=9, max_ctx=1500)
    st = State(w, 8, 32)
    need = pa.pa_decode_q8_workspace_size(9, 8, 32, st.max_ctx)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    first = st.decode(workspace=ws)
    for _ in range(3):
        assert torch.equal(st.decode(workspace=ws), first)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    assert torch.equal(st.decode(workspace=torch.zeros_like(ws), stream=None), first)
    q, out = st.q.cuda(), torch.empty_like(first)

    def step():
        pa.pa_decode_q8(out, q, *st.dev, st.bt, st.ctx, st.scale, st.max_ctx, workspace=ws)

    graph = graphs.StepGraph(step)
    out.zero_()
    graph.replay()
    assert torch.equal(out, first)
    with torch.cuda.stream(side):
        got = st.decode()
    side.synchronize()
    assert torch.equal(got, first)
    assert st.ok()


def test_decode_launch_flags():
    """Overlapped launches of several layers, and SM budgets, give the default's results (a
    budget moves the split points: within tolerance)."""
    w = wl.random_small(32, num_seqs=20, max_ctx=900)
    layers = [State(w, 8, 32, seed=s) for s in range(4)]
    ws = torch.zeros(pa.pa_decode_q8_workspace_size(20, 8, 32, layers[0].max_ctx), dtype=torch.uint8, device="cuda")
    plain = [st.decode() for st in layers]
    torch.cuda.synchronize()
    outs = [torch.empty_like(plain[0]) for _ in layers]
    qs = [st.q.cuda() for st in layers]
    torch.cuda.synchronize()
    for st, q, out in zip(layers, qs, outs):
        pa.pa_decode_q8(out, q, *st.dev, st.bt, st.ctx, st.scale, st.max_ctx, workspace=ws,
                        launch_flags=pa.PA_LAUNCH_OVERLAP_PREVIOUS, device_status=st.status)
    assert all(torch.equal(a, b) for a, b in zip(outs, plain))
    ref, tol = attend(layers[0].q, layers[0].k64, layers[0].v64, w.block_tables, w.context_lens, 0.125)
    for n in (1, 7, 90, 500):
        close(layers[0].decode(launch_flags=pa.PA_LAUNCH_MAX_SMS(n)), ref, tol, f"{n} SMs")
    assert all(st.ok() for st in layers)


def test_other_streams_allocate_and_run_in_order():
    """A stream of the caller's, with the call's own workspace and output: both belong to it."""
    w = wl.random_small(33, num_seqs=12, max_ctx=700)
    st = State(w, 8, 32)
    want = st.decode()
    q, out = st.q.cuda(), torch.empty_like(want)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        out.zero_()
        side.wait_stream(torch.cuda.current_stream())
        pa.pa_decode_q8(out, q, *st.dev, st.bt, st.ctx, st.scale, st.max_ctx, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(out, want)
    kc, vc, ks, vs = pa.new_q8_cache(w.num_blocks, 8)
    k = st.q[:, :8].contiguous().cuda()
    table = angles(800).cuda()
    torch.cuda.synchronize()
    rot = pa.pa_rope_append_q8(q, k, k, table, kc, vc, ks, vs, st.bt, st.ctx, stream=side)
    side.synchronize()
    ref = pa.pa_rope_append_q8(q, k, k, table, kc, vc, ks, vs, st.bt, st.ctx)
    assert torch.equal(rot, ref)


def test_wrong_device_is_refused(monkeypatch):
    """Tensors of another device than the current one never reach a kernel."""
    w = wl.random_small(34, num_seqs=2, max_ctx=30)
    st = State(w, 8, 32)
    q, out = st.q.cuda(), torch.empty_like(st.q, device="cuda")
    k, table = st.q[:, :8].contiguous().cuda(), angles(40).cuda()
    monkeypatch.setattr(pa, "_get_device", lambda: 1)
    for call in (lambda: pa.pa_decode_q8(out, q, *st.dev, st.bt, st.ctx, 0.125, st.max_ctx),
                 lambda: pa.pa_prefill_chunk_q8(out, q, i32([0, 1, 2]), 1, *st.dev, st.bt, st.ctx, 0.125),
                 lambda: pa.pa_rope_append_q8(q, k, k, table, *st.dev, st.bt, st.ctx),
                 lambda: pa.pa_copy_blocks_q8(*st.dev, torch.zeros(1, 2, dtype=torch.int64, device="cuda"))):
        with pytest.raises(ValueError, match="current device"):
            call()
    monkeypatch.undo()
    with pytest.raises(ValueError):  # a status word on the host
        pa.pa_decode_q8(out, q, *st.dev, st.bt, st.ctx, 0.125, st.max_ctx,
                        device_status=torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError):  # not contiguous
        pa.pa_decode_q8(out, q.transpose(0, 1), *st.dev, st.bt, st.ctx, 0.125, st.max_ctx)


def test_decode_bad_entries_are_reported():
    w = wl.make_workload("bad", [40, 100], [1, 1], seed=12, pool_slack=0.5)
    st = State(w, 8, 32)
    good = st.decode()
    bt = w.block_tables.copy()
    bt[0, 1] = w.num_blocks + 5
    st.bt = i32(bt)
    got = st.decode()
    assert int(st.status.item()) == pa.DEVFLAG_BAD_BLOCK
    assert torch.equal(got[1], good[1])
    st.bt, st.ctx = i32(w.block_tables), i32([41, 5000])
    st.status.zero_()
    st.decode()
    assert int(st.status.item()) == pa.DEVFLAG_BAD_CONTEXT


# ---- chunks ---------------------------------------------------------------------------------
@pytest.mark.parametrize("hq,hkv", [(32, 8), (8, 8), (2, 1), (6, 3), (64, 16)])
def test_chunk_head_layouts(hq, hkv):
    w = wl.make_workload("heads", [0, 40, 63, 130, 7], [45, 33, 65, 1, 128], num_prefill=5, seed=hq, pool_slack=0.3)
    check_chunk(w, hkv, hq)


@pytest.mark.parametrize("prior", [0, 1, 15, 16, 47, 63, 64, 200])
def test_chunk_lengths(prior):
    new = np.array([1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100])
    w = wl.make_workload("lengths", np.full(len(new), prior), new, num_prefill=len(new), seed=prior, pool_slack=0.2)
    check_chunk(w, 2, 8)
    check_chunk(w, 2, 2)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 1), (4, 1), (32, 8)])
def test_chunk_of_one_row(hq, hkv):
    """The smallest call: one row (a query box larger than the tensor), alone and with a prior."""
    check_chunk(wl.make_workload("first", [0], [1], num_prefill=1, seed=hq, pool_slack=2.0), hkv, hq)
    check_chunk(wl.make_workload("later", [333], [1], num_prefill=1, seed=hq, pool_slack=1.0), hkv, hq)


@pytest.mark.parametrize("hq,hkv,most", [(32, 8, 8), (32, 8, 5), (4, 1, 4), (4, 1, 2), (2, 1, 16), (2, 2, 32),
                                         (3, 3, 9)])
def test_chunk_of_few_rows(hq, hkv, most):
    """At most 32 rows per K/V head, every count of them, at every place in a block; from one
    segment (a cluster of CTAs) to many."""
    rng = np.random.default_rng(most)
    for seqs in (1, 3, 19, 90):
        new = np.concatenate([[most], rng.integers(0, most + 1, size=seqs - 1)]).astype(int)
        prior = rng.integers(0, 300, size=seqs)
        prior[0] = 3000 if seqs < 19 else 700
        w = wl.make_workload(f"few{seqs}", prior, new, num_prefill=seqs, seed=seqs, pool_slack=0.3)
        check_chunk(w, hkv, hq)


def test_chunk_of_few_rows_refuses_longer_ones_and_repeats():
    w = wl.make_workload("longer", [100, 40, 2000], [5, 7, 3], num_prefill=3, seed=4, pool_slack=0.3)
    st = State(w, 8, 32, rows=15)
    ref, tol = attend(st.q, st.k64, st.v64, w.block_tables, w.context_lens, st.scale, w.new_lens)
    got = st.chunk(5)  # the second chunk has more rows
    assert int(st.status.item()) == pa.DEVFLAG_BAD_CONTEXT
    assert bool(torch.isnan(got[5:12]).all())
    close(got[:5], ref[:5], tol[:5], "first")
    close(got[12:], ref[12:], tol[12:], "third")
    st.status.zero_()
    whole = st.chunk()
    assert st.ok() and torch.equal(st.chunk(), whole)
    close(whole, ref, tol, "all")
    bt = w.block_tables.copy()
    bt[1, 1], bt[2, 0] = w.num_blocks, -1
    st.bt = i32(bt)
    assert torch.equal(st.chunk()[:5], whole[:5])
    assert int(st.status.item()) == pa.DEVFLAG_BAD_BLOCK


def test_chunk_long():
    w = wl.make_workload("long", [1500, 0, 5000], [700, 1030, 3], num_prefill=3, seed=4)
    check_chunk(w, 1, 4)


@pytest.mark.parametrize("hq,hkv", [(32, 8), (2, 2)])
def test_chunk_many_units_per_cta(hq, hkv):
    """Several units per CTA, of one K/V tile and of several, with one query tile and with two."""
    rng = np.random.default_rng(hq)
    new = np.where(rng.random(200) < 0.7, rng.integers(1, 9, size=200), rng.integers(20, 150, size=200))
    w = wl.make_workload("units", rng.integers(0, 400, size=200), new, num_prefill=200, seed=hq)
    check_chunk(w, hkv, hq)


def test_chunk_many_short_ones():
    """More (sequence, tile) pairs than the kernel sorts: units in grid order."""
    new = np.random.default_rng(2).integers(1, 4, size=2200)
    w = wl.make_workload("short", np.random.default_rng(3).integers(0, 30, size=2200), new, num_prefill=2200, seed=5)
    check_chunk(w, 1, 4)


def test_chunk_empty_sequences_and_padding_rows():
    w = wl.make_workload("pad", [9, 4, 0, 20], [0, 30, 0, 5], num_prefill=4, seed=6, pool_slack=0.5)
    st = State(w, 8, 32, rows=35 + 9)
    got = st.chunk()
    assert st.ok()
    ref, tol = attend(st.q[:35], st.k64, st.v64, w.block_tables, w.context_lens, 0.125, w.new_lens)
    close(got[:35], ref, tol, "padded")
    assert bool(torch.isnan(got[35:]).all())  # left as they were


def test_chunk_equals_decode_on_single_rows():
    w = wl.random_small(41, num_seqs=12, max_ctx=400)
    st = State(w, 8, 32)
    a, b = st.decode(), st.chunk()
    ref, tol = attend(st.q, st.k64, st.v64, w.block_tables, w.context_lens, 0.125)
    close(a, ref, tol, "decode")
    close(b, ref, tol, "chunk")


def test_chunk_repeats_and_replays():
    w = wl.make_workload("again", [100, 37, 500], [64, 40, 129], num_prefill=3, seed=4, pool_slack=0.3)
    st = State(w, 8, 32, rows=233)
    first = st.chunk()
    assert torch.equal(st.chunk(), first)
    q, out, qsl = st.q.cuda(), torch.empty_like(first), i32(w.new_start_loc)

    def step():
        pa.pa_prefill_chunk_q8(out, q, qsl, 129, *st.dev, st.bt, st.ctx, 0.125)

    graph = graphs.StepGraph(step)
    out.zero_()
    graph.replay()
    assert torch.equal(out, first)


def test_chunk_bad_entries_are_reported():
    w = wl.make_workload("bad", [40, 100], [33, 20], num_prefill=2, seed=12, pool_slack=0.5)
    st = State(w, 8, 32, rows=53)
    good = st.chunk()
    bt = w.block_tables.copy()
    bt[0, 1] = -7
    st.bt = i32(bt)
    got = st.chunk()
    assert int(st.status.item()) & pa.DEVFLAG_BAD_BLOCK
    assert torch.equal(got[33:], good[33:])
    st.bt, st.ctx = i32(w.block_tables), i32([20, 120])  # shorter than its rows
    st.status.zero_()
    st.chunk()
    assert int(st.status.item()) == pa.DEVFLAG_BAD_CONTEXT


@pytest.mark.parametrize("q_exp,key_exp,value_exp", [
    (-14, "smallest", 0), (-30, "smallest", -126), (-14, "zero", 0), (-100, 100, 100), (-110, 110, -60),
    (60, -70, 118), (0, -126, 0)])
def test_extreme_scales(q_exp, key_exp, value_exp):
    """Queries and scales far apart: products of a block's scale and a row's that vanish (blocks
    of zero keys, whose scale is the smallest there is, or a scale of zero), and ones that meet
    again from both ends of the range."""
    w = wl.make_workload("far", [0, 40, 300, 7], [1, 130, 33, 16], num_prefill=4, seed=17, pool_slack=0.5)
    st = State(w, 2, 8, rows=180, spread=0.0)
    st.q = (st.q.double() * 2.0 ** q_exp).to(torch.bfloat16)
    k, v, ks, vs = (x.cpu() for x in st.dev)
    live = ~torch.isnan(ks)
    if key_exp == "smallest":
        zero = live[..., None, None] & (k.view(torch.uint8) != 0x7f)
        k = torch.where(zero, torch.zeros((), dtype=torch.uint8), k.view(torch.uint8)).view(torch.float8_e4m3fn)
        ks = torch.where(live, torch.full_like(ks, 2.0 ** -126), ks)
    elif key_exp == "zero":
        ks = torch.where(live, torch.zeros_like(ks), ks)
    else:
        ks = ks * 2.0 ** key_exp
    vs = vs * 2.0 ** (value_exp + (8 if value_exp < -100 else 0))  # (normal floats)
    st.dev = [x.cuda() for x in (k, v, ks, vs)]
    st.k64, st.v64 = dequantise(k, ks), dequantise(v, vs)
    ref, tol = attend(st.q, st.k64, st.v64, w.block_tables, w.context_lens, st.scale, w.new_lens)
    got = st.chunk()
    assert st.ok()
    close(got, ref, tol + 2.0 ** -126, "chunk")  # (what falls below the normal floats may vanish)
    last = torch.tensor(np.cumsum(w.new_lens) - 1)
    st.q = st.q[last]
    got = st.decode()
    assert st.ok()
    close(got, ref[last], tol[last] + 2.0 ** -126, "decode")


# ---- against the oracle, and far into a large pool --------------------------------------------
def test_agrees_with_the_oracle_on_the_dequantised_cache():
    """A code times a power of two is a bf16 value, so the oracle can read the same cache."""
    import oracle
    w = wl.make_workload("oracle", [100, 37, 300], [50, 40, 1], num_prefill=3, seed=14, pool_slack=0.3)
    st = State(w, 8, 32, rows=91)
    kc, vc = (torch.nan_to_num(x).to(torch.bfloat16) for x in (st.k64, st.v64))
    ref, err = oracle.prefill_chunk(wl.bf16_bits(st.q), w.new_start_loc, wl.bf16_bits(kc), wl.bf16_bits(vc),
                                    w.block_tables, w.context_lens, 0.125)
    assert err == 0
    diff = np.abs(st.chunk().float().cpu().numpy().astype(np.float64) - ref)
    assert diff.max() <= 2e-2 and diff.mean() <= 2e-3
    last = st.q[w.new_start_loc[1:] - 1]
    ref, err = oracle.decode(wl.bf16_bits(last), wl.bf16_bits(kc), wl.bf16_bits(vc), w.block_tables, w.context_lens,
                             0.125)
    assert err == 0
    st.q = last
    diff = np.abs(st.decode().float().cpu().numpy().astype(np.float64) - ref)
    assert diff.max() <= 2e-2 and diff.mean() <= 2e-3


def test_blocks_far_into_a_large_pool():
    """Pools above 4 GiB: append, copy, decode and chunk at their far end, bf16 append too."""
    nb, hkv, hq = 600_000, 8, 32
    kc, vc = (torch.empty(nb, hkv, 16, 64, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
              for _ in range(2))
    ks, vs = (torch.full((nb, hkv), float("nan"), device="cuda") for _ in range(2))
    g = torch.Generator().manual_seed(2)
    n = 75
    far = np.array([[nb - 1, 3, nb - 200, nb - 2, nb - 77]], np.int32)
    near = np.array([[0, 1, 2, 3, 4]], np.int32)
    k, v, q = (torch.randn(n, h, 64, generator=g).to(torch.bfloat16).cuda() for h in (hkv, hkv, hq))
    small = pa.new_q8_cache(5, hkv)
    status = pa.new_device_status()
    table, ctx, qsl = angles(n).cuda(), i32([n]), i32([0, n])
    outs = []
    for cache, bt in (((kc, vc, ks, vs), far), (small, near)):
        qr = pa.pa_rope_append_q8(q, k, v, table, *cache, i32(bt), ctx, qsl, device_status=status)
        if bt is far:  # one block moves, to the far end as well
            pa.pa_copy_blocks_q8(*cache, torch.tensor([[nb - 200, nb - 4]]).cuda(), device_status=status)
            bt = bt.copy()
            bt[0, 2] = nb - 4
        chunk, one = torch.empty_like(qr), torch.empty_like(qr[-1:])
        pa.pa_prefill_chunk_q8(chunk, qr, qsl, n, *cache, i32(bt), ctx, 0.125, device_status=status)
        pa.pa_decode_q8(one, qr[-1:].contiguous(), *cache, i32(bt), ctx, 0.125, n, device_status=status)
        outs.append((qr, chunk, one))
    assert pa.pa_check_device_status(status) == pa.PA_OK
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    del kc, vc
    big = [torch.empty(nb // 2, hkv, 16, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    bt = np.array([[nb // 2 - 1, 5, nb // 2 - 3, nb // 2 - 9, 6]], np.int32)
    pa.pa_rope_append(None, k, v, table, *big, i32(bt), ctx, qsl, device_status=status)
    low = [torch.empty(5, hkv, 16, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    pa.pa_rope_append(None, k, v, table, *low, i32(near), ctx, qsl, device_status=status)
    for x, y in zip(big, low):
        for i in range(n):
            assert torch.equal(x[int(bt[0, i // 16]), :, i % 16], y[i // 16, :, i % 16])
    assert pa.pa_check_device_status(status) == pa.PA_OK


# ---- together -------------------------------------------------------------------------------
def test_a_conversation_over_the_8bit_cache():
    """A prompt in two chunks, then token by token; a fork whose writers copy the shared block;
    every step's attention against 64-bit attention over what the definition stores."""
    hkv, hq, nb = 2, 8, 12
    g = torch.Generator().manual_seed(3)
    table = angles(200)
    dtab = table.cuda()
    cache = pa.new_q8_cache(nb, hkv)
    codes = [torch.zeros(nb, hkv, 16, 64, dtype=torch.float64) for _ in range(2)]
    scales = [torch.ones(nb, hkv, dtype=torch.float64) for _ in range(2)]
    status = pa.new_device_status()
    bm = pa.BlockManager(nb, 16)
    bm.add_sequence(0)
    held = {0: 0}

    def step(news):
        """news: {sequence: token count}; appends, then attends with every new row."""
        seqs = sorted(news)
        pairs = []
        for s in seqs:
            pairs += bm.append_tokens(s, news[s])
        if pairs:
            pa.pa_copy_blocks_q8(*cache, torch.tensor(pairs).cuda(), device_status=status)
            for a, b in pairs:
                for x in codes + scales:
                    x[b] = x[a]
        tables = np.array([bm.block_table(s, 8)[0] for s in seqs], np.int32)
        w = wl.Workload("step", np.array([held[s] for s in seqs]), np.array([news[s] for s in seqs]), len(seqs),
                        nb, tables, 0)
        n = int(w.new_lens.sum())
        q, k, v = ((1.5 * torch.randn(n, h, 64, generator=g)).to(torch.bfloat16) for h in (hq, hkv, hkv))
        one = max(news.values()) == 1
        bt, ctx, qsl = i32(tables), i32(w.context_lens), i32(w.new_start_loc)
        qr = pa.pa_rope_append_q8(q.cuda(), k.cuda(), v.cuda(), dtab, *cache, bt, ctx, None if one else qsl,
                                  device_status=status)
        out = torch.empty_like(qr)
        if one:
            pa.pa_decode_q8(out, qr, *cache, bt, ctx, 0.125, int(w.context_lens.max()), device_status=status)
        else:
            pa.pa_prefill_chunk_q8(out, qr, qsl, int(w.new_lens.max()), *cache, bt, ctx, 0.125, device_status=status)
        assert pa.pa_check_device_status(status) == pa.PA_OK
        pos = torch.tensor([p for _, p in tokens_of(w)])
        where = store_q8(rotate(k, table[pos], False), codes[0], scales[0], w)
        store_q8(v.double(), codes[1], scales[1], w)
        # round the definition's new codes as the cache did (within half a step: checked by the
        # append's own tests), then hold the attention to those
        blk, off = torch.tensor([b for b, _ in where]), torch.tensor([o for _, o in where])
        for c64, dev, s64, dsc in zip(codes, cache[:2], scales, cache[2:]):
            got = dev.cpu().float().double()
            assert torch.equal(dsc.cpu().double()[blk], s64[blk])
            assert ((got - c64)[blk, :, off].abs() <= (c64[blk, :, off].abs() / 16).clamp(min=2.0 ** -10) + 1e-4).all()
            c64[blk, :, off] = got[blk, :, off]
        ref, tol = attend(qr.cpu(), codes[0] * scales[0][..., None, None], codes[1] * scales[1][..., None, None],
                          tables, w.context_lens, 0.125, w.new_lens)
        close(out, ref, tol, "step")
        for s in seqs:
            held[s] += news[s]

    step({0: 37})
    step({0: 20})
    step({0: 1})
    bm.fork(0, 1)
    held[1] = held[0]
    step({0: 1, 1: 1})   # the shared, half-full block is copied for one of them
    step({0: 1, 1: 1})
    step({0: 12, 1: 3})
