"""Whether every K/V tile counts, and counts once, in the 8-bit attention calls: a tolerance on random
data cannot see one tile of some thousand come or go, these inputs can."""
import numpy as np
import pytest
import torch

from paged_kv_cache_299_gb300 import binding as pa
from paged_kv_cache_299_gb300 import workloads as wl
from _gpu import i32

gpu = pytest.mark.gpu

ONE = 0x38  # the e4m3 code of 1


def tables_of(w, hkv, seed):
    """Random key codes, poison in every slot and scale that no context holds."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    kc = torch.randint(0, 0x60, (w.num_blocks, hkv, 16, 64), generator=g, device="cuda", dtype=torch.uint8)
    ks, vs = (torch.full((w.num_blocks, hkv), float("nan"), device="cuda") for _ in range(2))
    used = torch.from_numpy(w.block_tables[w.block_tables >= 0].astype(np.int64)).cuda()
    ks[used], vs[used] = 0.25, 1.0
    return kc, torch.full_like(kc, 0x7f), ks, vs


def live_slots(w, s):
    """(block, place) of every token of sequence s."""
    n = int(w.context_lens[s])
    t = np.arange(n)
    return torch.from_numpy(w.block_tables[s][t // 16].astype(np.int64)).cuda(), torch.from_numpy(t % 16).cuda()


def views(kc, vc, ks, vs):
    return kc.view(torch.float8_e4m3fn), vc.view(torch.float8_e4m3fn), ks, vs


def half_step(x):
    """Half a step of bf16 at x > 0: eight significant bits."""
    return torch.exp2(torch.floor(torch.log2(x)) - 8)


# ---- equal weights ------------------------------------------------------------------------------
def coded(w, hkv, hq, q_lens=None, seed=0):
    """Zero queries make every weight 1 / n.  V of tile t is 1 in dim t % 64 and 0 elsewhere, so
    dim d of a row counts the visible tokens of the tiles d, d + 64, ...: up to 131,072 tokens a
    dim has at most 128 tiles, and one tile more or less moves it by at least 2^-7 of itself.

    All of a row's sums are whole numbers below 2^24 times a power of two (weights are exact powers
    of two, in f16 and bf16 alike), so they are exact in fp32; what rounds is 1 / sum and the product
    with it (2^-23 in all, 2^-22 allowed) and the bf16 output (half a step)."""
    kc, vc, ks, vs = tables_of(w, hkv, seed)
    counts = []
    for s in range(w.num_seqs):
        blocks, places = live_slots(w, s)
        n = len(blocks)
        kinds = torch.arange(n, device="cuda") // 16 % 64
        rows = torch.zeros(n, 64, dtype=torch.uint8, device="cuda")
        rows[torch.arange(n, device="cuda"), kinds] = ONE
        vc[blocks, :, places] = rows[:, None].expand(-1, hkv, -1)
        for i in range(1 if q_lens is None else int(q_lens[s])):
            seen = n if q_lens is None else n - int(q_lens[s]) + i + 1
            counts.append(torch.bincount(kinds[:seen], minlength=64).double() / max(seen, 1))
    ref = torch.stack(counts)[:, None].expand(-1, hq, -1)
    return views(kc, vc, ks, vs), torch.zeros(len(counts), hq, 64, dtype=torch.bfloat16, device="cuda"), ref


def off(got, ref):
    """Where a row of the kernels misses its counts."""
    tol = torch.where(ref > 0, half_step(ref.clamp(min=2.0 ** -60)) + 2.0 ** -22 * ref, 0.0)
    return ((got.double() - ref).abs() > tol) | ~torch.isfinite(got)


def counted(got, ref, what):
    bad = off(got, ref)
    assert not bad.any(), f"{what}: {int(bad.sum())} dims, first (row, head, dim) {bad.nonzero()[0].tolist()}"


@pytest.mark.parametrize("n", [48, 300, 2000, 9000, 40000, 100000, 131067, 131071, 131072])
def test_one_tile_more_or_less_is_seen(n):
    """On the CPU, in the reference: a whole tile left out or taken twice, in V alone or with its
    weights, misses the count of its dim; none left out misses nothing."""
    counts = torch.bincount(torch.arange(n) // 16 % 64, minlength=64).double()
    ref = counts / n
    assert not off(ref.to(torch.bfloat16), ref).any()
    for d in range(min(64, n // 16)):
        for tokens in (-16, 16):
            for total in (n, n + tokens):
                if total == 0:
                    continue
                wrong = counts.clone()
                wrong[d] += tokens
                assert off((wrong / total).to(torch.bfloat16), ref)[d]


@gpu
@pytest.mark.parametrize("hq,hkv,lens", [
    (32, 8, [131072]), (4, 1, [131072, 131072, 5, 0, 40000]), (32, 8, [131072] * 4), (2, 1, [131071] + [30] * 50),
    (8, 8, [9000]), (32, 8, [300]), (32, 8, [16, 17, 511, 512, 513, 2000]), (8, 2, [20000] + [30] * 40),
    (2, 2, [190] * 77), (32, 8, list(range(1, 1200, 7)))])
def test_decode_counts_every_tile(hq, hkv, lens):
    w = wl.make_workload("tiles", lens, np.zeros(len(lens), int), seed=len(lens), pool_slack=0.02)
    cache, q, ref = coded(w, hkv, hq)
    status = pa.new_device_status()
    for flags in (pa.PA_LAUNCH_DEFAULT, pa.PA_LAUNCH_MAX_SMS(1), pa.PA_LAUNCH_MAX_SMS(37)):
        out = torch.full_like(q, float("nan"))
        pa.pa_decode_q8(out, q, *cache, i32(w.block_tables), i32(w.context_lens), 0.125, max(lens), launch_flags=flags,
                        device_status=status)
        counted(out, ref, f"flags {flags:#x}")
    assert pa.pa_check_device_status(status) == pa.PA_OK


@gpu
@pytest.mark.parametrize("hq,hkv,prior,new", [
    (32, 8, [131067], [5]), (4, 1, [131064, 0, 100], [8, 3, 1]), (32, 8, [131071, 9000, 16, 511], [1, 4, 2, 8]),
    (2, 1, [50000] + [300] * 60, [16] + [7] * 60), (8, 8, [1] * 160, [32] * 160),
    (32, 8, list(range(0, 1500, 31)), [5] * 49)])
def test_few_rows_count_every_tile(hq, hkv, prior, new):
    chunks(hq, hkv, prior, new)


@gpu
@pytest.mark.parametrize("hq,hkv,prior,new", [
    (4, 1, [131000, 0], [72, 65]), (32, 8, [40000], [9]), (32, 8, [5000, 0, 63, 127], [130, 65, 64, 257]),
    (2, 1, [30000, 129], [300, 127]), (2, 2, [8191], [513]), (32, 8, list(range(0, 1500, 31)), [70] * 49)])
def test_chunks_count_every_tile(hq, hkv, prior, new):
    chunks(hq, hkv, prior, new)


def chunks(hq, hkv, prior, new):
    w = wl.make_workload("tiles", prior, new, num_prefill=len(new), seed=len(new), pool_slack=0.02)
    cache, q, ref = coded(w, hkv, hq, w.new_lens)
    status = pa.new_device_status()
    out = torch.full_like(q, float("nan"))
    pa.pa_prefill_chunk_q8(out, q, i32(w.new_start_loc), max(new), *cache, i32(w.block_tables), i32(w.context_lens),
                           0.125, device_status=status)
    counted(out, ref, "chunk")
    assert pa.pa_check_device_status(status) == pa.PA_OK


# ---- one key that outweighs the rest ----------------------------------------------------------------
PEAK = 20.0  # a planted key's score; every other score is 0


def planted(length, rows, places, seed):
    """One sequence, 8 K/V heads with a group of 4: every key is zero but head h's key of token
    places[h], whose score is 20 (64 codes of 2.5 under queries of 1, times 1 / 8: exact); random V.

    A row that sees the planted token: o = (e^20 v_p + sum of the others' v) / (e^20 + n - 1).  The
    others weigh at most 131,071 e^-20 < 2.8e-4 together; however their weights are rounded (each
    within a factor of 2), they move o by less than 3 x 2.8e-4 x 6 (no |v| is larger).  The rest:
    half a bf16 step of o, 2^-8 for the planted weight's own rounding at worst (bf16), 2^-16 for
    exponentials and sums."""
    hkv, hq = 8, 32
    w = wl.make_workload("peak", [length - rows], [rows], num_prefill=1, seed=seed, pool_slack=0.02)
    kc, vc, ks, vs = tables_of(w, hkv, seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    blocks, slots = live_slots(w, 0)
    v = torch.randn(length, hkv, 64, generator=g, device="cuda").to(torch.float8_e4m3fn)
    vc[blocks, :, slots] = v.view(torch.uint8)
    kc.zero_()
    ks[blocks] = 1.0
    code = int(torch.tensor(2.5).to(torch.float8_e4m3fn).view(torch.uint8))
    v = v.double()
    total = v.cumsum(0)
    ref = torch.empty(rows, hkv, 64, dtype=torch.float64, device="cuda")
    tol = torch.empty_like(ref)
    peak = float(np.exp(PEAK))
    for h, t in enumerate(places):
        kc[blocks[t], h, slots[t]] = code
        for i in range(rows):
            seen = length - rows + i + 1
            if t < seen:
                o = (total[seen - 1, h] + (peak - 1) * v[t, h]) / (peak + seen - 1)
                ref[i, h] = o
                tol[i, h] = 2.0 ** -8 * o.abs() + 3 * 2.8e-4 * 6.0 + (2.0 ** -8 + 2.0 ** -16) * v[t, h].abs()
            else:  # the plain mean of the others, all of weight 1: exact sums of codes, see coded()
                o = total[seen - 1, h] / seen
                ref[i, h], tol[i, h] = o, 2.0 ** -8 * o.abs() + 2.0 ** -12
    q = torch.ones(rows, hq, 64, dtype=torch.bfloat16, device="cuda")
    return w, views(kc, vc, ks, vs), q, ref.repeat_interleave(4, dim=1), tol.repeat_interleave(4, dim=1)


def at_edges(length, seed):
    """Token places at tile 0, the last tile, around multiples of 32 tiles, around the ends of twelfths
    and of the decode's runs, and anywhere."""
    nb = -(-length // 16)
    runs = np.arange(1, 152 * 12) * nb // (152 * 12 // 8 if nb > 1000 else 12)
    tiles = np.concatenate([[0, 1, nb - 1, nb - 2], np.arange(31, nb, 32)[:40], np.arange(32, nb, 32)[-40:],
                            np.arange(1, 12) * nb // 12, np.arange(1, 12) * nb // 12 - 1, runs[:60]])
    rng = np.random.default_rng(seed)
    tiles = np.unique(np.clip(tiles, 0, nb - 1))
    tiles = np.concatenate([rng.choice(tiles, 40), rng.integers(0, nb, 24)])
    return np.minimum(tiles * 16 + rng.integers(0, 16, len(tiles)), length - 1).reshape(-1, 8)


@gpu
@pytest.mark.parametrize("length", [300, 2000, 9000, 131072])
@pytest.mark.parametrize("rows", [1, 5, 40])
def test_a_planted_key_is_found(length, rows):
    for seed, places in enumerate(at_edges(length, length + rows)):
        w, cache, q, ref, tol = planted(length, rows, places.tolist(), seed)
        status = pa.new_device_status()
        bt, ctx = i32(w.block_tables), i32(w.context_lens)
        outs = {}
        if rows == 1:
            outs["decode"] = torch.full_like(q, float("nan"))
            pa.pa_decode_q8(outs["decode"], q, *cache, bt, ctx, 0.125, length, device_status=status)
        outs["chunk"] = torch.full_like(q, float("nan"))
        pa.pa_prefill_chunk_q8(outs["chunk"], q, i32(w.new_start_loc), rows, *cache, bt, ctx, 0.125,
                               device_status=status)
        for what, out in outs.items():
            bad = ~((out.double() - ref).abs() <= tol)
            assert not bad.any(), f"{what}: tokens {places.tolist()}, first (row, head, dim) {bad.nonzero()[0].tolist()}"
        assert pa.pa_check_device_status(status) == pa.PA_OK
