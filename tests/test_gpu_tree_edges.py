"""pa_tree_attention where rows, masks and codes are at the ends of what its documentation allows."""
import pytest
import torch

from paged_kv_cache_299_gb300 import binding as pa
from _gpu import i32
from test_gpu_tree import POOLS, Trees, close

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("code", [0x7f, 0xff])
@pytest.mark.parametrize("hist,n,hq,hkv", [(0, 7, 4, 1), (50, 8, 8, 2), (61, 30, 3, 3), (1000, 6, 4, 1), (0, 20, 4, 1),
                                           (60, 70, 2, 2)])
def test_codes_that_are_no_numbers_reach_no_row_that_does_not_see_them(code, hist, n, hq, hkv):
    """A drafted token's key or value codes, on the few-rows kernel (up to 32 rows per K/V head) and the other."""
    for which in (0, 1):
        t = Trees("q8", [hist, 10], [n, 5], hq, hkv, "tree", seed=11)
        pos = hist + n // 2
        clean = t.check().to(torch.bfloat16)
        t.dev[which].view(torch.uint8)[int(t.w.block_tables[0, pos // 16]), :, pos % 16, 5:40] = code
        got = t.run().cpu()
        assert t.ok()
        blind = [i for i in range(t.rows) if i >= n or not t.bits[0][i] >> (n // 2) & 1]
        assert 5 < len(blind) < t.rows
        assert torch.equal(got[blind], clean[blind])


@pytest.mark.parametrize("code", [0x7f, 0xff])
def test_codes_that_are_no_numbers_reach_no_earlier_row_of_a_chunk(code):
    t = Trees("q8", [100, 3], [8, 5], 4, 1, "chain", seed=12)

    def chunk():
        out = torch.zeros_like(t.q, device="cuda")
        pa.pa_prefill_chunk_q8(out, t.q.cuda(), t.starts, t.most, *t.dev, t.bt, t.ctx, 0.125)
        return out.cpu()

    clean = chunk()
    assert torch.isfinite(clean).all()
    t.dev[1].view(torch.uint8)[int(t.w.block_tables[0, 105 // 16]), :, 105 % 16, :] = code
    got = chunk()
    blind = [i for i in range(t.rows) if i < 5 or i >= 8]
    assert torch.equal(got[blind], clean[blind])


@pytest.mark.parametrize("pool", POOLS)
@pytest.mark.parametrize("most", [4, 9])  # over 8 bits the few-rows kernel and the other
def test_starts_that_fall_are_reported(pool, most):
    """A sequence of fewer than no rows has none; the others' rows are right, and no other row is written."""
    t = Trees(pool, [30, 40, 50], [4, 2, 3], 4, 1, seed=13)
    ref, tol = t.expected()
    at = {0: 6, 1: 7, 2: 8, 5: 0, 6: 1, 7: 2, 8: 3}  # rows of the call: the third sequence's, then the first's
    q, mask = t.q.clone(), t.mask.clone()
    for row, old in at.items():
        q[row], mask[row] = t.q[old], t.mask[old]
    got = t.run(q=q.cuda(), mask=mask, starts=i32([5, 9, 0, 3]), most=most).cpu().double()
    assert int(t.status.item()) == pa.DEVFLAG_BAD_CONTEXT
    close(got[list(at)], ref[list(at.values())], tol[list(at.values())])
    assert (got[[3, 4]] == 7.0).all()


@pytest.mark.parametrize("pool", POOLS)
@pytest.mark.parametrize("count", [1, 33])
def test_empty_sequences_are_not_reported(pool, count):
    """Also with a context of 0, as padding has it; among up to 32 sequences and among more."""
    t = Trees(pool, [30] + [0] * count, [4] + [0] * count, 4, 1, seed=14)
    t.check()
    t.check(t.run(ctx=i32([34] + [-1] * count)))


@pytest.mark.parametrize("pool", POOLS)
def test_two_calls_at_once(pool):
    """On two streams, each with a workspace of its own."""
    batches = [Trees(pool, [9000] * 3 + [200] * 9, [70] * 12, 8, 2, seed=15), Trees(pool, [20000, 30], [12, 9], 8, 2, seed=16)]
    spaces = [torch.zeros(pa.pa_tree_workspace_size(), dtype=torch.uint8, device="cuda") for _ in batches]
    want = [t.run(workspace=ws) for t, ws in zip(batches, spaces)]
    for t, got in zip(batches, want):
        t.check(got)
    f = pa.pa_tree_attention_q8 if pool == "q8" else pa.pa_tree_attention
    queries = [t.q.cuda() for t in batches]
    outs = [[torch.zeros_like(q) for _ in range(20)] for q in queries]
    streams = [torch.cuda.Stream() for _ in batches]
    torch.cuda.synchronize()
    for turn in range(20):
        for t, ws, q, out, stream in zip(batches, spaces, queries, outs, streams):
            f(out[turn], q, t.mask, t.starts, t.most, *t.dev, t.bt, t.ctx, 0.125, workspace=ws, device_status=t.status,
              stream=stream)
    torch.cuda.synchronize()
    for t, first, out in zip(batches, want, outs):
        assert t.ok() and all(torch.equal(x, first) for x in out)
