"""pa_tree_attention where neighbouring segments of many pieces meet in one CTA (test_tree_plan shows that these
batches' do): rows against attention in 64 bits, again and again on one workspace, whose counters stay zero."""
import pytest
import torch

from paged_kv_cache_299_gb300 import binding as pa
from _tree import MEETING_BATCHES
from test_gpu_tree import Trees

pytestmark = pytest.mark.gpu


def counters(workspace):
    """The workspace's counters: three arrays of 16 per SM ahead of the records."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return workspace[:3 * (-(-sms * 64 // 256) * 256)]


@pytest.mark.parametrize("name", sorted(MEETING_BATCHES))
def test_segments_that_meet_in_a_cta(name):
    pool, hkv, hist, nodes = MEETING_BATCHES[name]
    t = Trees(pool, hist, nodes, 4 * hkv, hkv, seed=len(hist), slack=0.05)
    ws = torch.zeros(pa.pa_tree_workspace_size(), dtype=torch.uint8, device="cuda")
    first = t.run(workspace=ws)
    t.check(first)
    assert not counters(ws).any()
    for _ in range(30):
        assert torch.equal(t.run(workspace=ws), first)
        assert not counters(ws).any()


@pytest.mark.parametrize("pool", ["bf16", "q8"])
def test_segments_that_meet_beside_another_stream(pool):
    """CTAs that another kernel holds up deliver in another order."""
    name = {"bf16": "bf16 one half", "q8": "q8 short ones behind"}[pool]
    pool, hkv, hist, nodes = MEETING_BATCHES[name]
    t = Trees(pool, hist, nodes, 4 * hkv, hkv, seed=3, slack=0.05)
    ws = torch.zeros(pa.pa_tree_workspace_size(), dtype=torch.uint8, device="cuda")
    want = t.run(workspace=ws)
    t.check(want)
    x = torch.zeros(64 << 20, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        with torch.cuda.stream(side):
            for _ in range(4):
                x.add_(1.0)
        assert torch.equal(t.run(workspace=ws), want)
    torch.cuda.synchronize()
    assert not counters(ws).any()
