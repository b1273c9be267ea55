"""pa_compact_tokens and its 8-bit form at the ends of their arguments' range."""
import pytest

from paged_kv_cache_299_gb300 import binding as pa
from _gpu import i32
from test_gpu_compact import POOLS, Cache

pytestmark = pytest.mark.gpu
LAST = (1 << 31) - 1


@pytest.mark.parametrize("pool", POOLS)
@pytest.mark.parametrize("first", [LAST, LAST - 2, LAST - 3, LAST - 4, LAST - 16, LAST - 40])
@pytest.mark.parametrize("entries", [4, 40])
def test_destinations_past_the_end_of_the_ints(pool, first, entries):
    """A wrong `first` whose list would end past 2^31 - 1 is reported and its sequence left alone."""
    c = Cache(pool, [20, 33, 0], [[1, 3, 9], list(range(1, 2 * entries, 2)), [4, 5]], 2, seed=8)
    c.run(first=i32([20, first, 0]))
    assert int(c.status.item()) == pa.DEVFLAG_BAD_CONTEXT
    c.check(skip=[1])
