"""What the Python side of the tree calls and the appends at positions takes, without a GPU."""
import numpy as np
import pytest
import torch

from paged_kv_cache_299_gb300 import binding as pa


def test_pair_axes_are_whole_numbers_of_any_type():
    """Equal numbers of another type must not depend on which came first."""
    want = sum(2 << (2 * i) for i in range(32))
    for axes in (np.full(32, 2), [np.int32(2)] * 32, torch.full((32,), 2, dtype=torch.int32), bytes([2] * 32), [2] * 32,
                 (2,) * 32, range(2, 3)):
        if len(axes) == 32:
            assert pa._pair_axes(axes, 3) == want
        else:
            with pytest.raises(ValueError):
                pa._pair_axes(axes, 3)
    assert pa._pair_axes([0, 1, 2, 3] * 8, 4) == sum((i % 4) << (2 * i) for i in range(32))


@pytest.mark.parametrize("axes", [[1.0] * 32, np.ones(32), torch.ones(32), [None] * 32, ["1"] * 32, 32, 1.5, [1] * 33, [],
                                  [1] * 31 + [256], [1] * 31 + [1 << 40], [1] * 31 + [-1], [1] * 31 + [4]])
def test_pair_axes_that_are_none_are_refused(axes):
    """Also after equal ones were taken."""
    for _ in range(2):
        with pytest.raises(ValueError):
            pa._pair_axes(axes, 4)
        pa._pair_axes([1] * 32, 4)


@pytest.mark.parametrize("rows", [0, 1, 5])
def test_masks_of_no_drafted_tokens(rows):
    packed = pa.pack_tree_mask(torch.zeros(rows, 0, dtype=torch.bool))
    assert packed.dtype is torch.int32 and packed.shape == (rows, 0)


def test_masks_that_are_not_contiguous():
    seen = torch.rand(40, 70, generator=torch.Generator().manual_seed(1)) < 0.5
    assert torch.equal(pa.pack_tree_mask(seen.t().contiguous().t()), pa.pack_tree_mask(seen))
    assert torch.equal(pa.pack_tree_mask(seen[:, :64]), pa.pack_tree_mask(seen)[:, :2])
