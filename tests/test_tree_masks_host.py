"""Trees' masks on the host: borders are looked at, all of them, before any parent is read."""
import numpy as np
import pytest
import torch

import paged_kv_cache_166_gb300 as pkv
from paged_kv_cache_166_gb300 import _native as N


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32)


# what lies behind the parents: no parent of anything, so that a look at it shows in the message
BEHIND = 1 << 24


def parents_with_room(n, room):
    room = torch.full((n + room,), BEHIND, dtype=torch.int32)
    room[:n] = torch.arange(-1, n - 1, dtype=torch.int32)
    return room[:n]


@pytest.mark.parametrize("starts", [[0, 500, 12], [0, 13, 12], [0, 4, 13, 12], [0, 12, 13, 12],
                                    [0, -1, 12], [0, 600, 3, 12]])
def test_borders_out_of_order_are_refused_before_parents_are_read(starts):
    parents = parents_with_room(12, 700)
    for words in (0, 40):
        with pytest.raises(pkv.PkvError, match="must not decrease"):
            pkv.tree_masks(parents, i32(starts), words=words)


def test_a_border_far_out_allocates_nothing_of_its_size():
    with pytest.raises(pkv.PkvError, match="must not decrease"):
        pkv.tree_masks(parents_with_room(12, 0), i32([0, 2 ** 31 - 1, 12]))


def test_nothing_is_written_for_borders_out_of_order():
    parents, starts = parents_with_room(12, 700), i32([0, 5, 600, 12])
    mask = torch.full((12, 20), 77, dtype=torch.int32)
    depths = torch.full((12,), 77, dtype=torch.int32)
    rc = N.lib().pkv_tree_masks(parents.data_ptr(), starts.data_ptr(), 3, 20, mask.data_ptr(),
                                depths.data_ptr())
    assert rc == N.PKV_ERR_INVALID_ARG
    assert (mask == 77).all() and (depths == 77).all()
