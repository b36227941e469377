"""Page calls with bad values: what is flagged, and that nothing else changes."""
import numpy as np
import pytest
import torch

import sparse_compressed_attention_gb300 as V

pytestmark = pytest.mark.gpu


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32).cuda()


def same(t, want):
    assert np.array_equal(t.cpu().numpy(), np.array(want, np.int32).reshape(tuple(t.shape)))


def flagged():
    s = V.v4_get_device_status()
    V.v4_reset_device_status()
    assert s in (0, 6)
    return s == 6


def moved(rows, keep):
    """Rows after the list, and whether an entry is not above the one before or below its own number."""
    out, bad, before = rows.clone(), False, -1
    for i, k in enumerate(keep):
        if k <= before or k < i:
            bad = True
        else:
            out[i] = rows[k]
        before = k
    return out, bad


BOUNDARY = list(range(127)) + [128, 128] + list(range(129, 200))      # the second 128 opens a round of 128 rows
LISTS = [([1, 1], True), ([5, 1], True), ([0, 3, 2], True), ([2, 2, 1], True), ([0, 1, 1], True), ([3, -1], True),
         ([0, 1, 2], False), ([0, 2, 3, 9], False), (BOUNDARY, True), (list(range(1, 201)), False)]


@pytest.mark.parametrize("width", [0, 20])                            # lists of up to 16 and longer ones have kernels of their own
@pytest.mark.parametrize("keep,bad", LISTS)
def test_kept_lists_that_do_not_ascend_are_flagged(keep, bad, width):
    V.v4_reset_device_status()
    page, pages = 8, 30
    cache = torch.from_numpy(np.random.default_rng(len(keep)).integers(0, 255, (1, pages, page, 288), dtype=np.uint8)).cuda()
    rows = cache[0].view(-1, 288).clone()
    want, expected = moved(rows, keep)
    assert expected == bad
    lists = np.full((1, max(len(keep), width)), 7)
    lists[0, :len(keep)] = keep
    V.v4_pages_compact(cache, i32([np.arange(pages)]), i32([0]), i32([len(keep)]), i32(lists))
    assert torch.equal(cache[0].view(-1, 288), want)
    assert flagged() == bad
