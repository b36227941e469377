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


@pytest.mark.parametrize("width", [0, 20])
@pytest.mark.parametrize("table,base,keep,bad", [
    ([[4, -1]], 0, [0, 1], False), ([[4, -1]], 0, [0, 1, 2], True), ([[4, 9]], 0, [0, 1, 2], True), ([[4, -7]], 2, [0], True),
    ([[4, 5]], 3, [0, 1], True), ([[4, 5]], 4, [0], True), ([[4, 5]], 2 ** 31 - 1, [0], True), ([[4, 5]], 2, [0, 1], False)])
def test_kept_rows_that_are_not_held_are_flagged(table, base, keep, bad, width):
    """Also where a row would stay at its place: a table that does not hold it is the caller's mistake all the same."""
    V.v4_reset_device_status()
    cache = torch.from_numpy(np.random.default_rng(3).integers(0, 255, (6, 2, 16), dtype=np.uint8)).cuda()
    was = cache.clone()
    lists = np.full((1, max(len(keep), width)), 7)
    lists[0, :len(keep)] = keep
    V.v4_pages_compact(cache, i32(table), i32([base]), i32([len(keep)]), i32(lists))
    assert torch.equal(cache, was)
    assert flagged() == bad
