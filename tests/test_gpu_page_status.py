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


def forked(table, ref, src, length, out_blocks, page):
    """Fork by its definition: a page whose count is 0 when the call begins is none."""
    free, shared = [p for p, n in enumerate(ref) if n == 0], list(ref)
    out, copies, bad = np.full((len(src), out_blocks), -1), [], False

    def held(p):
        nonlocal bad
        good = p == -1 or (0 <= p < len(ref) and ref[p] > 0)
        bad = bad or not good
        return p if good else -1
    for i, (s, n) in enumerate(zip(src, length)):
        copy = [-1, -1, 0]
        for k in range(n // page):
            out[i, k] = held(table[s][k])
            if out[i, k] >= 0:
                shared[out[i, k]] += 1
        if n % page:
            old = held(table[s][n // page])
            if old >= 0 and free:
                out[i, n // page] = free.pop(0)
                shared[out[i, n // page]] = 1
                copy = [old, out[i, n // page], n % page]
        copies.append(copy)
    return out, copies, shared, bad


@pytest.mark.parametrize("beams", [1, 3, 64, 1500, 6000])      # one launch up to 14336 entries, two above
@pytest.mark.parametrize("zero", [[], [0], [1], [2], [0, 1, 2], [0, 5]])
def test_fork_shares_and_copies_no_free_page(zero, beams):
    """Pages 0, 1 whole and 2 partly filled; some of them are free by their counts, so they are the first to be given."""
    V.v4_reset_device_status()
    page, pages, table = 4, 8 + beams, [[0, 1, 2]]
    ref = [1, 1, 1] + [0] * (pages - 3)
    for z in zero:
        ref[z] = 0
    src, length = [0] * beams, [10 - i % 3 for i in range(beams)]
    want, copies, shared, bad = forked(table, ref, src, length, 3, page)
    assert bad == bool(zero)
    for _ in range(20):
        counts, out, cp = i32(ref), i32(np.full((beams, 3), 9)), i32(np.full((beams, 3), 9))
        V.v4_pages_fork(i32(table), i32(src), i32(length), out, counts, page, cp)
        same(out, want), same(cp, copies), same(counts, shared)
        assert flagged() == bad


def test_beams_step_by_step_without_a_pause():
    """The beams of a step give their pages back and the next are forked at once, each call right behind the one before."""
    rng = np.random.default_rng(8)
    page, blocks, n, steps = 8, 6, 90, 60
    pages = 3 * blocks + n + 5
    perm = rng.permutation(pages)
    table = perm[:3 * blocks].reshape(3, blocks)
    ref = np.zeros(pages, int)
    ref[table] = 1
    src = rng.integers(-1, 3, (steps, n))
    length = rng.integers(0, page * blocks + 1, (steps, n))
    dt, dref = i32(table), i32(ref)
    dsrc, dlen = [i32(s) for s in src], [i32(s) for s in length]
    outs = [i32(np.full((n, blocks), -1)) for _ in range(steps + 1)]
    copies = [i32(np.full((n, 3), 9)) for _ in range(steps)]
    torch.cuda.synchronize()
    for k in range(steps):
        V.v4_pages_fork(dt, dsrc[k], dlen[k], outs[k + 1], dref, page, copies[k])
        V.v4_pages_free(outs[k + 1], dref, page)          # all of them: -1 again
    for k in range(steps):                                # and with the pages kept for a step
        V.v4_pages_free(outs[k], dref, page)
        V.v4_pages_fork(dt, dsrc[k], dlen[k], outs[k + 1], dref, page, copies[k])
    for k in range(steps):
        want, cp, ref2, bad = forked(table, list(ref), src[k], np.where(src[k] < 0, 0, length[k]), blocks, page)
        assert not bad
        same(copies[k], cp)
    same(outs[steps], want), same(dref, ref2)
    assert not flagged()


def test_pages_outside_the_pool_are_replaced_when_pages_are_given():
    """Taken for -1, as in a fork or a release: flagged, and the entry gets a page where its tokens want one."""
    V.v4_reset_device_status()
    table, ref, lack = i32([[4, 1, -5, 7], [-1, 2 ** 31 - 1, 0, -1]]), i32([1, 1, 0, 0]), i32([9])
    V.v4_pages_alloc(table, ref, i32([12, 8]), 4, lack=lack)
    same(table, [[2, 1, 3, 7], [-1, -1, 0, -1]])
    same(ref, [1, 1, 1, 1]), same(lack, [2])
    assert flagged()
    table = i32([[4, 1, 0, 7]])
    V.v4_pages_alloc(table, ref, i32([12]), 4, have=i32([4]))       # block 0 and block 3 are not looked at
    same(table, [[4, 1, 0, 7]])
    assert not flagged()


def test_tokens_that_the_table_does_not_hold_are_flagged():
    V.v4_reset_device_status()
    ref = i32([0, 0, 0])
    for have, need, bad in ((9, 4, True), (2 ** 31 - 1, 8, True), (8, 8, False), (8, 3, False), (-1, 3, True), (0, 9, True), (0, -1, True)):
        table = i32([[-1, -1]])
        V.v4_pages_alloc(table, ref, i32([need]), 4, have=i32([have]))
        same(table, [[-1, -1]]), same(ref, [0, 0, 0])
        assert flagged() == bad, (have, need)


def test_a_captured_beam_step_replays():
    """Release, fork and copies of 70 beams in a graph; the table, lengths and counts change between replays."""
    rng = np.random.default_rng(12)
    page, blocks, n, layers = 8, 5, 70, 2
    pages = 4 * blocks + n + 3
    dt, dref = i32(np.zeros((4, blocks))), i32(np.zeros(pages))
    dsrc, dlen, out, copies = i32(np.zeros(n)), i32(np.zeros(n)), i32(np.full((n, blocks), -1)), i32(np.zeros((n, 3)))
    lack = i32([9])
    cache = torch.zeros(layers, pages, page, 32, dtype=torch.uint8, device="cuda")

    def step():
        V.v4_pages_free(out, dref, page)
        V.v4_pages_fork(dt, dsrc, dlen, out, dref, page, copies, lack=lack)
        V.v4_pages_copy(cache, copies)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(4):
        table = rng.permutation(pages)[:4 * blocks].reshape(4, blocks)
        ref = np.zeros(pages, int)
        ref[table] = 1
        src, length = rng.integers(0, 4, n), rng.integers(0, page * blocks + 1, n)
        want, cp, counts, bad = forked(table, list(ref), src, length, blocks, page)
        rows = torch.from_numpy(rng.integers(0, 255, tuple(cache.shape), dtype=np.uint8))
        moved_rows = rows.clone()
        for a, b, r in cp:
            if a >= 0:
                moved_rows[:, b, :r] = rows[:, a, :r]
        dt.copy_(i32(table)), dref.copy_(i32(ref)), dsrc.copy_(i32(src)), dlen.copy_(i32(length)), out.fill_(-1), cache.copy_(rows)
        graph.replay()
        same(out, want), same(copies, cp), same(dref, counts), same(lack, [0])
        assert torch.equal(cache.cpu(), moved_rows) and not bad
    assert not flagged()
