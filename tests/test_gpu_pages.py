"""Pages of a cache: given, forked, released, copied, compacted, against the step-by-step oracle."""
import numpy as np
import pytest
import torch

import sparse_compressed_attention_gb300 as V
from oracle import cache_oracle as CO

pytestmark = pytest.mark.gpu


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32).cuda()


def same(t, want):
    assert np.array_equal(t.cpu().numpy(), np.array(want, np.int32).reshape(tuple(t.shape)))


@pytest.mark.parametrize("B,pages,page,most", [(1, 1, 1, 1), (3, 40, 4, 30), (40, 3000, 16, 900), (700, 9001, 8, 100),
                                               (5, 30000, 1, 5000), (8192, 8192, 4, 4)])
def test_pages_given_and_released(B, pages, page, most):
    """Sequences grow, give back their first and last tokens, and grow again."""
    rng = np.random.default_rng(B)
    blocks = -(-most // page) + 1
    used = rng.random(pages) < 0.3
    o = CO.Pages([[-1] * blocks] * B, used.astype(int), page)
    o.table = [list(r) for r in o.table]
    table, ref, lack = i32(o.table), i32(o.ref), torch.full((1,), 7, dtype=torch.int32, device="cuda")
    have = np.zeros(B, int)
    for step in range(3):
        need = np.maximum(have, rng.integers(0, most + 1, B))
        want = o.alloc([0] * B if step == 0 else list(have), list(need))
        V.v4_pages_alloc(table, ref, i32(need), page, have=None if step == 0 else i32(have), lack=lack)
        assert int(lack) == want
        same(table, o.table), same(ref, o.ref)
        lo = rng.integers(0, most // 2 + 1, B)
        hi = np.maximum(lo, rng.integers(0, most + 1, B))
        o.free(lo, hi)
        V.v4_pages_free(table, ref, page, lo=i32(lo), hi=i32(hi))
        same(table, o.table), same(ref, o.ref)
        have = hi
    V.v4_pages_free(table, ref, page)
    assert (table == -1).all()
    same(ref, used.astype(int))
    assert V.v4_get_device_status() == 0


def test_entries_that_hold_a_page_keep_it():
    table, ref = i32([[-1, 5, -1, -1], [2, -1, 0, -1]]), i32([1, 0, 1, 0, 0, 1, 0])
    V.v4_pages_alloc(table, ref, i32([16, 9]), 4, have=i32([3, 4]))
    same(table, [[-1, 5, 1, 3], [2, 4, 0, -1]])
    same(ref, [1, 1, 1, 1, 1, 1, 0])
    assert V.v4_get_device_status() == 0


def test_more_wanted_than_one_list_holds():
    """20000 entries of a few sequences, and more than there are pages."""
    o = CO.Pages([[-1] * 7000] * 3, np.arange(20500) % 41 == 3, 2)
    o.table = [list(r) for r in o.table]
    table, ref, lack = i32(o.table), i32(o.ref), i32([0])
    free = [p for p, n in enumerate(o.ref) if n == 0]
    V.v4_pages_alloc(table, ref, i32([14000, 14000, 13000]), 2, lack=lack)
    want = np.full((3, 7000), -1)
    flat = np.concatenate([want[0], want[1], want[2][:6500]])
    flat[:len(free)] = free[:len(flat)]
    want[0], want[1], want[2, :6500] = flat[:7000], flat[7000:14000], flat[14000:]
    same(table, want)
    assert int(lack) == max(0, 20500 - len(free)) and (ref == 1).all()


def beams(seed, B, n, page, most, pages, holes=False):
    rng = np.random.default_rng(seed)
    blocks = -(-most // page)
    lens = rng.integers(0, most + 1, B)
    o = CO.Pages([[-1] * blocks] * B, [0] * pages, page)
    o.table = [list(r) for r in o.table]
    perm, at = rng.permutation(pages), 0
    for b in range(B):
        for k in range(o.blocks(int(lens[b]))):
            if holes and rng.random() < 0.2:
                continue
            o.table[b][k] = int(perm[at])
            o.ref[perm[at]] = 1
            at += 1
    src = rng.integers(-1, B, n)
    length = np.array([0 if s < 0 else rng.integers(0, lens[s] + 1) for s in src])
    return o, src, length, blocks


@pytest.mark.parametrize("B,n,page,most,pages", [(1, 1, 4, 9, 8), (4, 9, 16, 200, 300), (16, 64, 64, 2000, 700), (3, 2000, 8, 60, 2100),
                                                 (2, 5, 1, 50, 400)])
@pytest.mark.parametrize("holes", [False, True])
def test_fork(B, n, page, most, pages, holes):
    o, src, length, blocks = beams(B + n, B, n, page, most, pages, holes)
    table, ref = i32(o.table), i32(o.ref)
    out = torch.full((n, blocks + 1), 99, dtype=torch.int32, device="cuda")
    copies, lack = torch.full((n, 3), 99, dtype=torch.int32, device="cuda"), i32([9])
    rows, want, short = o.fork(src, length, blocks + 1)
    V.v4_pages_fork(table, i32(src), i32(length), out, ref, page, copies, lack=lack)
    same(out, rows), same(copies, want), same(ref, o.ref), same(table, o.table)
    assert int(lack) == short and V.v4_get_device_status() == 0


def test_fork_without_pages_left():
    V.v4_reset_device_status()
    table, ref = i32([[0, 1]]), i32([1, 1, 0])
    out, copies = i32(np.zeros((3, 2))), i32(np.zeros((3, 3)))
    V.v4_pages_fork(table, i32([0, 0, 0]), i32([6, 8, 5]), out, ref, 4, copies)
    same(out, [[0, 2], [0, 1], [0, -1]])
    same(copies, [[1, 2, 2], [-1, -1, 0], [-1, -1, 0]])
    same(ref, [4, 2, 1])
    assert V.v4_get_device_status() == 6                          # nobody asked for `lack`
    V.v4_reset_device_status()


def test_bad_values_are_flagged_and_touch_nothing():
    def flagged():
        s = V.v4_get_device_status()
        V.v4_reset_device_status()
        return s == 6
    V.v4_reset_device_status()
    table, ref = i32([[0, 1], [-1, -1]]), i32([1, 1, 0, 0])
    V.v4_pages_alloc(table, ref, i32([8, 9]), 4)                  # sequence 1 does not fit its row
    same(table, [[0, 1], [-1, -1]])
    assert flagged()
    out, copies = i32(np.full((4, 2), 7)), i32(np.full((4, 3), 7))
    V.v4_pages_fork(table, i32([2, 0, -2, 0]), i32([1, 9, 1, -1]), out, ref, 4, copies)
    same(out, np.full((4, 2), -1))
    same(ref, [1, 1, 0, 0])
    assert flagged()
    bad = i32([[4, 1], [0, -5]])
    V.v4_pages_fork(bad, i32([0, 1]), i32([8, 8]), out[:2], ref, 4, copies[:2])
    same(out[:2], [[-1, 1], [0, -1]])
    assert flagged()
    ref = i32([1, 0, 0, 0])
    table = i32([[0, 3], [8, -1]])
    V.v4_pages_free(table, ref, 4)                                # page 3 is free, page 8 is none
    same(table, [[-1, -1], [-1, -1]])
    same(ref, [0, 0, 0, 0])
    assert flagged()
    cache = torch.arange(4 * 2 * 16, dtype=torch.uint8).view(4, 2, 16).cuda()
    was = cache.clone()
    V.v4_pages_copy(cache, i32([[0, 4, 1], [-1, 2, 1], [0, 1, 3], [1, 1, 2], [-1, -1, 0], [9, 9, 0]]))
    assert torch.equal(cache, was) and flagged()
    V.v4_pages_compact(cache, i32([[0, 1], [2, 9], [3, -1]]), i32([0, 1, -1]), i32([3, 1, 1]), i32([[2, 2, 1], [1, 0, 0], [0, 0, 0]]))
    was[0, 0] = was[1, 0]                                          # row 2 of sequence 0 to row 0; the rest is not ascending or not held
    assert torch.equal(cache, was) and flagged()


@pytest.mark.parametrize("width,dt,layers", [(288, torch.uint8, 3), (512, torch.bfloat16, 2), (8, torch.bfloat16, 1), (520, torch.float32, 2)])
def test_copies(width, dt, layers):
    rng = np.random.default_rng(width)
    page, pages, n = 24, 30, 9
    cache = torch.from_numpy(rng.integers(0, 100, (layers, pages, page, width))).to(dt).cuda()
    perm = rng.permutation(pages)
    copies = np.stack([perm[:n] % 30, perm[n:2 * n], rng.integers(0, page + 1, n)], 1)
    copies[2] = (-1, -1, 0)
    copies[3] = (perm[0], perm[n + 3], page)                      # one source twice
    want = cache.clone()
    for a, b, r in copies:
        if a >= 0:
            want[:, b, :r] = cache[:, a, :r]
    V.v4_pages_copy(cache, i32(copies))
    assert torch.equal(cache, want)
    one = cache[0]
    V.v4_pages_copy(one, i32([[1, 2, page]]))                     # three dims: one layer
    assert torch.equal(one[2], one[1]) and V.v4_get_device_status() == 0


@pytest.mark.parametrize("B,span,width,dt,layers", [(1, 1, 512, torch.bfloat16, 1), (7, 40, 288, torch.uint8, 5), (3, 900, 512, torch.bfloat16, 2),
                                                    (2, 3000, 512, torch.bfloat16, 1), (40, 16, 520, torch.float32, 3),
                                                    (2, 700, 16, torch.uint8, 1)])
@pytest.mark.parametrize("page", [1, 7, 64])
def test_compaction(B, span, width, dt, layers, page):
    rng = np.random.default_rng(B + span)
    base = rng.integers(0, 100, B)
    blocks = -(-(int(base.max()) + span) // page)
    pages = B * blocks + 2
    table = rng.permutation(pages)[:B * blocks].reshape(B, blocks)
    keep = [sorted(rng.choice(span, rng.integers(0, span + 1), replace=False).tolist()) for _ in range(B)]
    if B > 2:
        keep[0], keep[1] = list(range(span)), [span - 1]
    wide = max(1, max(len(k) for k in keep)) + 1
    lists = np.full((B, wide), -5)
    for b in range(B):
        lists[b, :len(keep[b])] = keep[b]
    cache = torch.from_numpy(rng.integers(0, 100, (layers, pages, page, width))).to(dt)
    want = CO.compact(cache.float().numpy(), table, page, base, keep)
    strided = torch.zeros(layers, pages + 1, page, width, dtype=dt, device="cuda")[:, :pages]
    strided.copy_(cache)
    V.v4_pages_compact(strided, i32(table), i32(base), i32([len(k) for k in keep]), i32(lists))
    assert np.array_equal(strided.cpu().float().numpy(), want) and V.v4_get_device_status() == 0
