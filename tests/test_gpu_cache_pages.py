"""GPU parity of the cache's page operations with the slot-by-slot reference:
tables, lengths, reference counts and every bf16 pattern of the pools, exactly."""
import numpy as np
import pytest
import torch

import cache_helpers as ch
from nvfp4_weight_streaming_decode_b200 import abi

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev(cuda_device):
    abi.load()
    torch.cuda.set_device(cuda_device)
    return cuda_device


@pytest.fixture(autouse=True)
def status(dev):
    ch.clean_status()
    yield
    assert ch.clean_status() == 0


LENS = [[0], [1], [16], [33, 0, 7], [100, 100, 100, 100], [5] * 8, list(range(0, 640, 10))]


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("page,dim", [(16, 64), (64, 128), (256, 256)])
def test_fork_then_reserve(dev, lens, page, dim):
    n = len(lens)
    for seed in range(3):
        c, r = ch.make(dev, seed, lens, [0] * n, layers=2, page=page, dim=dim, spare=2 * n + 2)
        rng = np.random.default_rng(seed + 100)
        parent = rng.integers(-1 if seed == 1 else 0, n, n)
        want = rng.integers(0, 2 * page, n) if seed else np.ones(n, int)
        c.fork(ch.ints(parent, dev))
        r.fork(parent)
        ch.assert_same(c, r, "fork")
        ok = torch.full((1,), 7, dtype=torch.int32, device=dev)
        while not r.reserve(want):  # too few pages: nothing changes, told by ok and the status
            c.reserve(ch.ints(want, dev), ok)
            ch.assert_same(c, r, "refused reserve")
            assert ok.item() == 0 and ch.clean_status() == 256
            want = want // 2
        c.reserve(ch.ints(want, dev), ok)
        ch.assert_same(c, r, "reserve")
        assert ok.item() == 1


def test_beam_steps_keep_every_lane(dev):
    """Twelve steps of fork, reserve and commit: shared pages, copies and releases in turn."""
    lens, n = [20] * 6, 6
    c, r = ch.make(dev, 5, lens, [0] * n, layers=3, spare=90, width_extra=16)
    rng = np.random.default_rng(9)
    for _ in range(12):
        parent = rng.integers(0, n, n)
        step = rng.integers(1, 20, n)
        for x in (c, r):
            t = (lambda a: ch.ints(a, dev)) if x is c else (lambda a: a)
            x.fork(t(parent))
            x.reserve(t(step))
            x.compact(t(step))
        ch.assert_same(c, r)
    assert (r.ref >= 0).all() and r.ref.sum() == (r.table >= 0).sum()
    c.fork(ch.ints([-1] * n, dev))
    r.fork([-1] * n)
    ch.assert_same(c, r, "all freed")
    assert not r.ref.any()


def test_reserve_takes_no_page_it_need_not(dev):
    """Reserving twice adds nothing; want <= 0 touches nothing; a page kept by the caller's own reference is copied."""
    c, r = ch.make(dev, 1, [17, 40, 0], [0, 0, 0], spare=6)
    for want in ([5, -3, 0], [5, -3, 0], [16, 8, 16]):
        c.reserve(ch.ints(want, dev))
        assert r.reserve(want)
        ch.assert_same(c, r)
    p = int(r.table[0, 1])
    c.ref[p] += 1
    r.ref[p] += 1
    c.reserve(ch.ints([1, 0, 0], dev))
    assert r.reserve([1, 0, 0])
    assert r.table[0, 1] != p
    ch.assert_same(c, r)


def test_reserve_over_a_long_pool(dev):
    """Free pages thin out over 20,000 ids (several steps of the search)."""
    rng = np.random.default_rng(3)
    pages, lanes, width = 20000, 5, 40
    k = rng.integers(0, 1 << 15, (1, pages, 1, 16, 64)).astype(np.uint16)
    ref = (rng.random(pages) < 0.999).astype(np.int32)
    table, length = np.full((lanes, width), -1, np.int32), np.zeros(lanes, np.int32)
    from cache_ref import RefCache
    c, r = ch.device_cache(dev, k, k, table, length, ref), RefCache(k, k, table, length, ref)
    free = int((ref == 0).sum())
    want = [16, 0, 33, 48, 16 * max(0, free - 1 - 3 - 3)] if free >= 8 else [1, 0, 0, 0, 0]
    want[4] = min(want[4], 16 * width)
    assert r.reserve(want)
    c.reserve(ch.ints(want, dev))
    ch.assert_same(c, r)


def test_reserve_past_the_table_is_refused(dev):
    c, r = ch.make(dev, 1, [10, 3], [0, 0], spare=60, width_extra=1)
    ok = torch.ones(1, dtype=torch.int32, device=dev)
    c.reserve(ch.ints([2**31 - 1, 1], dev), ok)
    ch.assert_same(c, r)
    assert ok.item() == 0 and ch.clean_status() == 256


@pytest.mark.parametrize("page,dim,hkv,layers", [(16, 64, 1, 1), (16, 128, 3, 5), (64, 256, 2, 2), (128, 128, 8, 1)])
def test_compact_moves_the_accepted_path(dev, page, dim, hkv, layers):
    lens, nodes = [0, 15, 16, 130, 63], 64
    c, r = ch.make(dev, 2, lens, [nodes] * 5, layers=layers, hkv=hkv, page=page, dim=dim)
    rng = np.random.default_rng(4)
    count = np.array([64, 1, 0, 20, 37], np.int32)
    path = np.zeros((5, nodes), np.int32)
    for b, n in enumerate(count):
        path[b, :n] = np.sort(rng.choice(nodes, n, replace=False))
    path[1, 0] = 63
    c.compact(ch.ints(count, dev), ch.ints(path, dev))
    r.compact(count, path)
    ch.assert_same(c, r)


def test_compact_without_a_path_commits_and_releases(dev):
    c, r = ch.make(dev, 2, [10, 0, 31, 5], [100, 90, 0, 64])
    c.compact(ch.ints([3, 16, 1, 0], dev))
    r.compact([3, 16, 1, 0])
    ch.assert_same(c, r)


def test_compact_leaves_a_lane_it_refuses(dev):
    """Counts, paths, pages that cannot be committed: those lanes stay as they were, the others go on."""
    lens = [10, 10, 10, 10, 10, 10, 10]
    c, r = ch.make(dev, 7, lens, [20] * 7, layers=2)
    shared = int(r.table[4, 0])
    c.ref[shared] += 1
    r.ref[shared] += 1
    bad = [(2, [3, 3]), (2, [4, 1]), (-1, [0, 1]), (3, [0, 1]), (2, [1, 2]), (2, [0, 64])]  # lanes 0..5; 3 > ld 2
    count = [n for n, _ in bad] + [2]
    path = [p for _, p in bad] + [[1, 5]]
    c.compact(ch.ints(count, dev), ch.ints(path, dev))
    r.compact([0] * 6 + [2], [[0, 0]] * 6 + [[1, 5]])
    for b in range(6):  # the reference releases reserved pages of lanes that commit nothing; a refused lane keeps them
        r.table[b] = c.table[b].cpu().numpy()
    torch.cuda.synchronize()
    assert np.array_equal(c.len.cpu().numpy(), r.len)
    assert np.array_equal(ch.host_bits(c.k), r.k) and np.array_equal(ch.host_bits(c.v), r.v)
    assert (c.table[:6].cpu().numpy() >= 0).sum() == 6 * 2 and (c.table[6].cpu().numpy() >= 0).sum() == 1
    assert ch.clean_status() == 128


def test_trim(dev):
    c, r = ch.make(dev, 3, [100, 0, 33, 16, 50], [40, 20, 0, 0, 900])
    new = [55, 3, -4, 16, 2**31 - 1]
    c.trim(ch.ints(new, dev))
    r.trim(new)
    ch.assert_same(c, r)


def test_bad_parent_empties_the_lane(dev):
    c, r = ch.make(dev, 3, [100, 20, 33], [0, 0, 0])
    c.fork(ch.ints([0, 3, -2], dev))
    r.fork([0, -1, -1])
    ch.assert_same(c, r)
    assert ch.clean_status() == 128


def test_a_captured_step_replays(dev):
    """Fork, reserve and commit in one graph: each replay reads what the tensors then hold."""
    n = 4
    c, r = ch.make(dev, 8, [13] * n, [0] * n, layers=2, spare=30)
    parent, step = ch.ints(range(n), dev), ch.ints([1] * n, dev)
    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream(dev))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        c.fork(parent)
        c.reserve(step)
        c.compact(step)
    rng = np.random.default_rng(1)
    for _ in range(6):
        p = rng.integers(0, n, n)
        parent.copy_(ch.ints(p, dev))
        g.replay()
        r.fork(p)
        assert r.reserve([1] * n)
        r.compact([1] * n)
        ch.assert_same(c, r)
