"""Reserved pages that a fork has shared: reserve gives every lane pages of its own
under all the slots it asks for, tables, counts and pools as the slot-by-slot
reference has them, and what is appended and attended to afterwards is the lane's."""
import numpy as np
import pytest
import torch

import cache_helpers as ch
import cache_ref
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


def reserve(c, r, want, dev, what=""):
    """On both; what they answer."""
    ok = torch.full((1,), 7, dtype=torch.int32, device=dev)
    c.reserve(ch.ints(want, dev), ok)
    good = r.reserve(want)
    ch.assert_same(c, r, what)
    assert ok.item() == int(good)
    return good


def own(r, want):
    """Whether every page under the slots asked for is one lane's alone."""
    return all(r.ref[r.where(b, n + j)[0]] == 1 for b, (n, w) in enumerate(zip(r.len, want)) for j in range(w))


def append_and_attend(c, r, rows, dev, seed):
    """`rows` drafted slots a lane of drawn keys and values; the attention sees each lane's own."""
    rng = np.random.default_rng(seed)
    lanes, hkv, dim = c.lanes, c.kv_heads, c.head_dim
    hq, n = 2 * hkv, c.lanes * rows
    y = rng.standard_normal((n, hq + 2 * hkv, dim)).astype(np.float32)
    start = list(range(0, n + 1, rows))
    q = abi.rope_append(c, 0, torch.from_numpy(y).to(dev).reshape(n, -1), hq, None, None, row_start=ch.ints(start, dev))
    out, lse = abi.attn_tree(c, 0, q, dim**-0.5, row_start=ch.ints(start, dev), max_nodes=rows, want_lse=True)
    torch.cuda.synchronize()
    bits = cache_ref.bf16_bits(y)
    for i in range(n):
        p, o = r.where(i // rows, int(r.len[i // rows]) + i % rows)
        r.k[0, p, :, o], r.v[0, p, :, o] = bits[i, hq:hq + hkv], bits[i, hq + hkv:]
    ch.assert_same(c, r, "append")
    qh = cache_ref.bf16_value(bits[:, :hq]).astype(np.float64)
    want, wl, wabs, err, seen = cache_ref.attention(r, 0, qh, np.float32(dim**-0.5).astype(np.float64), start, None)
    # the scores' errors, the weights' rounding to bf16 (2^-8), the sums', and the result's rounding
    tol = wabs * (2 * err[:, :, None] + 2.0**-20 + 2.0**-8 + 2 * seen[:, None, None] * 2.0**-24) * 1.01 \
        + np.abs(want) * 2.0**-8 * 1.01
    assert (np.abs(out.float().cpu().numpy() - want) <= tol).all()


@pytest.mark.parametrize("length", [0, 1, 15, 16, 17, 31, 32, 200])
@pytest.mark.parametrize("first,second", [(1, 1), (4, 4), (40, 3), (3, 40), (16, 17)])
def test_reserve_fork_reserve(dev, length, first, second):
    """One lane reserves, two more become its twins, all three reserve, append and attend."""
    c, r = ch.make(dev, length, [length, 3, 0], [0, 0, 0], layers=2, spare=20, width_extra=6)
    assert reserve(c, r, [first, 0, 0], dev)
    for x, t in ((c, lambda a: ch.ints(a, dev)), (r, list)):
        x.fork(t([0, 0, 0]))
    ch.assert_same(c, r, "fork")
    want = [second, second, second]
    assert reserve(c, r, want, dev, "reserve after the fork") and own(r, want)
    append_and_attend(c, r, min(second, 20), dev, length)  # (60 rows: the attention takes 64)
    for x, t in ((c, lambda a: ch.ints(a, dev)), (r, list)):
        x.compact(t(want))
    ch.assert_same(c, r, "commit")


def test_a_lane_that_asks_for_nothing_keeps_its_pages(dev):
    """Twins of which one reserves: the page behind its length is replaced, the other's stays; then the other alone."""
    c, r = ch.make(dev, 2, [16, 5], [30, 0], spare=6)
    for x, t in ((c, lambda a: ch.ints(a, dev)), (r, list)):
        x.fork(t([0, 0]))
    kept = r.table[0].copy()
    assert reserve(c, r, [0, 20], dev)
    assert np.array_equal(r.table[0], kept) and own(r, [0, 20])
    assert reserve(c, r, [20, 0], dev)
    assert np.array_equal(r.table[0], kept) and own(r, [20, 20])


def test_a_page_that_the_caller_keeps_is_replaced(dev):
    """The caller's own reference on a reserved page."""
    c, r = ch.make(dev, 3, [16, 7], [40, 0], spare=6)
    p = int(r.table[0, 2])
    c.ref[p] += 1
    r.ref[p] += 1
    assert reserve(c, r, [16, 1], dev) and r.table[0, 2] == p  # not asked for
    assert reserve(c, r, [17, 1], dev) and r.table[0, 2] != p and r.ref[p] == 1


def test_committed_in_one_lane_reserved_in_the_other(dev):
    """A twin commits into the shared page without appending: half filled for it, behind the length of the other."""
    c, r = ch.make(dev, 4, [16, 2], [8, 0], layers=3, spare=8)
    for x, t in ((c, lambda a: ch.ints(a, dev)), (r, list)):
        x.fork(t([0, 0]))
        x.len[1] += 5  # (as a commit of five slots of the other lane's would have it)
    for want in ([1, 1], [9, 14]):
        assert reserve(c, r, want, dev) and own(r, want)
    c, r = ch.make(dev, 4, [16, 2], [8, 0], layers=3, spare=8)
    for x, t in ((c, lambda a: ch.ints(a, dev)), (r, list)):
        x.fork(t([0, 0]))
        x.len[0] += 5
    for want in ([1, 1], [9, 14]):
        assert reserve(c, r, want, dev) and own(r, want)


def test_too_few_pages_changes_nothing(dev):
    """Twelve reserved pages shared by three lanes and fifteen free ones: two lanes' replacements do not fit, one's do."""
    c, r = ch.make(dev, 5, [16, 0, 0], [192, 0, 0], spare=15)
    for x, t in ((c, lambda a: ch.ints(a, dev)), (r, list)):
        x.fork(t([0, 0, 0]))
    assert not reserve(c, r, [192, 192, 192], dev)
    assert ch.clean_status() == 256
    assert reserve(c, r, [192, 0, 0], dev) and own(r, [192, 0, 0])


def test_replacements_over_a_long_pool(dev):
    """Some 700 shared pages a lane, in a pool whose free pages lie in many steps of the search; own ones between."""
    rng = np.random.default_rng(6)
    pages, lanes, width = 20000, 4, 800
    k = rng.integers(0, 1 << 15, (1, pages, 1, 16, 64)).astype(np.uint16)
    ref = (rng.random(pages) < 0.8).astype(np.int32)
    order = rng.permutation(np.flatnonzero(ref == 0))
    table, length = np.full((lanes, width), -1, np.int32), np.array([33, 33, 0, 40], np.int32)
    table[:2, :700] = order[:700]  # twins
    table[2, :700], table[2, 3:700:5] = order[700:1400], order[3:700:5]  # a third holder of every fifth page
    table[3, :3] = order[1400:1403]
    ref[:] = np.maximum(ref, np.bincount(table[table >= 0], minlength=pages))
    c, r = ch.device_cache(dev, k, k, table, length, ref), cache_ref.RefCache(k, k, table, length, ref)
    for want in ([1, 1, 1, 1], [3000, 3000, 5000, 100], [11500, 11500, 12000, 7]):
        assert reserve(c, r, want, dev) and own(r, want)


@pytest.mark.parametrize("seed", range(8))
def test_any_order_of_the_page_operations(dev, seed):
    """Forks, reserves, trims and commits as they come, reserved pages shared or not; counts add up to the end."""
    rng = np.random.default_rng(seed)
    lanes = int(rng.integers(2, 9))
    c, r = ch.make(dev, seed, [int(x) for x in rng.integers(0, 50, lanes)], [int(x) for x in rng.integers(0, 40, lanes)],
                   layers=2, spare=int(rng.integers(4, 60)), width_extra=12)
    t = lambda a: ch.ints(a, dev)  # noqa: E731
    for i in range(40):
        op = rng.choice(["fork", "reserve", "reserve", "trim", "compact"])
        if op == "fork":
            p = np.where(rng.random(lanes) < 0.1, -1, rng.integers(0, lanes, lanes))
            c.fork(t(p))
            r.fork(p)
        elif op == "reserve":
            want = rng.integers(-2, 40, lanes)
            want = np.minimum(want, r.table.shape[1] * 16 - r.len)
            if reserve(c, r, want, dev, f"{i}: reserve"):
                assert own(r, np.maximum(want, 0))
            else:
                assert ch.clean_status() == 256
        elif op == "trim":
            n = rng.integers(0, 120, lanes)
            c.trim(t(n))
            r.trim(n)
        else:
            room = np.array([(row >= 0).sum() * 16 - n for row, n in zip(r.table, r.len)])
            n = np.minimum(rng.integers(0, 20, lanes), room)
            c.compact(t(n))
            r.compact(n)
        ch.assert_same(c, r, f"{i}: {op}")
        assert r.ref.sum() == (r.table >= 0).sum()


def test_a_captured_reserve_replays(dev):
    """Reserve ahead, fork, reserve in one graph, replayed: what a beam step with room reserved ahead does."""
    n = 4
    c, r = ch.make(dev, 8, [13] * n, [0] * n, layers=2, spare=40, width_extra=8)
    parent, ahead, step = ch.ints(range(n), dev), ch.ints([40] * n, dev), ch.ints([20] * n, dev)
    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream(dev))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        c.reserve(ahead)
        c.fork(parent)
        c.reserve(step)
        c.compact(step)
    rng = np.random.default_rng(1)
    for _ in range(4):
        p = rng.integers(0, n, n)
        parent.copy_(ch.ints(p, dev))
        g.replay()
        assert r.reserve([40] * n)
        r.fork(p)
        assert r.reserve([20] * n) and own(r, [20] * n)
        r.compact([20] * n)
        ch.assert_same(c, r)


@pytest.mark.parametrize("col,entry", [(1, -1), (1, 1 << 24), (2, 1 << 20), (3, 2**31 - 1)])
@pytest.mark.parametrize("shared", [False, True])
def test_a_lane_with_a_bad_page_there_is_left_as_it_was(dev, col, entry, shared):
    """No page under a partly filled last one, or an id outside the pool under the slots asked for: no room, and told
    so; the other lanes get theirs."""
    c, r = ch.make(dev, 9, [10, 20, 17], [0, 40, 0], layers=2, spare=12, width_extra=3)
    t = lambda a: ch.ints(a, dev)  # noqa: E731
    if shared:
        for x, u in ((c, t), (r, list)):
            x.fork(u([0, 1, 0]))
    kept = int(r.table[1, col])
    c.table[1, col] = entry
    ok = torch.full((1,), 7, dtype=torch.int32, device=dev)
    c.reserve(t([30, 40, 30]), ok)
    assert r.reserve([30, 0, 30])
    torch.cuda.synchronize()
    assert ok.item() == 0 and ch.clean_status() == 128
    c.table[1, col] = kept
    ch.assert_same(c, r)
    # not under the slots asked for, it does not matter
    c.table[1, 3] = 1 << 24
    c.reserve(t([0, 5, 0]), ok)
    torch.cuda.synchronize()
    assert ok.item() == 1
