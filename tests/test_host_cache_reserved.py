"""The reference's reserve on hand-worked cases: pages that a fork has shared behind the length."""
import numpy as np

import cache_ref


def pool(table, length, ref):
    k = np.arange(len(ref) * 16 * 2, dtype=np.uint16).reshape(1, len(ref), 1, 16, 2)
    return cache_ref.RefCache(k, k + 1000, np.array(table, np.int32), np.array(length, np.int32),
                              np.array(ref, np.int32))


def test_shared_pages_behind_the_length_are_replaced():
    c = pool([[0, -1, -1], [-1, -1, -1]], [16, 0], [1, 0, 0, 0, 0])
    assert c.reserve([1, 0]) and c.table.tolist() == [[0, 1, -1], [-1, -1, -1]]
    c.fork([0, 0])
    assert c.table.tolist() == [[0, 1, -1], [0, 1, -1]] and c.ref.tolist() == [2, 2, 0, 0, 0]
    k = c.k.copy()
    assert c.reserve([1, 1])  # lane 0 takes page 2, lane 1 keeps page 1, the last holder
    assert c.table.tolist() == [[0, 2, -1], [0, 1, -1]] and c.ref.tolist() == [2, 1, 1, 0, 0]
    assert np.array_equal(c.k, k)  # nothing is committed there: nothing to copy


def test_partly_filled_and_the_pages_behind_it():
    c = pool([[0, 1, 2], [0, 1, 2]], [19, 19], [2, 2, 2, 0, 0, 0, 0])
    assert c.reserve([14, 13])  # lane 0: slots 19..32 in pages 1 (copied to 3) and 2 (replaced by 4); lane 1 keeps its own
    assert c.table.tolist() == [[0, 3, 4], [0, 1, 2]] and c.ref.tolist() == [2, 1, 1, 1, 1, 0, 0]
    assert np.array_equal(c.k[0, 3, 0, :3], c.k[0, 1, 0, :3]) and not np.array_equal(c.k[0, 3, 0, 3], c.k[0, 1, 0, 3])


def test_pages_past_what_is_asked_for_stay_shared_and_all_or_nothing():
    c = pool([[0, 1, 2], [0, 1, 2]], [16, 16], [2, 2, 2, 0])
    assert c.reserve([16, 0]) and c.table.tolist() == [[0, 3, 2], [0, 1, 2]] and c.ref.tolist() == [2, 1, 2, 1]
    assert not c.reserve([17, 17]) and c.table.tolist() == [[0, 3, 2], [0, 1, 2]] and c.ref.tolist() == [2, 1, 2, 1]
