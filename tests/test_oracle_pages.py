"""The page operations of the oracle on hand-worked pools, and the invariant that ref counts
the table entries that name a block."""
import numpy as np

from oracle.sinkkv_oracle import pages_compact, pages_fork, pages_reserve


def counts(table, NB):
    return np.bincount(table[table >= 0].ravel(), minlength=NB)


def test_reserve_takes_the_lowest_free_ids_in_order():
    table = np.full((3, 4), -1)
    ref = np.zeros(8, int)
    ref[[0, 3]] = 1                                      # held by somebody else
    granted, copies = pages_reserve(table, ref, [0, 0, 0], [5, 0, 9], 4, 0, 0, 0)
    assert granted == [1, 1, 1] and copies == []
    assert table.tolist() == [[1, 2, -1, -1], [-1] * 4, [4, 5, 6, -1]]
    assert ref.tolist() == [1, 1, 1, 1, 1, 1, 1, 0]
    # one token more falls into a block that is there; the next request finds one block, then none
    granted, _ = pages_reserve(table, ref, [5, 0, 9], [1, 4, 8], 4, 0, 0, 0)
    assert granted == [1, 1, 0] and table[1].tolist() == [7, -1, -1, -1] and table[2, 3] == -1


def test_reserve_copies_shared_blocks_and_the_last_writer_keeps():
    table = np.array([[2, 5, -1], [2, 5, -1], [2, 5, -1]])
    ref = counts(table, 8)
    granted, copies = pages_reserve(table, ref, [6, 6, 6], [1, 1, 1], 4, 0, 0, 0)
    assert granted == [1, 1, 1] and copies == [(5, 0), (5, 1)]
    assert table[:, 1].tolist() == [0, 1, 5] and ref.tolist() == counts(table, 8).tolist()
    # not all of the holders write: everyone who does takes a copy
    table = np.array([[2, 5, -1], [2, 5, -1], [2, 5, -1]])
    ref = counts(table, 8)
    granted, copies = pages_reserve(table, ref, [6, 6, 6], [1, 0, 1], 4, 0, 0, 0)
    assert copies == [(5, 0), (5, 1)] and table[:, 1].tolist() == [0, 5, 1] and ref[5] == 1


def test_reserve_gives_back_what_the_window_left():
    table = np.array([[0, 1, 2, 3, -1]])
    ref = counts(table, 6)
    # 16 tokens in blocks of 4, window 5, one sink: the query at position 16 sees 12.. and key 0
    granted, _ = pages_reserve(table, ref, [16], [1], 4, 1, 5, 0)
    assert granted == [1] and table.tolist() == [[0, -1, -1, 3, 1]] and ref.tolist() == [1, 1, 0, 1, 0, 0]


def test_fork_reorders_and_releases():
    table = np.array([[0, 1], [2, -1], [3, 4]])
    ref = counts(table, 6)
    lens = np.array([[7, 3, 8], [6, 2, 7]])
    pages_fork(table, ref, lens, [1, 0, -1])
    assert table.tolist() == [[2, -1], [0, 1], [-1, -1]] and lens.tolist() == [[3, 7, 0], [2, 6, 0]]
    assert ref.tolist() == [1, 1, 1, 0, 0, 0]
    pages_fork(table, ref, lens, [0, 1, 1])
    assert table[2].tolist() == [0, 1] and ref.tolist() == [2, 2, 1, 0, 0, 0]


def test_compact():
    table = np.array([[7, 1], [4, -1]])
    ref = counts(table, 8)
    ref[2] = 1                                           # a static sink block, which stays
    block_map, used, moves = pages_compact(table, ref, [2])
    assert moves == [(4, 0), (7, 3)] and used == 4
    assert table.tolist() == [[3, 1], [0, -1]] and ref.tolist() == [1, 1, 1, 1, 0, 0, 0, 0]
    assert block_map.tolist() == [-1, 1, 2, -1, 0, -1, -1, 3]
