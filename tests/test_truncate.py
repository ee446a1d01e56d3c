"""Cutting sequences back, next to sequences that share their blocks."""

import pytest

from paged_kv_cache_254_gb300 import BlockManager


@pytest.mark.parametrize("cut", ["a", "b"])
def test_stats_count_a_shared_block_as_its_fullest_owner(cut):
    # a cut sequence and its fork hold different counts of tokens in one block
    bm = BlockManager(8, 4)
    bm.add_sequence("a", 8)
    bm.fork("a", "b")
    bm.truncate(cut, 5)
    s = bm.stats()
    assert s["blocks_used"] == 2 and s["tokens"] == 13 and s["internal_waste_slots"] == 0 and s["fragmentation"] == 0.0
    bm.truncate("a" if cut == "b" else "b", 6)
    assert bm.stats()["internal_waste_slots"] == 2


def test_a_cut_fork_grows_into_blocks_of_its_own():
    bm = BlockManager(8, 4)
    bm.add_sequence("a", 8)
    bm.fork("a", "b")
    bm.truncate("b", 5)
    shared = bm.table("a")[1]
    slots = bm.append_slots([("b", 4)]).tolist()
    new = bm.table("b")
    assert bm.take_copies().tolist() == [[shared, new[1]]] and new[1] != shared and bm.table("a")[1] == shared
    assert slots == [new[1] * 4 + 1, new[1] * 4 + 2, new[1] * 4 + 3, new[2] * 4]


def test_a_block_that_a_queued_copy_reads_is_not_given_back():
    # its next owner could be another copy's destination: a batch of copies has no block as both
    bm = BlockManager(8, 4)
    bm.add_sequence("a", 6)
    bm.fork("a", "b")
    bm.append_slots([("b", 1)])                    # queues a copy from a's second block
    with pytest.raises(RuntimeError, match="take_copies"):
        bm.truncate("a", 4)
    assert bm.length("a") == 6 and len(bm.table("a")) == 2
    bm.truncate("a", 5)                            # the block stays
    assert bm.take_copies().tolist() == [[bm.table("a")[1], bm.table("b")[1]]]
    bm.truncate("a", 4)
    bm.add_sequence("c", 8)
    bm.fork("c", "d")
    bm.fork("d", "e")
    bm.append_slots([("b", 1)])
    bm.truncate("e", 0)                            # shared blocks stay with the others: fine at any time
    assert bm.length("e") == 0
