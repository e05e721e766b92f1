"""A request that pa_bm_shrink has cut takes no prefix hashes any more: its
blocks hold what an eviction chose, not the tokens of their places (CPU)."""
import pytest

from oracle import block_pool as ob
from paged_kv_cache_69_gb300 import block_manager as hbm

BS = 4


def _pair(nb=16):
    order = list(range(nb))
    return hbm.HostBlockManager(nb, BS, order), ob.BlockManager(nb, BS, order)


def _fill(m, o, req, n):
    for _ in range(n):
        assert m.append_slot(req) == o.append_slot(req)


def _refused(m, o, req, j, h):
    with pytest.raises(hbm.BlockManagerError):
        m.cache_block(req, j, h)
    with pytest.raises(RuntimeError):
        o.cache_block(req, j, h)


def test_a_block_filled_after_the_cut_is_not_findable():
    m, o = _pair()
    tokens = list(range(20))
    h = hbm.block_hashes(tokens, BS)
    for x in (m, o):
        assert x.allocate(0, 18, h) == (0, True)
        x.shrink(0, 6)
    _fill(m, o, 0, 6)                                 # 12 tokens: blocks 1 and 2 are full again
    for j in range(3):
        _refused(m, o, 0, j, h[j])
    for x in (m, o):
        assert x.allocate(1, 16, h) == (0, True)      # nothing of it is found
    assert m.free_queue() == o.free_queue()


def test_forks_and_swaps_keep_the_mark():
    m, o = _pair()
    h = hbm.block_hashes(list(range(8)), BS)
    for x in (m, o):
        x.allocate(0, 12)
        x.shrink(0, 8)
        x.fork(0, 1)
    _refused(m, o, 1, 0, h[0])
    for x in (m, o):
        x.free(0)
        x.set_host_pool(8)
        x.swap_out(1)
        x.swap_in(1)
    _refused(m, o, 1, 1, h[1])


def test_a_cut_that_changes_nothing_marks_nothing():
    m, o = _pair()
    h = hbm.block_hashes(list(range(8)), BS)
    for x in (m, o):
        x.allocate(0, 8)
        x.shrink(0, 8)
        x.cache_block(0, 1, h[1])
        x.cache_block(0, 0, h[0])
        assert x.allocate(1, 8, h) == (8, True)
        x.free(0)                                     # the same id, used again, starts afresh
        x.free(1)
        x.allocate(0, 9)
        x.shrink(0, 4)
        x.free(0)
        x.allocate(0, 4)
        x.cache_block(0, 0, hbm.block_hashes([5, 6, 7, 8], BS)[0])
