"""Cutting requests down for an eviction in place: the C++ manager against the
oracle on random traces, refusals, tables kept across steps (CPU)."""
import numpy as np
import pytest

from oracle import block_pool as ob
from paged_kv_cache_69_gb300 import block_manager as hbm


def _state(m, o, reqs):
    assert m.free_queue() == o.free_queue()
    for r in reqs:
        assert m.block_table(r) == o.block_table(r)
        assert m.num_tokens(r) == o.reqs[r].num_tokens
    for b in range(m.num_blocks):
        assert m.ref_count(b) == o.ref_cnt(b)


@pytest.mark.parametrize("seed", range(8))
def test_random_traces_equal_the_oracle(seed):
    rng = np.random.default_rng(seed)
    nb, bs = 40, int(rng.choice([4, 8, 16]))
    order = rng.permutation(nb).tolist()
    m, o = hbm.HostBlockManager(nb, bs, order), ob.BlockManager(nb, bs, order)
    buf = hbm.BlockTableBuffer(32, nb)
    live, nxt = [], 0
    for _ in range(300):
        op = rng.choice(["new", "append", "shrink", "fork", "free"], p=[0.2, 0.4, 0.2, 0.1, 0.1])
        if op == "new" and len(live) < 20:
            n = int(rng.integers(0, 5 * bs))
            h = hbm.block_hashes(rng.integers(0, 3, n).tolist(), bs)        # few tokens: prefixes repeat
            if -(-n // bs) > m.num_free():
                continue
            assert m.allocate(nxt, n, h) == o.allocate(nxt, n, h)
            live.append(nxt)
            nxt += 1
        elif op == "append" and live:
            r = int(rng.choice(live))
            a, b = m.append_slot(r), o.append_slot(r)
            assert a == b
        elif op == "shrink" and live:
            r = int(rng.choice(live))
            n = int(rng.integers(0, m.num_tokens(r) + bs))
            try:
                o.shrink(r, n)
            except RuntimeError:
                with pytest.raises(hbm.BlockManagerError):
                    m.shrink(r, n)
            else:
                m.shrink(r, n)
        elif op == "fork" and live and len(live) < 20:
            r = int(rng.choice(live))
            m.fork(r, nxt)
            o.fork(r, nxt)
            live.append(nxt)
            nxt += 1
        elif op == "free" and live:
            r = live.pop(int(rng.integers(len(live))))
            m.free(r)
            o.free(r)
        _state(m, o, live)
        t = buf.update(m, live)
        for k, r in enumerate(live):
            row = m.block_table(r)
            assert t[k, :len(row)].tolist() == row and (t[k, len(row):] == -1).all()


def test_worked_example():
    m = hbm.HostBlockManager(8, 4)
    h = hbm.block_hashes(list(range(16)), 4)
    m.allocate(0, 18, h)                              # blocks 0..4, the first four findable
    m.shrink(0, 18)                                   # no longer than that: unchanged
    assert m.block_table(0) == [0, 1, 2, 3, 4] and m.num_free() == 3
    m.shrink(0, 6)
    assert m.block_table(0) == [0, 1] and m.num_tokens(0) == 6
    # released last first to the head: 2 is handed out next, none carries a hash
    assert m.free_queue() == [(2, False), (3, False), (4, False), (5, False), (6, False), (7, False)]
    assert m.allocate(1, 16, h) == (0, True)          # nothing of the rewritten prefix is found
    slot, pair = m.append_slot(0)
    assert slot == 1 * 4 + 2 and pair is None
    m.shrink(0, 0)
    assert m.block_table(0) == [] and m.num_tokens(0) == 0


def test_refusals():
    m = hbm.HostBlockManager(8, 4)
    m.allocate(0, 10)
    m.fork(0, 1)
    for bad in (lambda: m.shrink(0, 5), lambda: m.shrink(7, 5), lambda: m.shrink(0, -1)):
        with pytest.raises(hbm.BlockManagerError):
            bad()
    assert m.block_table(0) == m.block_table(1) and m.num_tokens(0) == 10
    m.shrink(0, 10)                                   # shared, but nothing to cut
    m.free(1)
    m.set_host_pool(8)
    m.swap_out(0)
    with pytest.raises(hbm.BlockManagerError):
        m.shrink(0, 5)
    m.swap_in(0)
    m.shrink(0, 5)
    assert m.num_tokens(0) == 5 and len(m.block_table(0)) == 2
    m.allocate(2, 4 * m.num_free() + 1)               # waits for a block
    with pytest.raises(hbm.BlockManagerError):
        m.shrink(2, 1)
