"""CPU: forks, block listings and remaps of the host scheduler -- by hand, and as invariants over random workloads (every block
is free or held, shared only between a parent's and its children's common full blocks, and none is lost)."""
import random

import numpy as np
import pytest

from continuous_batching_paged_ragged_gb300 import pkv
from continuous_batching_paged_ragged_gb300.pkv import PkvError, Scheduler


def _refused(status, fn, *args):
    with pytest.raises(PkvError) as e:
        fn(*args)
    assert e.value.status == status


def test_fork_by_hand(built):
    s = Scheduler(4, 100, 16, 10)
    s.add(7, 40, 5)
    s.step()  # 40 computed tokens: blocks 0, 1, 2; one output
    assert s.fork(7, 8, 5) == 3  # 8 tokens past the second full block
    ids, tables = s.tables()
    assert ids.tolist() == [7, 8] and tables.tolist() == [[0, 1, 2], [0, 1, 3]]
    b = s.step()
    assert b["req_ids"].tolist() == [7, 8] and b["q_lens"].tolist() == [1, 1] and b["context_lens"].tolist() == [41, 41]
    assert b["slot_mapping"].tolist() == [2 * 16 + 8, 3 * 16 + 8]  # each into its own block
    s.abort(7)
    assert s.free_list() == [4, 5, 6, 7, 8, 9, 2]  # the shared blocks stay the child's
    while not s.done():
        s.step()
    assert sorted(s.free_list()) == list(range(10))


def test_fork_on_a_block_boundary_needs_no_block(built):
    s = Scheduler(4, 100, 16, 3)
    s.add(1, 32, 3)
    s.step()
    assert s.fork(1, 2, 2) == -1
    assert s.tables()[1].tolist() == [[0, 1], [0, 1]]
    b = s.step()  # both need a block for their next token, one is free: the child is preempted
    assert b["req_ids"].tolist() == [1] and b["preempted"] == [2]
    assert s.tables()[1].tolist() == [[0, 1, 2]]


def test_remap_by_hand(built):
    s = Scheduler(4, 100, 16, 8, free_order=[7, 3, 5, 0, 1, 2, 4, 6])
    s.add(1, 20, 9)
    s.add(2, 10, 9)
    s.step()
    assert s.tables()[1].tolist() == [[7, 3], [5, -1]]
    remap = [-1] * 8
    remap[7], remap[3], remap[5] = 0, 1, 2
    s.remap(remap)
    assert s.tables()[1].tolist() == [[0, 1], [2, -1]] and s.free_list() == [3, 4, 5, 6, 7]
    for bad in ([-1] * 8, [0] * 8, [0, 1, 9, 3, 4, 5, 6, 7]):
        _refused(pkv.PKV_ERR_INVALID_ARG, s.remap, bad)
    assert s.tables()[1].tolist() == [[0, 1], [2, -1]] and s.free_list() == [3, 4, 5, 6, 7]


def test_refusals(built):
    s = Scheduler(2, 100, 16, 3)
    s.add(1, 20, 4)
    s.add(5, 20, 4)
    _refused(pkv.PKV_ERR_NOT_FOUND, s.fork, 9, 2, 4)
    _refused(pkv.PKV_ERR_INVALID_ARG, s.fork, 1, 2, 4)  # waiting
    s.step()  # request 1 runs, 5 does not fit beside it
    _refused(pkv.PKV_ERR_INVALID_ARG, s.fork, 1, 5, 4)  # the id is taken
    _refused(pkv.PKV_ERR_INVALID_ARG, s.fork, 1, 2, 1)  # the parent has one output already
    _refused(pkv.PKV_ERR_NO_BLOCKS, s.fork, 1, 2, 30)
    before = (s.tables()[1].tolist(), s.free_list())
    assert s.fork(1, 2, 4) == 2
    _refused(pkv.PKV_ERR_OUT_OF_RANGE, s.fork, 1, 3, 4)  # two run
    s.set_max_num_seqs(3)
    _refused(pkv.PKV_ERR_NO_BLOCKS, s.fork, 1, 3, 4)  # no block left
    s.abort(2)
    assert (s.tables()[1].tolist(), s.free_list()) == before
    r = Scheduler(2, 100, 16, 8, alloc=pkv.PKV_ALLOC_RESERVE)
    r.add(1, 20, 4, 4)
    r.step()
    _refused(pkv.PKV_ERR_UNSUPPORTED, r.fork, 1, 2, 4)
    assert r.tables()[1].shape == (1, 2)
    n = None
    assert built.pkv_sched_fork(n, 1, 2, 3, n) == pkv.PKV_ERR_INVALID_ARG
    assert built.pkv_sched_remap(n, n) == pkv.PKV_ERR_INVALID_ARG and built.pkv_sched_tables(n, 0, 0, n, n, n) == 0
    empty = Scheduler(2, 100, 16, 8)
    ids, tables = empty.tables()
    assert ids.size == 0 and tables.shape == (0, 1)


@pytest.mark.parametrize("seed", range(8))
def test_random_workloads_keep_every_block(built, seed):
    rng = random.Random(seed)
    bs, blocks = rng.choice([4, 16]), rng.randint(12, 60)
    order = list(range(blocks))
    rng.shuffle(order)
    s = Scheduler(rng.randint(2, 12), rng.randint(8, 64), bs, blocks, order, prefix_caching=bool(seed & 1))
    content = {}  # (block, row) -> (lineage, position): what a cache would hold
    lineage, next_id, forks = {}, 0, 0

    def held():
        ids, tables = s.tables()
        return {int(i): [int(b) for b in row if b >= 0] for i, row in zip(ids, tables)}

    for _ in range(250):
        if rng.random() < 0.3:
            prompt, out = rng.randint(1, 3 * bs), rng.randint(1, 3 * bs)
            if (prompt + out + bs - 1) // bs <= blocks:
                s.add(next_id, prompt, out)
                lineage[next_id] = {}
                next_id += 1
        step = s.step()
        for b, rid in enumerate(step["req_ids"].tolist()):
            q0, q1 = step["query_start_loc"][b], step["query_start_loc"][b + 1]
            ctx = int(step["context_lens"][b])
            for i, t in enumerate(range(q0, q1)):
                p = ctx - (q1 - q0) + i
                lineage[rid].setdefault(p, (rid, p))
                content[int(step["slot_mapping"][t])] = lineage[rid][p]
            for p in range(ctx):  # every token of the row is where its table says, written by it or by an ancestor
                slot = int(step["block_tables"][b, p // bs]) * bs + p % bs
                assert content[slot] == lineage[rid][p], (rid, p)
        h = held()
        running = list(h)
        if running and rng.random() < 0.4:
            parent = rng.choice(running)
            before = {k: list(v) for k, v in h.items()}
            try:
                block = s.fork(parent, next_id, rng.randint(1, 4 * bs))
            except PkvError:
                assert held() == before
            else:
                forks += 1
                h = held()
                mine = h[next_id]
                lineage[next_id] = dict(lineage[parent])
                if block >= 0:
                    assert mine[-1] == block and mine[:-1] == before[parent][:len(mine) - 1]
                    src = before[parent][len(mine) - 1]
                    for r in range(bs):
                        if src * bs + r in content:
                            content[block * bs + r] = content[src * bs + r]
                else:
                    assert mine == before[parent][:len(mine)]
                next_id += 1
        if running and rng.random() < 0.1:
            s.abort(rng.choice(running))
        if rng.random() < 0.15:  # a compaction, as pkv_compact defines it
            h = held()
            used = sorted({b for v in h.values() for b in v})
            n = len(used)
            remap = [-1] * blocks
            for b in used:
                remap[b] = b
            for src, dst in zip([b for b in used if b >= n], [b for b in range(n) if remap[b] < 0]):
                remap[src] = dst
                for r in range(bs):
                    content.pop(dst * bs + r, None)
                    if src * bs + r in content:
                        content[dst * bs + r] = content[src * bs + r]
            s.remap(remap)
            assert s.free_list() == list(range(n, blocks))
        h, free = held(), s.free_list()
        used = {b for v in h.values() for b in v}
        assert len(set(free)) == len(free) and not used & set(free) and len(used) + len(free) == blocks
        assert all(len(set(v)) == len(v) for v in h.values())
    assert forks > 5
    while not s.done():
        s.step()
    assert sorted(s.free_list()) == list(range(blocks)) and held() == {}
