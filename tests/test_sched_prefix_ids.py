"""CPU: prefix caching and request ids that are used again: what a request that has left computed is nobody's prefix."""
from continuous_batching_paged_ragged_gb300.pkv import Scheduler


def _preempted(s, keep, gone):
    """Two requests of 16 tokens on 4 blocks of 8: the second is preempted; of its two full blocks, registered as its prefix, the
    first request takes the later one for its 17th token."""
    s.add(keep, 16, 9)
    s.add(gone, 16, 9)
    s.step()
    assert s.step()["preempted"] == [gone]


def test_an_id_used_again_after_an_abort_finds_nothing(built):
    s = Scheduler(4, 100, 8, 4, prefix_caching=True)
    _preempted(s, 1, 2)
    s.abort(2)
    s.abort(1)
    s.add(2, 16, 3)  # another prompt under the old id
    b = s.step()
    assert b["req_ids"].tolist() == [2] and b["q_lens"].tolist() == [16] and b["context_lens"].tolist() == [16]
    assert s.stats()["prefix_hit_tokens"] == 0


def test_a_child_under_an_old_id_finds_nothing(built):
    """A fork's child named as a request that was aborted while preempted: preempted in its turn, it computes its own prefix again."""
    s = Scheduler(4, 100, 8, 6, prefix_caching=True)
    s.add(1, 24, 20)
    s.add(2, 24, 9)
    s.step()
    assert s.step()["preempted"] == [2]  # three full blocks of 2 stay registered, two of them free
    s.abort(2)
    child = 2
    assert s.fork(1, child, 20) >= 0
    hits = s.stats()["prefix_hit_tokens"]
    preempted = False
    for _ in range(60):
        b = s.step()
        preempted |= child in b["preempted"]
        if child in b["admitted"]:
            i = b["req_ids"].tolist().index(child)
            assert b["context_lens"][i] == b["q_lens"][i], "the child took blocks that another request computed"
        if s.done():
            break
    assert preempted and s.done() and s.stats()["prefix_hit_tokens"] == hits


def test_a_preempted_request_still_takes_its_own_blocks_back(built):
    s = Scheduler(4, 100, 8, 4, prefix_caching=True)
    _preempted(s, 1, 2)
    s.abort(1)
    b = s.step()
    assert b["req_ids"].tolist() == [2] and b["context_lens"].tolist() == [17] and b["q_lens"].tolist() == [17 - 8]
    assert s.stats()["prefix_hit_tokens"] == 8


def test_the_oracle_agrees(built):
    import oracle
    native = Scheduler(4, 100, 8, 4, prefix_caching=True)
    plain = oracle.scheduler.Scheduler(4, 100, 8, list(range(4)), prefix_caching=True)
    for s in (native, plain):
        s.add(1, 16, 9)
        s.add(2, 16, 9)
    for gone in (None, 2, 1):
        if gone:
            native.abort(gone)
            plain.abort(gone)
        else:
            native.step(), plain.step(), native.step(), plain.step()
    for s in (native, plain):
        s.add(2, 16, 3)
    while not native.done():
        a, b = native.step(), plain.step()
        assert a["slot_mapping"].tolist() == b.slot_mapping.tolist() and a["q_lens"].tolist() == b.q_lens.tolist()
    assert plain.done()
