"""Groups of samples in the continuous batcher: forked sequences share their
prompt's pages, wait when nothing fits, and give every page back (host only)."""
import numpy as np
import pytest
import torch

pkv = pytest.importorskip("paged_kv_decode_pagetable_gb300")
from paged_kv_decode_pagetable_gb300 import engine  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def lib():
    pkv.load_library()


def test_group_shares_the_prompt_and_waits_for_slots():
    """Prompt of 9 tokens in pages of 4 (3 pages with the first new token). Two of
    three more samples find a slot: each takes one page of its own for the half-filled
    third page; the last one waits and is admitted when a sample finishes."""
    pt = pkv.PageTable(3, 4, 20, 8)
    cb = engine.ContinuousBatcher(pt, [engine.Sequence(0, 9, 4)])
    assert cb.step()                                  # prefill: 1 token generated
    s = cb.running[0]
    new = cb.fork(s, [1, 2, 3], caches=[])
    assert [f.slot for f in new] == [2, 3, -1] and [f.generated for f in new] == [1, 1, 1]
    assert pt.pages(2)[:2] == pt.pages(s.slot)[:2]
    assert [pt.page_refs(p) for p in pt.pages(s.slot)] == [3, 3, 1]
    assert len({pt.pages(x)[2] for x in (1, 2, 3)}) == 3
    done = cb.run()
    assert sorted(f.rid for f in done) == [0, 1, 2, 3]
    assert all(f.generated == 4 for f in done)
    assert len(pt.free_page_list()) == 19
    assert [e for e in cb.events if e[0] == "fork"] == [("fork", 0, 1), ("fork", 0, 2)]
    with pytest.raises(ValueError):
        cb.fork(s, [4], caches=[])


def test_groups_under_pressure_keep_their_invariants():
    """Random prompts, each forked after its prefill, in a pool that has to preempt:
    no running sequence appends into a shared page, and all pages come back."""
    rng = np.random.default_rng(3)
    ps, n_pages = 8, 1 + 60
    pt = pkv.PageTable(12, ps, n_pages, 20)
    seqs = [engine.Sequence(i, int(rng.integers(3, 70)), int(rng.integers(2, 40)))
            for i in range(10)]
    state = {"next": 100}

    def prefill(batch):
        state["fork"] = [s for s in batch if s.rid < 100 and s.generated == 0]

    def decode(batch):
        for s in batch:
            at = s.total_length - 1
            assert pt.page_refs(pt.pages(s.slot)[at // ps]) == 1, (s.rid, at)
        assert len({s.slot for s in batch}) == len(batch)

    cb = engine.ContinuousBatcher(pt, seqs, prefill=prefill, decode=decode)
    expected = 10
    for _ in range(10000):
        if not cb.step():
            break
        for s in state.pop("fork", []):
            if s in cb.running:
                n = int(rng.integers(1, 5))
                cb.fork(s, range(state["next"], state["next"] + n), caches=[])
                state["next"] += n
                expected += n
    assert len(cb.done) == expected > 20 and all(s.generated == s.max_new_tokens for s in cb.done)
    assert {e[0] for e in cb.events} >= {"fork", "preempt", "finish"}
    assert len(pt.free_page_list()) == n_pages - 1
    assert all(pt.page_refs(p) == 0 for p in range(n_pages))


def test_compact_cache_counts_moves():
    pt = pkv.PageTable(4, 4, 20, 8)
    a, b = pt.assign(20), pt.assign(12)
    pt.free(a)
    assert engine.compact_cache(pt, []) == len([p for p in range(6, 9)])
    assert sorted(pt.pages(b)) == [1, 2, 3]
    assert engine.compact_cache(pt, []) == 0


def test_refused_caches_change_nothing():
    """Caches that cannot be copied are refused before pages change hands."""
    pt = pkv.PageTable(3, 4, 20, 8)
    cb = engine.ContinuousBatcher(pt, [engine.Sequence(0, 9, 4)])
    assert cb.step()
    s = cb.running[0]
    bad = torch.zeros((2, 19 * 4, 8))                 # 76 rows are not 20 pages
    for caches in ([bad], [torch.zeros((2, 80, 8))]):   # ... and not on a CUDA device
        with pytest.raises(pkv.BadArgError):
            cb.fork(s, [1, 2], caches)
        assert list(cb.running) == [s] and not cb.waiting
        assert [pt.page_refs(p) for p in pt.pages(s.slot)] == [1, 1, 1]
    a = pt.assign(20)
    b = pt.assign(8)
    pt.free(a)
    before = pt.pages(b)
    with pytest.raises(pkv.BadArgError):
        engine.compact_cache(pt, [bad])
    assert pt.pages(b) == before
