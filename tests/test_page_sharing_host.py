"""Sharing, taking back and moving pages (pt_fork, pt_unshare, pt_truncate,
pt_compact) through the C ABI, host only: a worked example, a model of the
policy that keeps token contents, and every refusal leaving the state as it was."""
import ctypes

import numpy as np
import pytest
import torch

pkv = pytest.importorskip("paged_kv_decode_pagetable_gb300")


@pytest.fixture(scope="module", autouse=True)
def lib():
    pkv.load_library()


def state(pt):
    return (pt.host_table().tolist(), pt.free_page_list(),
            [pt.capacity(s) for s in range(pt.n_slots)], [pt.pages(s) for s in range(pt.n_slots)],
            [pt.page_refs(p) for p in range(pt.n_pages)])


def test_fork_truncate_free_worked_example():
    """5 slots, pages of 4 tokens, 9 usable pages [9..1]. Slot 1 takes the tail
    [3, 2, 1] for 11 tokens; two forks at 10 tokens share pages 3, 2 and get the
    next pages 4, 5 for the half-filled third."""
    pt = pkv.PageTable(5, 4, 10, 4)
    assert pt.assign(11) == 1 and pt.pages(1) == [3, 2, 1]
    slots, pairs = pt.fork(1, 10, 2)
    assert slots == [2, 3] and pairs.tolist() == [[1, 4], [1, 5]]
    assert pt.pages(2) == [3, 2, 4] and pt.pages(3) == [3, 2, 5]
    assert [pt.page_refs(p) for p in range(10)] == [0, 1, 3, 3, 1, 1, 0, 0, 0, 0]
    assert pt.capacity(2) == 12 and pt.host_table()[3].tolist() == [3, 2, 5, -1]
    # a fork at a page boundary copies nothing
    slots, pairs = pt.fork(2, 8)
    assert slots == [4] and pairs.shape == (0, 2) and pt.pages(4) == [3, 2]
    # taking back two pages of slot 3 frees only its own
    pt.truncate(3, 3)
    assert pt.pages(3) == [3] and pt.host_table()[3].tolist() == [3, -1, -1, -1]
    assert pt.free_page_list() == [9, 8, 7, 6, 5]
    # the source may go first; shared pages stay
    pt.free(1)
    assert pt.free_page_list() == [9, 8, 7, 6, 5, 1] and pt.page_refs(3) == 3
    # rewriting token 4 of slot 4 (page 2, shared with slot 2)
    assert pt.unshare(4, 4, 5).tolist() == [[2, 1]]
    assert pt.pages(4) == [3, 1] and pt.pages(2) == [3, 2, 4] and pt.page_refs(2) == 1
    assert pt.unshare(4, 4, 8).shape == (0, 2) and pt.unshare(4, 3, 3).shape == (0, 2)
    # pages in use: 1, 2, 3, 4 - already in front
    assert pt.compact().shape == (0, 2) and pt.free_page_list() == [9, 8, 7, 6, 5]
    pt.free(4)                                   # page 1 free: page 4 moves there
    assert pt.compact().tolist() == [[4, 1]]
    assert pt.pages(2) == [3, 2, 1] and pt.host_table()[2].tolist() == [3, 2, 1, -1]
    assert pt.free_page_list() == [9, 8, 7, 6, 5, 4]


class Model:
    """Slots as lists of tokens, and the bytes of the pages beside them."""

    def __init__(self, pt):
        self.pt, self.ps = pt, pt.page_size
        self.tokens = {}                                # slot -> list of token ids
        self.data = np.zeros((pt.n_pages, pt.page_size), np.int64)
        self.next = 1

    def copy(self, pairs):
        new = {int(b): self.data[a].copy() for a, b in pairs.tolist()}
        for b, v in new.items():
            self.data[b] = v

    def append(self, slot, n):
        for _ in range(n):
            t = len(self.tokens[slot])
            page = self.pt.pages(slot)[t // self.ps]
            assert self.pt.page_refs(page) == 1         # never into a shared page
            self.data[page, t % self.ps] = self.next
            self.tokens[slot].append(self.next)
            self.next += 1

    def check(self):
        pt = self.pt
        held = np.zeros(pt.n_pages, np.int64)
        table = pt.host_table().numpy()
        for slot, toks in self.tokens.items():
            pages = pt.pages(slot)
            assert pt.capacity(slot) == len(pages) * self.ps >= len(toks)
            assert table[slot, :len(pages)].tolist() == pages
            assert (table[slot, len(pages):] == -1).all()
            held[pages] += 1
            got = self.data[pages].reshape(-1)[:len(toks)] if pages else np.zeros(0)
            assert got.tolist() == toks, slot
        assert held.tolist() == [pt.page_refs(p) for p in range(pt.n_pages)]
        free = pt.free_page_list()
        assert len(set(free)) == len(free) and 0 not in free
        assert set(free) == {p for p in range(1, pt.n_pages) if held[p] == 0}


@pytest.mark.parametrize("seed,ps", [(0, 4), (1, 1), (2, 8)])
def test_random_operations_keep_every_sequence(seed, ps):
    rng = np.random.default_rng(seed)
    pt = pkv.PageTable(9, ps, 60, 12)
    m = Model(pt)
    done = {k: 0 for k in ("assign", "grow", "fork", "truncate", "free", "compact", "rewrite")}
    for _ in range(1500):
        live = sorted(m.tokens)
        op = rng.choice(list(done))
        try:
            if op == "assign":
                n = int(rng.integers(0, 5 * ps))
                slot = pt.assign(n)
                m.tokens[slot] = []
                m.append(slot, n)
            elif not live:
                continue
            else:
                slot = int(rng.choice(live))
                n = len(m.tokens[slot])
                if op == "grow":
                    k = int(rng.integers(1, 2 * ps + 1))
                    m.copy(pt.unshare(slot, n, pt.capacity(slot)))
                    pt.reserve(slot, n + k)
                    m.append(slot, k)
                elif op == "fork":
                    at, count = int(rng.integers(0, n + 1)), int(rng.integers(1, 4))
                    slots, pairs = pt.fork(slot, at, count)
                    assert len(pairs) == (count if at % ps else 0)
                    m.copy(pairs)
                    for s in slots:
                        m.tokens[s] = m.tokens[slot][:at]
                elif op == "truncate":
                    at = int(rng.integers(0, n + 1))
                    pt.truncate(slot, at)
                    m.tokens[slot] = m.tokens[slot][:at]
                elif op == "rewrite" and n:
                    at = int(rng.integers(0, n))
                    m.copy(pt.unshare(slot, at, n))
                    m.tokens[slot] = m.tokens[slot][:at]
                    m.append(slot, n - at)
                elif op == "free":
                    pt.free(slot)
                    del m.tokens[slot]
                elif op == "compact":
                    m.copy(pt.compact())
                    used = pt.n_pages - 1 - len(pt.free_page_list())
                    assert pt.free_page_list() == list(range(pt.n_pages - 1, used, -1))
            done[op] += 1
        except (pkv.NoPagesError, pkv.NoSlotError, pkv.BadArgError):
            pass
        m.check()
    assert min(done.values()) > 20, done


def test_refusals_leave_the_state():
    pt = pkv.PageTable(3, 4, 8, 4)
    a = pt.assign(10)                            # three of seven pages
    before = state(pt)
    for call, err in ((lambda: pt.fork(0, 0), pkv.BadSlotError),
                      (lambda: pt.fork(2, 0), pkv.BadSlotError),
                      (lambda: pt.fork(9, 0), pkv.BadSlotError),
                      (lambda: pt.fork(a, 13), pkv.BadArgError),
                      (lambda: pt.fork(a, -1), pkv.BadArgError),
                      (lambda: pt.fork(a, 4, 0), pkv.BadArgError),
                      (lambda: pt.fork(a, 4, -2), pkv.BadArgError),
                      (lambda: pt.fork(a, 4, 3), pkv.NoSlotError),
                      (lambda: pt.truncate(0, 0), pkv.BadSlotError),
                      (lambda: pt.truncate(a, 13), pkv.BadArgError),
                      (lambda: pt.truncate(a, -1), pkv.BadArgError),
                      (lambda: pt.unshare(a, 2, 1), pkv.BadArgError),
                      (lambda: pt.unshare(a, 0, 13), pkv.BadArgError),
                      (lambda: pt.unshare(3, 0, 0), pkv.BadSlotError),
                      (lambda: pt.page_refs(8), pkv.BadArgError),
                      (lambda: pt.page_refs(-1), pkv.BadArgError)):
        with pytest.raises(err):
            call()
        assert state(pt) == before
    slots, _ = pt.fork(a, 10, 2)                 # two more pages; two free
    pt.reserve(slots[0], 16)
    pt.reserve(slots[1], 16)
    before = state(pt)
    with pytest.raises(pkv.NoPagesError):        # two shared pages, none free
        pt.unshare(a, 0, 8)
    pt.truncate(slots[1], 12)
    before = state(pt)
    with pytest.raises(pkv.NoPagesError):
        pt.unshare(a, 0, 8)
    assert state(pt) == before
    pt.free(slots[1])
    pt.truncate(slots[0], 12)                    # three pages free, one slot
    assert pt.assign(12) == slots[1]
    pt.free(slots[0])
    assert len(pt.free_page_list()) == 1
    c = pt.fork(a, 9)[0][0]
    assert pt.free_page_list() == []
    pt.free(c)
    pt.reserve(a, 16)
    before = state(pt)
    with pytest.raises(pkv.NoPagesError):
        pt.fork(a, 9)
    assert state(pt) == before


def test_copy_refusals_need_no_gpu():
    """Pairs and shapes are refused on the host, before any launch."""
    cache = torch.zeros((2, 6 * 4, 8), dtype=torch.bfloat16)     # never reached
    with pytest.raises(pkv.BadArgError):
        pkv.kv_copy_pages([cache], 5, [(1, 2)])                  # 24 rows are not 5 pages
    with pytest.raises(pkv.BadArgError):
        pkv.kv_copy_pages([cache.transpose(0, 1)], 6, [(1, 2)])
    with pytest.raises(pkv.BadArgError):
        pkv.kv_copy_pages([cache], 6, torch.zeros((1, 2), dtype=torch.int64))
    with pytest.raises(pkv.BadArgError):
        pkv.kv_copy_pages([cache], 0, [(0, 0)])
    with pytest.raises(pkv.BadArgError):
        pkv.kv_copy_pages([cache], 6, [(1, 2)])                  # not on a CUDA device
    pkv.kv_copy_pages([], 6, [(1, 2)])                           # nothing to do


def test_copy_library_refusals():
    """The library's own checks, on an address that nothing follows."""
    lib = pkv.load_library()

    def call(pairs, heads=2, page_bytes=64, n_pages=6, cache=1 << 20, n_pairs=None):
        flat = (ctypes.c_int32 * max(2 * len(pairs), 1))(*[x for p in pairs for x in p])
        return lib.kv_copy_pages((ctypes.c_void_p * 1)(cache), (ctypes.c_int * 1)(heads),
                                 (ctypes.c_int64 * 1)(page_bytes), 1, n_pages, flat,
                                 len(pairs) if n_pairs is None else n_pairs, None)

    for pairs in ([(1, 6)], [(-1, 2)], [(6, 1)], [(1, -1)], [(1, 2), (3, 2)], [(1, 2), (2, 3)],
                  [(2, 3), (1, 2)], [(4, 4)]):
        assert call(pairs) == pkv.PKV_E_BAD_ARG, pairs
    for kw in (dict(heads=0), dict(heads=65536), dict(page_bytes=0), dict(n_pages=0),
               dict(cache=0), dict(n_pairs=-1), dict(page_bytes=1 << 45)):
        assert call([(1, 2)], **kw) == pkv.PKV_E_BAD_ARG, kw
    assert call([]) == pkv.PKV_OK
    assert lib.kv_copy_pages(None, None, None, 0, 6, None, 3, None) == pkv.PKV_OK
    assert lib.kv_copy_pages(None, None, None, 1, 6, None, 3, None) == pkv.PKV_E_BAD_ARG


def test_copy_of_no_pairs_checks_the_caches():
    """n_pairs 0 launches nothing, but refuses what any copy of these caches would."""
    lib = pkv.load_library()

    def call(cache=1 << 20, heads=2, page_bytes=64):
        return lib.kv_copy_pages((ctypes.c_void_p * 1)(cache), (ctypes.c_int * 1)(heads),
                                 (ctypes.c_int64 * 1)(page_bytes), 1, 6, None, 0, None)

    assert call() == pkv.PKV_OK
    for kw in (dict(cache=0), dict(heads=0), dict(page_bytes=0)):
        assert call(**kw) == pkv.PKV_E_BAD_ARG, kw
