"""Forks and compaction where the page table was made on one stream and the engine is
called on another (GPU): whoever reads through the table, on either stream, finds the
moved pages."""
import pytest
import torch

pytestmark = pytest.mark.gpu
pkv = pytest.importorskip("paged_kv_decode_pagetable_gb300")
from paged_kv_decode_pagetable_gb300 import engine  # noqa: E402

PS, P, MP, HEADS, WIDTH = 4, 40, 12, 2, 64


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pkv.load_library()
    return torch.device("cuda:0")


def spin():
    torch.cuda._sleep(100_000_000)   # about 50 ms of the current stream


def tokens_of(pt, cache, slot, n):
    """Rows of a slot's first n tokens, read through the device table on the current
    stream."""
    t = torch.arange(n, device=cache.device)
    rows = pt.dev_table[slot].long()[t // PS] * PS + t % PS
    return cache[:, rows]


def made(dev, table_stream):
    with torch.cuda.stream(table_stream):
        pt = pkv.PageTable(6, PS, P, MP, device=dev)
    caches = [torch.randn((HEADS, P * PS, WIDTH), device=dev).bfloat16() for _ in range(2)]
    caches.append(torch.randn((HEADS, P * PS), device=dev))
    torch.cuda.synchronize()
    return pt, caches


WAYS = [("default", "side", True), ("default", "side", False), ("side", "default", False),
        ("side", "other", True), ("side", "other", False), ("side", "side", True)]


def streams(table, caller):
    s = {"default": torch.cuda.default_stream(), "side": torch.cuda.Stream(),
         "other": torch.cuda.Stream()}
    return s[table], s[caller]


def under(caller, by_argument):
    """(context, argument) that hand the caller's stream to the engine."""
    if by_argument:
        return torch.cuda.stream(torch.cuda.default_stream()), caller
    return torch.cuda.stream(caller), None


@pytest.mark.parametrize("table,caller,by_argument", WAYS)
def test_compaction_is_seen_by_both_streams(dev, table, caller, by_argument):
    own, use = streams(table, caller)
    for reader in (own, use):
        pt, caches = made(dev, own)
        a, b = pt.assign(9 * PS), pt.assign(10 * PS + 3)
        pt.free(a)
        torch.cuda.synchronize()
        want = [tokens_of(pt, c, b, 10 * PS + 3).clone() for c in caches]
        torch.cuda.synchronize()
        with torch.cuda.stream(use):       # the caller's stream is busy for a while
            spin()
        context, argument = under(use, by_argument)
        with context:
            assert engine.compact_cache(pt, caches, stream=argument) > 0
        with torch.cuda.stream(reader):
            got = [tokens_of(pt, c, b, 10 * PS + 3).clone() for c in caches]
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want)), reader is own


@pytest.mark.parametrize("table,caller,by_argument", WAYS)
def test_fork_is_seen_by_both_streams(dev, table, caller, by_argument):
    own, use = streams(table, caller)
    for reader in (own, use):
        pt, caches = made(dev, own)
        cb = engine.ContinuousBatcher(pt, [engine.Sequence(0, 2 * PS + 3, 5)])
        assert cb.step()
        s = cb.running[0]
        n = 2 * PS + 3
        torch.cuda.synchronize()
        with torch.cuda.stream(use):   # the prompt's last tokens are still being written
            spin()
            for c in caches:
                c[:, pt.pages(s.slot)[2] * PS:(pt.pages(s.slot)[2] + 1) * PS] += 1
        context, argument = under(use, by_argument)
        with context:
            new = cb.fork(s, [1, 2], caches, stream=argument)
        with torch.cuda.stream(reader):
            got = [[tokens_of(pt, c, f.slot, n).clone() for c in caches] for f in new]
        torch.cuda.synchronize()
        want = [tokens_of(pt, c, s.slot, n) for c in caches]
        for g in got:
            assert all(torch.equal(x, y) for x, y in zip(g, want)), reader is own


def test_pending_reads_come_before_the_move(dev):
    """Work in flight on the table's stream that still reads pages freed since, while the
    engine is called on another stream."""
    own, use = streams("side", "other")
    pt, caches = made(dev, own)
    a, b = pt.assign(9 * PS), pt.assign(10 * PS)
    torch.cuda.synchronize()
    rows = [p * PS + i for p in pt.pages(a) for i in range(PS)]
    rows = torch.tensor(rows, device=dev)
    want = [c[:, rows].clone() for c in caches]
    torch.cuda.synchronize()
    with torch.cuda.stream(own):
        spin()
        got = [c[:, rows].clone() for c in caches]
    pt.free(a)
    with torch.cuda.stream(use):
        assert engine.compact_cache(pt, caches) > 0
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_after_pt_set_stream_the_new_stream_counts(dev):
    own, use = streams("side", "other")
    pt, caches = made(dev, torch.cuda.default_stream())
    pkv.pt_set_stream(pt.handle, own)
    a, b = pt.assign(9 * PS), pt.assign(10 * PS)
    pt.free(a)
    torch.cuda.synchronize()
    want = [tokens_of(pt, c, b, 10 * PS).clone() for c in caches]
    torch.cuda.synchronize()
    with torch.cuda.stream(use):
        spin()
        assert engine.compact_cache(pt, caches) > 0
    with torch.cuda.stream(own):
        got = [tokens_of(pt, c, b, 10 * PS).clone() for c in caches]
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
