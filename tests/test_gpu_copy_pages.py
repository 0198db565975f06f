"""kv_copy_pages on the GPU: pages of bf16 and 8-bit caches and of scales, exactly
the named ones, for every alignment and more pairs or caches than one launch takes;
captured and replayed; and a forked sequence that reads as its source."""
import numpy as np
import pytest
import torch

import workloads as wl

pytestmark = pytest.mark.gpu
pkv = pytest.importorskip("paged_kv_decode_pagetable_gb300")


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pkv.load_library()
    return torch.device("cuda:0")


def random_bytes(rng, shape, dev):
    return torch.from_numpy(rng.integers(0, 256, shape, dtype=np.uint8)).to(dev)


def expect(cache, n_pages, pairs):
    v = cache.cpu().numpy().copy().reshape(cache.shape[0], n_pages, -1)
    src = v[:, [a for a, _ in pairs]].copy()
    v[:, [b for _, b in pairs]] = src
    return v.reshape(cache.shape)


def random_pairs(rng, P, n):
    perm = rng.permutation(P)
    few = max(1, n // 2)
    return [(int(perm[i % few]), int(perm[few + i])) for i in range(n)]


@pytest.mark.parametrize("P,n", [(2, 1), (9, 5), (200, 64), (200, 65), (9000, 3501), (9000, 4400)])
def test_several_caches_of_several_kinds(dev, P, n):
    """Page bytes that are multiples of 16, of 4 and odd, in one call."""
    rng = np.random.default_rng(P + n)
    caches = [random_bytes(rng, (h, P, b), dev)
              for h, b in ((3, 2048), (1, 16), (2, 48), (2, 4), (5, 12), (1, 7), (2, 1040))]
    pairs = random_pairs(rng, P, n)
    want = [expect(c, P, pairs) for c in caches]
    pkv.kv_copy_pages(caches, P, torch.tensor(pairs, dtype=torch.int32))
    for c, w in zip(caches, want):
        assert np.array_equal(c.cpu().numpy(), w)


def test_unaligned_bases_and_guards(dev):
    """Caches inside a larger buffer at every offset; the bytes around stay."""
    rng = np.random.default_rng(5)
    P, pairs = 12, [(3, 7), (3, 1), (11, 0)]
    for off in (0, 1, 4, 8, 16):
        buf = random_bytes(rng, (64 + 2 * P * 160,), dev)
        before = buf.cpu().numpy().copy()
        cache = buf[off:off + 2 * P * 160].view(2, P, 160)
        want = expect(cache, P, pairs)
        pkv.kv_copy_pages([cache], P, pairs)
        got = buf.cpu().numpy()
        assert np.array_equal(got[off:off + want.size], want.reshape(-1))
        assert np.array_equal(got[:off], before[:off])
        assert np.array_equal(got[off + want.size:], before[off + want.size:])


def test_many_layers_and_heads(dev):
    """More caches than one launch describes, and more heads than a grid row."""
    rng = np.random.default_rng(6)
    pairs = [(1, 4), (2, 3)]
    caches = [random_bytes(rng, (2, 6, 32), dev) for _ in range(150)]
    caches += [random_bytes(rng, (40000, 6, 16), dev) for _ in range(2)]
    want = [expect(c, 6, pairs) for c in caches]
    pkv.kv_copy_pages(caches, 6, pairs)
    assert all(np.array_equal(c.cpu().numpy(), w) for c, w in zip(caches, want))


def test_past_32_bit_offsets(dev):
    """A 5 GB head: the last pages lie past 2^32 bytes."""
    P, nb = 5 * 1024, 1 << 20
    cache = torch.zeros((1, P, nb), dtype=torch.uint8, device=dev)
    cache[0, P - 2] = 7
    cache[0, 3] = 9
    pkv.kv_copy_pages([cache], P, [(P - 2, P - 1), (3, P - 5), (P - 2, 1)])
    for p, v in ((P - 1, 7), (P - 5, 9), (1, 7), (0, 0), (2, 0), (P - 4, 0), (P - 6, 0)):
        assert bool((cache[0, p] == v).all()), p


def test_captured_and_other_stream(dev):
    rng = np.random.default_rng(8)
    cache = random_bytes(rng, (2, 10, 64), dev)
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    want = expect(cache, 10, [(1, 2)])
    pkv.kv_copy_pages([cache], 10, [(1, 2)], stream=other)
    other.synchronize()
    assert np.array_equal(cache.cpu().numpy(), want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv.kv_copy_pages([cache], 10, [(5, 6), (5, 9)])
    for _ in range(2):
        cache[:, 5] = torch.randint(0, 256, (2, 64), dtype=torch.uint8, device=dev)
        want = expect(cache, 10, [(5, 6), (5, 9)])
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(cache.cpu().numpy(), want)


def test_forked_compacted_and_unshared_sequences_attend_alike(dev):
    """Samples forked from a prompt, moved and rewritten give the attention of
    their tokens written page by page into a cache of their own."""
    rng = np.random.default_rng(9)
    Hq, Hkv, D, ps, P, mp = 8, 2, 64, 16, 64, 8
    pt = pkv.PageTable(6, ps, P, mp, device=dev)
    kc = torch.zeros((Hkv, P * ps, D), dtype=torch.bfloat16, device=dev)
    vc = torch.zeros_like(kc)

    def put(slot, pos, k, v):
        n = len(pos)
        pkv.kv_append(k, v, torch.full((n,), slot, dtype=torch.int32, device=dev),
                      torch.tensor(pos, dtype=torch.int32, device=dev), pt.dev_table, pt.n_slots,
                      mp, ps, P, kc, vc)

    def rand(n):
        return wl.randn_bf16(rng, (n, Hkv, D)).to(dev), wl.randn_bf16(rng, (n, Hkv, D)).to(dev)

    filler = pt.assign(3 * ps)
    prompt = pt.assign(42)
    pk, pv = rand(42)
    put(prompt, range(42), pk, pv)
    slots, pairs = pt.fork(prompt, 42, 3)
    pkv.kv_copy_pages([kc, vc], P, pairs)
    seq = {s: [pk, pv] for s in slots}
    for s in slots:                              # each sample goes its own way
        pt.reserve(s, 50)
        k, v = rand(8)
        put(s, range(42, 50), k, v)
        seq[s] = [torch.cat([pk, k]), torch.cat([pv, v])]
    s = slots[1]                                 # rewritten from token 20 on
    pairs = pt.unshare(s, 20, 50)
    assert len(pairs) == 1
    pkv.kv_copy_pages([kc, vc], P, pairs)
    k, v = rand(30)
    put(s, range(20, 50), k, v)
    seq[s] = [torch.cat([pk[:20], k]), torch.cat([pv[:20], v])]
    pt.free(filler)
    pt.free(prompt)
    pairs = pt.compact()
    assert len(pairs) > 0
    pkv.kv_copy_pages([kc, vc], P, pairs)
    q = wl.randn_bf16(rng, (3, Hq, D)).to(dev)
    lens = torch.full((3,), 50, dtype=torch.int32, device=dev)

    def attend(table, n_slots, kc, vc, n_pages, bidx):
        out = torch.empty((3, Hq, D), dtype=torch.bfloat16, device=dev)
        n = pkv.paged_decode_attn_workspace(3, Hq, D, pkv.paged_decode_attn_splits(3, Hkv, D, mp,
                                                                                   ps))
        ws = torch.zeros(n, dtype=torch.uint8, device=dev)
        pkv.paged_decode_attn(q, kc, vc, table, n_slots, mp, ps, n_pages, bidx, lens, 0, 0.125, 0,
                              ws, out)
        return out

    got = attend(pt.dev_table, pt.n_slots, kc, vc, P,
                 torch.tensor(slots, dtype=torch.int32, device=dev))
    own = torch.zeros((4, mp), dtype=torch.int32, device=dev)
    for i in range(3):
        own[i + 1, :4] = torch.arange(1 + 4 * i, 5 + 4 * i, dtype=torch.int32)
    k2 = torch.zeros((Hkv, 13 * ps, D), dtype=torch.bfloat16, device=dev)
    v2 = torch.zeros_like(k2)
    for i, s in enumerate(slots):
        k2[:, (1 + 4 * i) * ps:(1 + 4 * i) * ps + 50] = seq[s][0].transpose(0, 1)
        v2[:, (1 + 4 * i) * ps:(1 + 4 * i) * ps + 50] = seq[s][1].transpose(0, 1)
    want = attend(own, 4, k2, v2, 13, torch.arange(1, 4, dtype=torch.int32, device=dev))
    assert torch.equal(got, want)


def test_more_words_than_31_bits_count(dev):
    """2100 pages of 2^20 + 1 bytes, copied byte by byte."""
    n, nb = 2100, (1 << 20) + 1
    P = 2 * n + 3
    cache = torch.empty((1, P, nb), dtype=torch.uint8, device=dev).random_(0, 256)
    before = cache[0, n:n + 3].clone()
    pairs = torch.stack([torch.arange(n - 1, -1, -1), torch.arange(n + 3, P)], 1).int()
    pkv.kv_copy_pages([cache], P, pairs)
    assert torch.equal(cache[0, :n].flip(0), cache[0, n + 3:])
    assert torch.equal(cache[0, n:n + 3], before)
