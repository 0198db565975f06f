"""Tokens of one scale block that stand apart in a call of many tokens (GPU): reported
wherever both stand among the first 4096, over several checking CTAs; and the largest
calls in order are not."""
import numpy as np
import pytest
import torch

import oracle
from test_gpu_q8 import Cache, dev, tokens  # noqa: F401

pytestmark = pytest.mark.gpu
pkv = pytest.importorskip("paged_kv_decode_pagetable_gb300")

H, D, PS, G, PER_SLOT = 1, 16, 8, 4, 100


def scattered(N):
    """Every token in a block of its own: N leading tokens."""
    i = np.arange(N)
    return 1 + i // PER_SLOT, i % PER_SLOT * G


def packed(N):
    """Prompts of 400 tokens, one after the other: a leading token in four."""
    i = np.arange(N)
    return 1 + i // (PER_SLOT * G), i % (PER_SLOT * G)


def bits(rng, dev, slot, pos):
    N, n = len(slot), int(slot.max())
    max_pages = PER_SLOT * G // PS
    P = n * max_pages + 1
    c = Cache(rng, dev, H, D, PS, P, G)
    table = np.zeros((n + 1, max_pages), np.int32)
    table[1:] = rng.permutation(np.arange(1, P)).reshape(n, max_pages)
    t = lambda a: torch.from_numpy(np.asarray(a, np.int32)).to(dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    x = tokens(rng, N, H, D).to(dev)
    pkv.kv_append_q8(x, x, t(slot), t(pos), t(table), n + 1, max_pages, PS, P, c.kc, c.vc, c.ks,
                     c.vs, err)
    return pkv.pkv_read_error_word(err)


@pytest.mark.parametrize("N", [1025, 2049, 3000, 4096, 5000])
@pytest.mark.parametrize("layout", [scattered, packed])
def test_calls_in_order_are_not_reported(dev, N, layout):
    assert bits(np.random.default_rng(N), dev, *layout(N)) == 0


@pytest.mark.parametrize("N,i,j", [(1025, 0, 1024), (1025, 31, 33), (1025, 5, 7),
                                   (1100, 1000, 1030), (1100, 1023, 1025), (2050, 1022, 2049),
                                   (3000, 0, 2999), (3000, 2047, 2050), (4096, 0, 4095),
                                   (4096, 4000, 4095), (5000, 17, 4095), (5000, 255, 257)])
@pytest.mark.parametrize("same", [False, True])
def test_one_clash_among_many_blocks(dev, N, i, j, same):
    """Token j falls into token i's block (or on its very position); all others have
    blocks of their own."""
    slot, pos = scattered(N)
    slot[j], pos[j] = slot[i], pos[i] + (0 if same else 1)
    assert bits(np.random.default_rng(i), dev, slot, pos) == oracle.ERR_ORDER


@pytest.mark.parametrize("N", [1500, 4096])
def test_a_clash_at_every_distance(dev, N):
    rng = np.random.default_rng(N)
    for _ in range(60):
        i = int(rng.integers(0, N - 3))
        j = int(rng.integers(i + 2, N))
        layout = (scattered, packed)[int(rng.integers(2))]
        slot, pos = layout(N)
        slot[j], pos[j] = slot[i], pos[i]     # one position twice, another token between
        assert bits(rng, dev, slot, pos) == oracle.ERR_ORDER, (layout, i, j)


@pytest.mark.parametrize("i,j", [(0, 4096), (4095, 4097), (4200, 4900)])
def test_past_4096_tokens_the_order_is_the_callers(dev, i, j):
    """The header's limit: only a call's first 4096 tokens are looked at."""
    slot, pos = scattered(5000)
    slot[j], pos[j] = slot[i], pos[i] + 1
    assert bits(np.random.default_rng(j), dev, slot, pos) == 0
