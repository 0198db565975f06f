"""kv_keep_path of caches that are named more than once, or in any order of their addresses: each
one's tokens move once."""
import numpy as np
import pytest
import torch

from oracle import tree
from tree_util import TreeCase, random_tree

pytestmark = pytest.mark.gpu
pkv = pytest.importorskip("paged_kv_decode_pagetable_gb300")


@pytest.mark.parametrize("names", [
    [0, 0], [0, 1, 0, 1], [2, 1, 0], [1, 0, 1, 2, 2, 0], [3, 5, 4, 3] * 20, list(range(90)),
    list(range(90))[::-1], [i * 37 % 90 for i in range(180)]], ids=len)
def test_each_cache_moves_once(names):
    rng = np.random.default_rng([63, len(names)])
    c = TreeCase(rng, 1, 1, 64, 8, [20, 3, 40], [random_tree(rng, 16, 3)] * 3).device(pkv)
    # chains of moves: each source is a later move's destination or the other way round
    path, acc = np.array([[0, 2, 4, 6, 8, 10, 12], [0, 2, 3, 4, 5, 6, 7], [0, 1, 3, 5, 6, 9, 15]]
                         ), np.array([6, 6, 6])
    rows = c.P * 8
    pool = torch.randint(0, 256, (max(names) + 1, 2, rows, 48), dtype=torch.uint8, device="cuda")
    want = pool.cpu().numpy().copy()
    for i in set(names):
        tree.keep_path(want[i], c.table, c.slots, c.ctx, acc, path, 8)
    i32 = lambda x: torch.from_numpy(x.astype(np.int32)).cuda()  # noqa: E731
    pkv.kv_keep_path([pool[i] for i in names], c.t["table"], c.n_slots, c.max_pages, 8, c.P,
                     c.t["slots"], c.t["ctx"], i32(acc), i32(path), c.err)
    torch.cuda.synchronize()
    assert int(c.err) == 0 and np.array_equal(pool.cpu().numpy(), want)


def test_the_same_pair_of_every_layer():
    """K and V of every layer, as a model whose layers share them lists them, through the engine's
    own check of tensors; a part of a cache is refused."""
    rng = np.random.default_rng(64)
    c = TreeCase(rng, 2, 2, 64, 8, [9], [[-1, 0, 0, 2]]).device(pkv)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    k, v = c.t["kc"].nan_to_num_(), c.t["vc"].nan_to_num_()
    args = (c.t["table"], c.n_slots, c.max_pages, 8, c.P, c.t["slots"], c.t["ctx"], i32([2]),
            i32([[0, 2, 3]]), c.err)
    want = [x.cpu().view(torch.int16).numpy().copy() for x in (k, v)]
    for w in want:
        tree.keep_path(w, c.table, c.slots, c.ctx, [2], [[0, 2, 3]], 8)
    pkv.kv_keep_path([k, v] * 12, *args)
    torch.cuda.synchronize()
    for x, w in zip((k, v), want):
        assert np.array_equal(x.cpu().view(torch.int16).numpy(), w)
    with pytest.raises(pkv.BadArgError, match="overlap"):
        pkv.kv_keep_path([k, v, k[1:]], *args)
