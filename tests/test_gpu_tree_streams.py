"""The attention on several streams at once, each with a workspace of its own: zeroed before the
first call, alive until the stream has ended, outputs that show what was not written."""
import numpy as np
import pytest
import torch

from tree_util import TreeCase, random_tree

pytestmark = pytest.mark.gpu
pkv = pytest.importorskip("paged_kv_decode_pagetable_gb300")


@pytest.mark.parametrize("Hq,Hkv,D,nodes", [(16, 4, 128, 6), (16, 4, 128, 40), (8, 1, 64, 30),
                                            (8, 1, 256, 20), (8, 1, 512, 12)])
def test_streams_of_their_own(Hq, Hkv, D, nodes):
    rng = np.random.default_rng([66, D, nodes])
    c = TreeCase(rng, Hq, Hkv, D, 16, rng.integers(1, 900, 9),
                 [random_tree(rng, nodes, 2) for _ in range(9)]).device(pkv)
    c.check(pkv)
    want = c.out.clone()
    runs = [(torch.cuda.Stream(), torch.zeros_like(c.ws),
             [torch.full_like(c.out, float("nan")) for _ in range(5)]) for _ in range(3)]
    torch.cuda.synchronize()
    for s, ws, outs in runs:
        with torch.cuda.stream(s):
            for out in outs:
                c.call(pkv, ws=ws, out=out)
    torch.cuda.synchronize()
    assert int(c.err) == 0
    for _, _, outs in runs:
        for out in outs:
            assert torch.equal(out, want)
