"""tree_verify where a cluster's CTAs meet soonest after their start: the smallest vocabularies that
2, 4 and 8 CTAs share, and no drafts at all."""
import numpy as np
import pytest
import torch

from oracle import tree

pytestmark = pytest.mark.gpu
pkv = pytest.importorskip("paged_kv_decode_pagetable_gb300")


@pytest.mark.parametrize("V", [2048, 2049, 4097, 8193])
@pytest.mark.parametrize("B", [1, 19, 38, 76, 300])
def test_short_passes(B, V):
    """Probabilities are multiples of 2^-20, so that sums are exact in the oracle too."""
    rng = np.random.default_rng([61, B, V])
    w = rng.multinomial(1 << 20, np.full(V, 1 / V), size=B)
    p = w / 2.0 ** 20
    up = rng.random(B).astype(np.float32)
    start = np.arange(B + 1)
    want = tree.tree_verify(p, None, np.zeros(B, int), start, np.full(B, -1), np.zeros(B), up,
                            path_cols=1)
    t = lambda x, d: torch.from_numpy(np.ascontiguousarray(x)).to("cuda", d)  # noqa: E731
    args = (t(p, torch.float32), None, t(np.zeros(B), torch.int32), t(start, torch.int32),
            t(np.full(B, -1), torch.int32), t(np.zeros(B), torch.float32), t(up, torch.float32))
    outs = [[torch.full(s, 7, dtype=torch.int32, device="cuda") for s in ((B,), (B, 1), (B,))]
            for _ in range(200)]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for o in outs:
        pkv.tree_verify(*args, *o, err)
    torch.cuda.synchronize()
    assert int(err) == 0
    for o in outs:
        for got, ref in zip(o, want):
            assert np.array_equal(got.cpu().numpy(), ref)
