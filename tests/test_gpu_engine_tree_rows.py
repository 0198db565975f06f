"""engine.accept_drafts on buffers kept for the largest batch: a smaller batch leaves the tokens
of the other rows where they are."""
import numpy as np
import pytest
import torch

import workloads as wl
from tree_util import TreeCase

pytestmark = pytest.mark.gpu
pkv = pytest.importorskip("paged_kv_decode_pagetable_gb300")


def test_a_batch_that_shrinks():
    from paged_kv_decode_pagetable_gb300 import engine
    rng = np.random.default_rng(62)
    B, V, n = 4, 30, 5
    forks = [-1, 0, 0, 1, 2]            # node 2 is accepted, then node 4
    c = TreeCase(rng, 1, 1, 64, 8, [3, 20, 31, 9], [forks] * B, slots=[2, 4, 1, 3]).device(pkv)
    pt = pkv.PageTable(B, 8, c.P, c.max_pages)        # geometry only
    kc = wl.randn_bf16(rng, (2, c.P * 8, 64)).cuda()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    tokens = i32([0, 1, 2, 3, 4] * B)
    p = torch.zeros((B * n, V), device="cuda")
    p[0::n, 2], p[2::n, 4], p[4::n, 7] = 1.0, 1.0, 1.0
    u, up = torch.full((B * n,), 0.5, device="cuda"), torch.full((B,), 0.5, device="cuda")
    acc, nxt, path, err = i32([0] * B), i32([0] * B), i32([[0] * 6] * B), i32([0])

    def step(rows):
        engine.accept_drafts(pt, [kc], p, None, tokens, c.t["slots"], c.t["ctx"],
                             c.t["row_start"][:rows + 1], c.t["parents"], u, up, acc, path, nxt,
                             err, table=c.t["table"])
        torch.cuda.synchronize()
        assert int(err) == 0

    step(B)
    assert acc.tolist() == [2] * B and nxt.tolist() == [7] * B
    assert path.tolist() == [[0, 2, 4, -1, -1, -1]] * B
    kept = kc.clone()
    kc.copy_(wl.randn_bf16(rng, kc.shape).cuda())     # every row's tokens are others now
    before = kc.clone()
    step(2)
    changed = (kc != before).any(-1).any(0).nonzero()[:, 0].tolist()
    mine = {int(c.table[c.slots[b], (c.ctx[b] + t) // 8]) * 8 + int(c.ctx[b] + t) % 8
            for b in range(2) for t in (1, 2)}
    assert set(changed) == mine and not torch.equal(kept, kc)
