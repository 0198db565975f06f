"""Rows whose nodes lie outside the packed ones are reported by every call that reads them, also
where no packed node belongs to them."""
import numpy as np
import pytest
import torch

import workloads as wl

pytestmark = pytest.mark.gpu
pkv = pytest.importorskip("paged_kv_decode_pagetable_gb300")

N, D, PS = 8, 64, 16


@pytest.mark.parametrize("starts", [
    [0, 8], [0, 3, 3, 8], [0, 8, 8], [2, 5], [0, 8, 20], [0, 8, 9], [-5, 0, 8], [0, 3, 12], [9, 9],
    [9, 4], [-1, 8], [-3, -1], [0, 4, 4, 8, 9, 10], [0, 8] + [8] * 300 + [9]], ids=str)
def test_every_call_says_so(starts):
    rng = np.random.default_rng(65)
    B = len(starts) - 1
    good = [b for b in range(B) if 0 <= starts[b] <= starts[b + 1] <= N]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    q = wl.randn_bf16(rng, (N, 2, D)).cuda()
    table = torch.arange(1, B + 2, dtype=torch.int32, device="cuda")[:, None].contiguous()
    P = B + 2
    kc, vc = (torch.zeros((1, P * PS, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    rows = (i32(list(range(1, B + 1))), i32([2] * B), i32(starts), i32([-1] * N))
    qo, out = torch.full_like(q, 7), torch.full_like(q, 7)
    words = [i32([0]) for _ in range(3)]
    geometry = (table, B + 1, 1, PS, P)
    pkv.tree_qkv_norm_rope_append(q, q[:, :1], q[:, :1], None, None, *rows, 1e4, 1e-6, None, False,
                                  *geometry, kc, vc, qo, words[0])
    ws = torch.zeros(pkv.paged_tree_attn_workspace(2, 1, D), dtype=torch.uint8, device="cuda")
    pkv.paged_tree_attn(qo, kc, vc, *geometry, *rows, 0, 0.1, ws, out, words[1])
    p = torch.full((N, 4), 0.25, device="cuda")
    acc, nxt, path = i32([7] * B), i32([7] * B), i32([[7] * N] * B)
    pkv.tree_verify(p, None, i32([0] * N), rows[2], rows[3], torch.zeros(N, device="cuda"),
                    torch.zeros(B, device="cuda"), acc, path, nxt, words[2])
    torch.cuda.synchronize()
    assert [int(w) for w in words] == [pkv.PKV_ERR_TREE if len(good) < B else 0] * 3
    mine = sorted(n for b in good for n in range(starts[b], starts[b + 1]))
    for x in (qo, out):       # nodes of the good rows, and no others, are written
        assert ((x != 7).flatten(1).any(1).nonzero()[:, 0]).tolist() == mine
