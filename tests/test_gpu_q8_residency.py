"""8-bit attention beside work that leaves it few places (GPU): calls whose rows are cut
over every CTA end, without a wait that gives up, and give the same bits."""
import numpy as np
import pytest
import torch

from test_gpu_q8 import Case, dev  # noqa: F401

pytestmark = pytest.mark.gpu
pkv = pytest.importorskip("paged_kv_decode_pagetable_gb300")


@pytest.mark.parametrize("D,Hq,Hkv,lens", [(128, 32, 8, [30000]), (64, 8, 1, [70001, 5]),
                                           (256, 8, 2, [9000, 40, 12000]),
                                           (512, 8, 1, [7000, 3000, 20000])])
def test_beside_a_kernel_that_fills_every_sm(dev, D, Hq, Hkv, lens):
    """The other stream runs bf16 attention at D = 512, whose CTAs take an SM's shared
    memory each, so a call's CTAs come in a few at a time as those end."""
    rng = np.random.default_rng(D)
    c = Case(rng, len(lens), Hq, Hkv, D, 64, 16, lens).device(dev)
    want = c.run().clone()
    i32 = dict(dtype=torch.int32, device=dev)
    B, L, P = 64, 16384, 258                     # 64 queries of one sequence
    kc = torch.randn((1, P * 64, 512), device=dev).bfloat16()
    q = torch.randn((B, 8, 512), device=dev).bfloat16()
    table = torch.zeros((2, 256), **i32)
    table[1] = torch.arange(1, 257, **i32)
    n = pkv.paged_decode_attn_workspace(B, 8, 512, pkv.paged_decode_attn_splits(B, 1, 512, 256, 64))
    ws = torch.zeros(n, dtype=torch.uint8, device=dev)
    out = torch.empty_like(q)
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    slots, full = torch.ones(B, **i32), torch.full((B,), L, **i32)
    torch.cuda.synchronize()
    with torch.cuda.stream(other):
        for _ in range(60):
            pkv.paged_decode_attn(q, kc, kc, table, 2, 256, 64, P, slots, full, 0, 512 ** -0.5, 0,
                                  ws, out)
    outs = []
    for _ in range(60):
        c.out = torch.full_like(want, float("nan"))
        outs.append(c.run())
    torch.cuda.synchronize()
    assert pkv.pkv_read_error_word(c.err) == 0
    assert all(torch.equal(o, want) for o in outs) and not c.ws.any()
