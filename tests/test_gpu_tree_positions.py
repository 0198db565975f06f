"""The append at the last position that a 32-bit number holds, in table rows with room for more."""
import pytest
import torch

pytestmark = pytest.mark.gpu
pkv = pytest.importorskip("paged_kv_decode_pagetable_gb300")

D, PS, PAGES = 64, 1 << 19, (1 << 12) + 8       # a row of 2^31 + 2^22 tokens
LAST = (1 << 31) - 1


@pytest.mark.parametrize("ctx,n,fits", [(LAST - 8, 8, True), (LAST - 7, 8, False), (LAST, 1, False),
                                        (LAST, 64, False), (LAST - 63, 63, True), (-1, 1, False),
                                        (-(1 << 31), 64, False)])
def test_rows_that_reach_beyond_32_bits_are_reported(ctx, n, fits):
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    q = torch.ones((n, 1, D), dtype=torch.bfloat16, device="cuda")
    table = torch.ones((3, PAGES), dtype=torch.int32, device="cuda")
    kc, vc = (torch.zeros((1, 2 * PS, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    qo, err = torch.full_like(q, 7), i32([0])
    pkv.tree_qkv_norm_rope_append(q, q, q, None, None, i32([1]), i32([ctx]), i32([0, n]),
                                  i32([-1] * n), 1e4, 1e-6, None, False, table, 3, PAGES, PS, 2, kc,
                                  vc, qo, err)
    torch.cuda.synchronize()
    assert int(err) == (0 if fits else pkv.PKV_ERR_POS)
    assert int((vc[0] != 0).any(1).sum()) == (n if fits else 0)
    assert bool((qo == 7).all()) != fits
