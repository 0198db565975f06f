"""Angles of tree_qkv_norm_rope_append at positions up to 2^31 and for any accepted theta, against
decimal arithmetic of 80 digits (64-bit floats hold neither such an angle nor its frequency)."""
from decimal import Decimal, localcontext

import numpy as np
import pytest
import torch

from gpu_util import f64
from tree_util import BF16_STEP

pytestmark = pytest.mark.gpu
pkv = pytest.importorskip("paged_kv_decode_pagetable_gb300")

D, PS = 64, 1 << 19


def atan_inverse(n):
    x = Decimal(1) / n
    total, term, k = x, x, 1
    while abs(term) > Decimal(10) ** -85:
        term = -term / (n * n)
        k += 2
        total += term / k
    return total


def turns(theta, pos):
    """float64 [pos][D / 2]: the fraction of a turn of position * theta^(-2i/D) radians."""
    with localcontext() as c:
        c.prec = 130
        two_pi = 2 * (16 * atan_inverse(5) - 4 * atan_inverse(239))
        ln = Decimal(float(np.float32(theta))).ln()
        f = [(-ln * 2 * i / D).exp() / two_pi for i in range(D // 2)]
        return np.array([[float(int(p) * x % 1) for x in f] for p in pos])


@pytest.mark.parametrize("theta", [2.0 ** -56, 1e-12, 1e-6, 0.5, 1.0, 1e4, 1e9, 3e38])
@pytest.mark.parametrize("ctx", [0, 4_000_000, (1 << 30) - 3, (1 << 31) - 9])
def test_far_angles(theta, ctx):
    """Pairs (1, 0): the results are the angle's cosine and sine. Each is rounded to bf16 once; the
    angle is off by 2^-24 of a half turn, a factor by 2 ulp more."""
    n, Hq = 8, 2
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    q = torch.zeros((n, Hq, D), dtype=torch.bfloat16, device="cuda")
    q[..., :D // 2] = 1
    pages = (ctx + n - 1) // PS + 1
    table = torch.full((2, pages), 1, dtype=torch.int32, device="cuda")
    kc, vc = (torch.zeros((1, 2 * PS, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    qo, err = torch.empty_like(q), i32([0])
    pkv.tree_qkv_norm_rope_append(q, q[:, :1], q[:, :1], None, None, i32([1]), i32([ctx]),
                                  i32([0, n]), i32(list(range(-1, n - 1))), theta, 1e-6, None,
                                  False, table, 2, pages, PS, 2, kc, vc, qo, err)
    assert int(err) == 0
    pos = ctx + np.arange(n, dtype=np.int64)
    angle = 2 * np.pi * turns(theta, pos)
    want = np.concatenate([np.cos(angle), np.sin(angle)], 1)
    bound = BF16_STEP * np.abs(want) + (np.pi * 2.0 ** -24 + 2.0 ** -22) * (1 + BF16_STEP)
    rows = torch.from_numpy(PS + pos % PS).cuda()
    for got in (f64(qo[:, 0]), f64(qo[:, 1]), f64(kc[0, rows])):
        off = np.abs(got - want) / bound
        assert off.max() <= 1, (float(off.max()), np.unravel_index(off.argmax(), off.shape))
