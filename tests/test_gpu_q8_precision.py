"""paged_decode_attn_q8 where its 32- and 16-bit arithmetic could lose what matters:
scores of any size. Bounds: test_gpu_q8's."""
import numpy as np
import pytest
import torch

from test_gpu_q8 import Case, dev  # noqa: F401

pytestmark = pytest.mark.gpu
pkv = pytest.importorskip("paged_kv_decode_pagetable_gb300")


@pytest.mark.parametrize("e", [0, 8, 14, 20, 26])
def test_equal_scores_of_any_size(dev, e):
    """All keys alike, scores of about 2^e and -2^e: the output is the mean of the values,
    whatever a score's last bit is worth and whatever the scale of V."""
    rng = np.random.default_rng(72)
    for sign in (1.0, -1.0):
        c = Case(rng, 3, 8, 2, 64, 64, 8, [300, 64, 5])
        c.c[0] = np.where(np.isnan(c.c[0]), np.nan, 1.0)
        c.s[0] = np.where(np.isnan(c.s[0]), np.nan, 2.0 ** -6)
        sv = float(np.float32(0.7 * 2.0 ** -6))
        c.s[1] = np.where(np.isnan(c.s[1]), np.nan, sv)
        c.q = torch.full_like(c.q, sign)
        c.device(dev).run(scale=2.0 ** e)
        got = c.out.cpu().double().numpy()
        for b in range(c.B):
            L = int(c.lens[b])
            t = np.arange(L)
            r = c.table[c.slots[b], t // 64].astype(np.int64) * 64 + t % 64
            v = c.c[1][:, r] * sv
            o, A = v.mean(1).repeat(4, 0), np.abs(v).mean(1).repeat(4, 0)
            # the scores are equal to the last bit: weights 2^-11 and sums in fp32
            tol = 2.0 ** -8 * np.abs(o) + (2.0 ** -11 + 2.0 ** -18) * A
            assert (np.abs(got[b] - o) <= tol).all(), (b, sign)
