"""paged_decode_attn_q8 where its 32- and 16-bit arithmetic could lose what matters:
scores of any size, keys of very little weight beside a heavy one, scales of V at the
ends of their range, queries with one very large element.

Bounds: test_gpu_q8's; for light keys with the absolute part of a weight's rounding that
the header states: weights enter the product with V times 2^15, so half a step below
fp16's normal range is 2^-25 * 2^-15 = 2^-40 of the largest."""
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


def light_keys(rng, D, L, heavy, by_scale, B=2):
    """Rows of L keys whose key 0 is 2^heavy times as heavy as each other one, by its
    score or by its scale of V, and has no value: the output is the light keys'."""
    G = 1 if by_scale else 8
    c = Case(rng, B, 8, 2, D, 64, G, [L] * B)
    c.c[0] = np.where(np.isnan(c.c[0]), np.nan, 0.0)
    c.s = [np.where(np.isnan(s), np.nan, 1.0) for s in c.s]
    for b in range(B):
        r = c.table[c.slots[b], 0] * 64
        c.c[1][:, r] = 0.0
        if by_scale:
            c.s[1][:, r] = 2.0 ** heavy
        else:
            c.c[0][:, r, 0] = 32.0
    c.q = torch.zeros_like(c.q)
    c.q[:, :, 0] = 1.0
    return c


@pytest.mark.parametrize("by_scale", [False, True])
@pytest.mark.parametrize("heavy", [12, 18, 24, 27, 31])
@pytest.mark.parametrize("D,L", [(64, 64), (64, 9000), (128, 150), (128, 4000), (256, 300),
                                 (256, 2500), (512, 300), (512, 2500)])
def test_light_keys_beside_a_heavy_one(dev, D, L, heavy, by_scale):
    rng = np.random.default_rng(D + L + heavy)
    c = light_keys(rng, D, L, heavy, by_scale)
    scale = 1.0 if by_scale else heavy * np.log(2) / 32
    c.device(dev).run(scale=scale)
    got = c.out.cpu().double().numpy()
    scale = float(np.float32(scale))
    for b in range(c.B):
        t = np.arange(L)
        r = c.table[c.slots[b], t // 64].astype(np.int64) * 64 + t % 64
        for h in range(c.Hq):
            g = h // 4
            s = scale * c.c[0][g, r, 0]
            sv, cv = c.s[1][g, r // c.G], c.c[1][g, r]
            p = np.exp(s - s.max())
            p /= p.sum()
            o, A, W = (p * sv) @ cv, (p * sv) @ np.abs(cv), (p * sv).max()
            d = 2.0 ** -24 * (D + 8) * s.max() + 2.0 ** -20 * (1 + s.max() / 4)
            tol = (2.0 ** -8 * np.abs(o) + (2.0 ** -11 + 2.0 ** -18) * A
                   + 2.0 ** -40 * W * np.abs(cv).sum(0) + 2 * d * (A + np.abs(o)))
            e = np.abs(got[b, h] - o)
            assert (e <= tol).all(), (b, h, float((e / tol).max()), float((e / A).max()))
    assert pkv.pkv_read_error_word(c.err) == 0


def test_scales_of_v_at_their_ends(dev):
    """Scales of V near the smallest and largest of fp32, whose outputs bf16 still holds."""
    rng = np.random.default_rng(71)
    for e in (-124, -112, -100, 100, 112):
        c = Case(rng, 2, 8, 2, 128, 64, 16, [700, 30], v_spread=1)
        c.s[1] = c.s[1] * 2.0 ** (e + 7)
        c.device(dev).run()
        c.check()


@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("large", [8, 14, 20])
def test_one_large_query_element(dev, D, large):
    """q has an element of 2^large where every key is 0: the scores come from the others,
    and the bound knows only those."""
    rng = np.random.default_rng(D + large)
    c = Case(rng, 3, 8, 2, D, 64, 16, [500, 64, 131])
    c.c[0][:, :, 5] = np.where(np.isnan(c.c[0][:, :, 5]), np.nan, 0.0)
    c.q[:, :, 5] = 2.0 ** large
    c.device(dev).run()
    c.check()
