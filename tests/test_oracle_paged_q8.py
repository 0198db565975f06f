"""Pins of the 8-bit cache's oracle: the e4m3 rounding against torch's type over
every bf16 value, the scale's defining inequality, a block worked by hand, and the
properties of an append (CPU only)."""
import numpy as np
import pytest
import torch

import oracle


def all_bf16():
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16)
    return bits.view(torch.bfloat16)


def test_round_e4m3_equals_torch_on_every_bf16():
    x = all_bf16().double()
    want = x.clamp(-448, 448).to(torch.float8_e4m3fn).double().numpy()
    got = oracle.round_e4m3(x.numpy())
    assert np.array_equal(got, want, equal_nan=True)


def test_round_e4m3_halves_go_to_even():
    # spacing 1 in [8, 16): 8.5 -> 8, 9.5 -> 10; 2^-9 below 2^-6; 17 halves 16 and 18
    assert oracle.round_e4m3([8.5, 9.5, -9.5, 17, 19, 449, -1e9]).tolist() == \
        [8, 10, -10, 16, 20, 448, -448]
    assert oracle.round_e4m3([1.5 * 2.0 ** -9, 2.5 * 2.0 ** -9, 2.0 ** -10]).tolist() == \
        [2 * 2.0 ** -9, 2 * 2.0 ** -9, 0.0]


def test_scale_is_the_smallest_power_of_two_that_fits():
    a = all_bf16().double().abs()
    a = a[torch.isfinite(a)].numpy()
    for v in np.unique(a)[::37].tolist() + [0.0, 448.0, 449.0, 224.0, 1e-45, 3.3e38]:
        s = oracle.need_scale(v)
        assert np.frexp(s)[0] == 0.5 and s >= 2.0 ** -126
        assert v / s <= 448
        assert s == 2.0 ** -126 or v / (s / 2) > 448, v


def test_block_worked_by_hand():
    """Page of 4 rows, blocks of 4, one head, D = 2. Token 0 (7, 1): 7/448 = 2^-6, so
    codes 448, 64. Token 1 (8, 0): needs 2^-5: token 0's codes halve to 224, 32, token 1
    gets 256, 0. Token 2 (1, 1) fits: 32, 32. Token 4 opens the next block at 2^-9."""
    table = np.array([[0, 0], [2, 1]])
    codes, scales = np.zeros((1, 12, 2)), np.zeros((1, 3))

    def put(pos, *x):
        return oracle.kv_append_q8(codes, scales, np.array([[x]], float), table, [1], [pos], 4, 3,
                                   4)

    assert put(0, 7, 1) == 0
    assert scales[0].tolist() == [0, 0, 2.0 ** -6] and codes[0, 8].tolist() == [448, 64]
    put(1, 8, 0)
    assert scales[0, 2] == 2.0 ** -5
    assert codes[0, 8:10].tolist() == [[224, 32], [256, 0]]
    put(2, 1, 1)
    assert scales[0, 2] == 2.0 ** -5 and codes[0, 10].tolist() == [32, 32]
    put(4, 0.875, -0.5)
    assert scales[0, 1] == 2.0 ** -9 and codes[0, 4].tolist() == [448, -256]
    put(0, 1, 1)                      # the block's first row starts it anew
    assert scales[0, 2] == 2.0 ** -8 and codes[0, 8].tolist() == [256, 256]


@pytest.mark.parametrize("G", [1, 4, 16])
def test_one_call_and_token_by_token_agree(G):
    """With values in the codes' normal range (ratio to the largest above 2^-8)
    a block filled token by token holds the codes of one call; every value is within
    half a step (2^-4 relative) or 2^-10 scales."""
    rng = np.random.default_rng(G)
    H, D, ps, n = 2, 8, 16, 45
    x = rng.uniform(1, 2, (n, H, D)) * rng.choice([-1, 1], (n, H, D)) \
        * np.exp2(rng.integers(-3, 4, (n, 1, 1)))
    x = torch.from_numpy(x).bfloat16().double().numpy()
    table = np.array([[0, 0, 0], [3, 1, 2]])
    a = [np.zeros((H, 64, D)), np.zeros((H, 64 // G))]
    b = [np.zeros((H, 64, D)), np.zeros((H, 64 // G))]
    pos = np.arange(n)
    assert oracle.kv_append_q8(*a, x, table, np.ones(n, int), pos, ps, 4, G) == 0
    for i in range(n):
        oracle.kv_append_q8(*b, x[i:i + 1], table, [1], pos[i:i + 1], ps, 4, G)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])
    rows = np.array([oracle.physical_row(table, 1, p, ps) for p in pos])
    got = oracle.dequantise(a[0], a[1], G)[:, rows].transpose(1, 0, 2)
    s = np.repeat(a[1], G, axis=1)[:, rows].T[:, :, None]
    assert (np.abs(got - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * s)).all()


def test_specials_and_errors():
    table = np.array([[0, 0], [1, -1], [1, 9]])
    codes, scales = np.zeros((1, 16, 2)), np.zeros((1, 4))
    x = np.array([[[np.inf, 3.0]], [[np.nan, -np.inf]]])
    assert oracle.kv_append_q8(codes, scales, x, table, [1, 1], [0, 1], 8, 2, 4) == 0
    assert scales[0, 2] == 2.0 ** -7 and codes[0, 8].tolist() == [448, 384]
    assert np.isnan(codes[0, 9, 0]) and codes[0, 9, 1] == -448
    before = codes.copy()
    for slot, pos, bit in ((1, 8, oracle.ERR_PAGE_NEG), (2, 8, oracle.ERR_PAGE_RANGE),
                           (3, 0, oracle.ERR_SLOT), (1, 16, oracle.ERR_POS),
                           (1, -1, oracle.ERR_POS), (0, 0, 0)):
        assert oracle.kv_append_q8(codes, scales, x[:1], table, [slot], [pos], 8, 2, 4) == bit
    assert np.array_equal(codes, before, equal_nan=True)
    for held in (0.0, np.inf, np.nan, -1.0):          # no usable scale: the rows before clear
        codes[0, 8:12], scales[0, 2] = 5.0, held
        oracle.kv_append_q8(codes, scales, np.full((1, 1, 2), 448.0), table, [1], [2], 8, 2, 4)
        assert scales[0, 2] == 1 and codes[0, 8:12, 0].tolist() == [0, 0, 448, 5]
    codes[0, 8:12], scales[0, 2] = 4.0, 3.0           # rounded up to 4
    oracle.kv_append_q8(codes, scales, np.full((1, 1, 2), 8.0), table, [1], [2], 8, 2, 4)
    assert scales[0, 2] == 4 and codes[0, 8:11, 0].tolist() == [3, 3, 2]
