"""The 8-bit cache on the GPU: the quantising append bit for bit against the
oracle, the decode attention against a 64-bit computation from the same codes.

Bounds of the attention, per output (u = 2^-24, p the softmax weights, w = p * scale
of v relative to the row's largest, |cv| the codes of v):
  * the output rounded once to bf16: 2^-8 |o| (half a step of 2^-7);
  * w rounded to fp16 (half a step 2^-11 relative, 2^-25 absolute below its normal
    range), in fp32 sums before and after: (2^-11 + 2^-18) A + 2^-25 W sum|cv|, with
    A = sum p |v| and W the row's largest p * scale of v;
  * a score off by d moves its weight, and the sum, by a factor e^d: 2 d (A + |o|) with
    d = (D + 8) u S + 2^-20 (1 + |s|max / 4): the fp32 sum over D terms whose magnitudes
    sum to S (that of the scores, largest over keys), exponentials and logarithms
    good to 2^-21 and arguments rounded at |s| log2(e) u.
Nothing else enters: e4m3 codes are exact in fp16, and so is q scaled to its row's
largest (its smallest elements lose at most 2^-25 of that: within (D + 8) u S's slack).
"""
import numpy as np
import pytest
import torch

import oracle
import workloads as wl

pytestmark = pytest.mark.gpu
pkv = pytest.importorskip("paged_kv_decode_pagetable_gb300")
FP8 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pkv.load_library()
    return torch.device("cuda:0")


def codes_f64(t):
    return t.detach().cpu().double().numpy()


def to_codes(a, dev):
    """e4m3 tensor holding the (exactly representable) values a; NaN allowed."""
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(FP8).to(dev)


# ------------------------------------------------------------------ append ---

class Cache:
    """A random cache in use, on the GPU and as the oracle's arrays."""

    def __init__(self, rng, dev, H, D, ps, P, G, scale_lo=-9, scale_hi=3):
        self.H, self.D, self.ps, self.P, self.G, self.dev = H, D, ps, P, G, dev
        rows = P * ps
        self.np = []
        for _ in range(2):
            codes = oracle.round_e4m3(rng.standard_normal((H, rows, D)) * 60)
            scale = np.exp2(rng.integers(scale_lo, scale_hi + 1, (H, rows // G)))
            self.np.append([codes, scale])
        self.kc, self.vc = (to_codes(c, dev) for c, _ in self.np)
        self.ks, self.vs = (torch.from_numpy(s.astype(np.float32)).to(dev) for _, s in self.np)

    def append(self, k, v, table, bidx, pos, err=None, prefill=False, stream=None):
        """Both sides; returns the oracle's error bits."""
        t = lambda a: None if a is None else torch.from_numpy(np.asarray(a, np.int32)).to(self.dev)
        kk, vv = (x.transpose(0, 1).contiguous() if prefill else x for x in (k, v))
        call = pkv.kv_append_prefill_q8 if prefill else pkv.kv_append_q8
        call(kk.to(self.dev), vv.to(self.dev), t(bidx), t(pos), t(table), table.shape[0],
             table.shape[1], self.ps, self.P, self.kc, self.vc, self.ks, self.vs, err)
        bits = 0
        for x, (codes, scale) in zip((k, v), self.np):
            bits |= oracle.kv_append_q8(codes, scale, x.double().numpy(), table, bidx, pos,
                                        self.ps, self.P, self.G)
        return bits

    def check(self):
        for got, scale, (codes, s) in ((self.kc, self.ks, self.np[0]),
                                       (self.vc, self.vs, self.np[1])):
            assert np.array_equal(codes_f64(got), codes, equal_nan=True)
            assert np.array_equal(scale.cpu().double().numpy(), s, equal_nan=True)


def tokens(rng, N, H, D):
    """Tokens of very different size, so that scales grow and stay."""
    size = np.exp2(rng.integers(-6, 7, (N, 1, 1)))
    x = rng.standard_normal((N, H, D)) * size
    return torch.from_numpy(x.astype(np.float32)).bfloat16()


def slot_table(rng, n, max_pages, P):
    table = np.full((n + 1, max_pages), -1, np.int32)
    table[0] = 0
    table[1:] = rng.permutation(np.arange(1, P))[:n * max_pages].reshape(n, max_pages)
    return table


@pytest.mark.parametrize("H,D,ps,G", [(1, 64, 16, 16), (8, 128, 64, 16), (2, 256, 32, 32),
                                      (1, 512, 64, 64), (3, 128, 64, 1), (2, 16, 8, 8),
                                      (5, 48, 48, 16), (2, 80, 128, 128), (1, 1040, 8, 4)])
@pytest.mark.parametrize("prefill", [False, True])
def test_steps_after_prompts_match_the_oracle(dev, H, D, ps, G, prefill):
    """Packed prompts of odd lengths, then several decode steps of all slots in a
    shuffled order with padding rows between, then a few tokens at once."""
    rng = np.random.default_rng(H * 1000 + D + G)
    n, max_pages = 6, 5
    P = n * max_pages + 2
    c = Cache(rng, dev, H, D, ps, P, G)
    table = slot_table(rng, n, max_pages, P)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    lens = rng.integers(0, 3 * ps, n)
    lens[0], lens[1] = 1, ps
    slots = np.repeat(np.arange(1, n + 1), lens)
    pos = np.concatenate([np.arange(x) for x in lens])
    assert c.append(tokens(rng, len(pos), H, D), tokens(rng, len(pos), H, D), table, slots, pos,
                    err, prefill) == 0
    c.check()
    for _ in range(6):
        order = rng.permutation(n)
        bidx = np.concatenate([order[:3] + 1, [0], order[3:] + 1, [0, 0]])
        at = np.concatenate([lens[order[:3]], [0], lens[order[3:]], [0, 7]])
        assert c.append(tokens(rng, n + 3, H, D), tokens(rng, n + 3, H, D), table, bidx, at, err,
                        prefill) == 0
        lens += 1
        c.check()
    k = min(5, 5 * ps - int(lens.max()))
    slots = np.repeat(np.arange(1, n + 1), k)
    pos = (lens[:, None] + np.arange(k)).reshape(-1)
    assert c.append(tokens(rng, n * k, H, D), tokens(rng, n * k, H, D), table, slots, pos, err,
                    prefill) == 0
    c.check()
    assert pkv.pkv_read_error_word(err) == 0


def test_long_prompt_and_many_rows(dev):
    """More tokens than a launch gives one warp each, and windows that cut runs."""
    rng = np.random.default_rng(3)
    for H, D, ps, G, lens in ((2, 64, 16, 8, [4001, 3, 977]), (4, 128, 64, 64, [2500]),
                              (1, 64, 8, 1, [3000, 5])):
        max_pages = max(-(-x // ps) for x in lens)
        P = len(lens) * max_pages + 1
        c = Cache(rng, dev, H, D, ps, P, G)
        table = slot_table(rng, len(lens), max_pages, P)
        slots = np.repeat(np.arange(1, len(lens) + 1), lens)
        pos = np.concatenate([np.arange(x) for x in lens])
        err = torch.zeros(1, dtype=torch.int32, device=dev)
        N = len(pos)
        assert c.append(tokens(rng, N, H, D), tokens(rng, N, H, D), table, slots, pos, err,
                        True) == 0
        c.check()
        assert pkv.pkv_read_error_word(err) == 0


def test_token_by_token_grows_the_scale(dev):
    """A block filled in ascending and descending sizes, zeros first."""
    rng = np.random.default_rng(4)
    H, D, ps, G = 2, 64, 16, 16
    c = Cache(rng, dev, H, D, ps, 5, G)
    table = slot_table(rng, 1, 4, 5)
    for i in range(64):
        size = 2.0 ** (i % 16 - 20 if i < 32 else -(i % 16))
        x = tokens(rng, 1, H, D) * (0 if i % 16 == 0 else size)
        c.append(x, -x, table, [1], [i])
        c.check()


def test_special_values_and_held_scales(dev):
    """Infinities, NaN, zeros, the largest and the subnormal bf16; held scales
    that are no power of two, zero, negative, infinite or NaN."""
    rng = np.random.default_rng(5)
    H, D, ps, G = 1, 16, 8, 8
    table = slot_table(rng, 1, 8, 10)
    c = Cache(rng, dev, H, D, ps, 10, G)
    vals = np.array([np.inf, -np.inf, np.nan, 0.0, -0.0, 3.38e38, 1e-40, 2.0 ** -133, 1.0, -448.0,
                     1e30, 2.0 ** -126, -3e38, 7.0, 1e-3, -2.0 ** -130], np.float32)
    rows = []
    for i in range(64):
        m = [1, 16, 3, 16, 8, 16, 16, 5][i % 8]
        x = np.where(rng.random(16) < m / 16, rng.permutation(vals), 0)
        rows.append(x)
    x = torch.from_numpy(np.stack(rows).astype(np.float32)).bfloat16().view(64, 1, 16)
    held = [0.0, np.inf, np.nan, -1.0, 3.0, 2.0 ** -140, 2.0 ** 127, 0.3]
    for i in range(64):
        if i % 8 == 3:                  # the block's scale is replaced by an odd one
            blk = oracle.physical_row(table, 1, i, ps) // G
            for t, (_, s) in ((c.ks, c.np[0]), (c.vs, c.np[1])):
                t[0, blk] = held[i // 8]
                s[0, blk] = held[i // 8]
        c.append(x[i:i + 1], x[63 - i:64 - i], table, [1], [i])
        c.check()


def test_errors_without_fault(dev):
    """Every invalid token is reported and skipped, the others are written."""
    rng = np.random.default_rng(6)
    H, D, ps, G, P = 2, 32, 8, 4, 6
    table = np.array([[0, 0], [3, P], [-1, 2], [-7, 2**31 - 1]], np.int32)
    c = Cache(rng, dev, H, D, ps, P, G)
    bidx = [1, 4, -1, 1, 2, 2, 1, 3, 3, 2**31 - 1, -2**31, 2]
    pos = [0, 0, 0, 8, 0, 16, -1, 0, 8, 0, 0, 2**31 - 1]
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    x, y = tokens(rng, 12, H, D), tokens(rng, 12, H, D)
    want = c.append(x, y, table, bidx, pos, err)
    assert want == 15 and pkv.pkv_read_error_word(err) == want
    c.check()
    c.append(x, y, table, bidx, pos, None)              # without an error word
    c.check()
    # batch_idx None: row b is slot b, row 0 the padding slot
    table = np.array([[0], [1], [2]], np.int32)
    assert c.append(x[:3], y[:3], table, None, [0, 1, 5]) == 0
    c.check()


@pytest.mark.parametrize("bidx,pos", [([1, 1], [3, 3]), ([1, 2, 1], [0, 0, 1]),
                                      ([1, 1], [1, 0]), ([1, 1, 2, 1], [6, 7, 0, 5]),
                                      ([1, 1, 1], [4, 6, 5])])
def test_tokens_of_a_block_apart_are_reported(dev, bidx, pos):
    rng = np.random.default_rng(7)
    H, D, ps, G, P = 1, 32, 8, 4, 6
    c = Cache(rng, dev, H, D, ps, P, G)
    before = c.kc.clone()
    table = np.array([[0], [3], [4]], np.int32)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    t = lambda a: torch.tensor(a, dtype=torch.int32, device=dev)
    x = tokens(rng, len(pos), H, D).to(dev)
    pkv.kv_append_q8(x, x, t(bidx), t(pos), t(table.tolist()), 3, 1, ps, P, c.kc, c.vc, c.ks, c.vs,
                     err)
    assert pkv.pkv_read_error_word(err) == pkv.PKV_ERR_ORDER == oracle.ERR_ORDER
    # the damage stays in the named slots' pages
    for p in (0, 1, 2, 5):
        assert torch.equal(c.kc.view(torch.uint8)[:, p * ps:(p + 1) * ps],
                           before.view(torch.uint8)[:, p * ps:(p + 1) * ps])


def test_tokens_of_one_page_in_separate_blocks_are_fine(dev):
    """Only a block's tokens must stand together; blocks may come in any order."""
    rng = np.random.default_rng(8)
    H, D, ps, G, P = 2, 32, 16, 4, 6
    c = Cache(rng, dev, H, D, ps, P, G)
    table = slot_table(rng, 2, 2, P)
    bidx = [1, 1, 2, 1, 1, 1, 2, 1]
    pos = [8, 9, 4, 0, 1, 2, 16, 13]
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    assert c.append(tokens(rng, 8, H, D), tokens(rng, 8, H, D), table, bidx, pos, err) == 0
    c.check()
    assert pkv.pkv_read_error_word(err) == 0


def test_captured_append_follows_its_inputs(dev):
    rng = np.random.default_rng(9)
    H, D, ps, G, n = 2, 128, 16, 16, 4
    P = 1 + 2 * n
    c = Cache(rng, dev, H, D, ps, P, G)
    table = slot_table(rng, n, 2, P)
    d_table = torch.from_numpy(table).to(dev)
    k = torch.zeros((n, H, D), dtype=torch.bfloat16, device=dev)
    v = torch.zeros_like(k)
    bidx = torch.arange(1, n + 1, dtype=torch.int32, device=dev)
    pos = torch.zeros(n, dtype=torch.int32, device=dev)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv.kv_append_q8(k, v, bidx, pos, d_table, n + 1, 2, ps, P, c.kc, c.vc, c.ks, c.vs)
    for i in range(20):
        x, y = tokens(rng, n, H, D), tokens(rng, n, H, D)
        k.copy_(x)
        v.copy_(y)
        pos.fill_(i)
        g.replay()
        for a, (codes, s) in zip((x, y), c.np):
            oracle.kv_append_q8(codes, s, a.double().numpy(), table, np.arange(1, n + 1),
                                np.full(n, i), ps, P, G)
    torch.cuda.synchronize()
    c.check()


# --------------------------------------------------------------- attention ---

class Case:
    """A paged 8-bit cache; codes that no row may read are NaN, their blocks'
    scales too unless a readable token shares them."""

    def __init__(self, rng, B, Hq, Hkv, D, ps, G, lens, slots=None, extra=3, max_pages=None,
                 v_spread=3, pow2=True):
        self.B, self.Hq, self.Hkv, self.D, self.ps, self.G = B, Hq, Hkv, D, ps, G
        self.lens = np.asarray(lens, np.int64)
        nb = -(-self.lens // ps)
        self.P = int(nb.sum()) + extra + 1
        self.max_pages = max_pages or max(int(nb.max()), 1)
        self.slots = np.arange(1, B + 1) if slots is None else np.asarray(slots)
        self.n_slots = max(B, int(self.slots.max())) + 1
        self.table = np.full((self.n_slots, self.max_pages), -1, np.int32)
        self.table[0] = 0
        it = iter(rng.permutation(np.arange(1, self.P)))
        live = np.zeros(self.P * ps, bool)
        for b in range(B):
            if self.slots[b] == 0:
                continue
            for j in range(nb[b]):
                p = self.table[self.slots[b], j] = next(it)
                live[p * ps:p * ps + min(ps, int(self.lens[b]) - j * ps)] = True
        rows = self.P * ps
        self.c, self.s = [], []
        for spread in (3, v_spread):
            codes = oracle.round_e4m3(rng.standard_normal((Hkv, rows, D)) * 100)
            codes[:, ~live] = np.nan
            s = np.exp2(rng.uniform(-7 - spread, -7 + spread, (Hkv, rows // G)))
            s = np.exp2(np.round(np.log2(s))) if pow2 else s.astype(np.float32).astype(np.float64)
            s[:, ~live.reshape(-1, G).any(1)] = np.nan
            self.c.append(codes)
            self.s.append(s)
        self.q = wl.randn_bf16(rng, (B, Hq, D))

    def device(self, dev):
        t = lambda a: torch.from_numpy(np.asarray(a, np.int32)).to(dev)
        self.t = dict(q=self.q.to(dev), kc=to_codes(self.c[0], dev), vc=to_codes(self.c[1], dev),
                      ks=torch.from_numpy(self.s[0].astype(np.float32)).to(dev),
                      vs=torch.from_numpy(self.s[1].astype(np.float32)).to(dev),
                      table=t(self.table), bidx=t(self.slots), lens=t(self.lens))
        self.ws = workspace(self.Hq, self.Hkv, self.D, dev)
        self.out = torch.full((self.B, self.Hq, self.D), float("nan"), dtype=torch.bfloat16,
                              device=dev)
        self.err = torch.zeros(1, dtype=torch.int32, device=dev)
        return self

    def run(self, window=0, scale=None, lens=None):
        t = self.t
        pkv.paged_decode_attn_q8(t["q"], t["kc"], t["vc"], t["ks"], t["vs"], t["table"],
                                 self.n_slots, self.max_pages, self.ps, self.P, t["bidx"],
                                 t["lens"] if lens is None else lens, window,
                                 scale or self.D ** -0.5, self.ws, self.out, self.err)
        return self.out

    def expect(self, window=0, scale=None, rows=None):
        """(output, bound) in 64 bits; the bound is the module's."""
        scale = scale or self.D ** -0.5
        out = np.zeros((self.B, self.Hq, self.D))
        tol = np.zeros_like(out)
        u, G = 2.0 ** -24, self.Hq // self.Hkv
        for b in range(self.B) if rows is None else rows:
            L = int(self.lens[b])
            if self.slots[b] == 0 or L <= 0:
                continue
            t = np.arange(max(0, L - window) if window > 0 else 0, L)
            r = self.table[self.slots[b], t // self.ps].astype(np.int64) * self.ps + t % self.ps
            for h in range(self.Hq):
                g = h // G
                q = self.q[b, h].double().numpy()
                k = self.c[0][g, r] * self.s[0][g, r // self.G][:, None]
                sv = self.s[1][g, r // self.G]
                cv = self.c[1][g, r]
                s = scale * (k @ q)
                S = scale * (np.abs(k) @ np.abs(q)).max()
                p = np.exp(s - s.max())
                p /= p.sum()
                o = (p * sv) @ cv
                A = (p * sv) @ np.abs(cv)
                W = (p * sv).max()
                d = (self.D + 8) * u * S + 2.0 ** -20 * (1 + np.abs(s).max() / 4)
                out[b, h] = o
                tol[b, h] = (2.0 ** -8 * np.abs(o) + (2.0 ** -11 + 2.0 ** -18) * A
                             + 2.0 ** -25 * W * np.abs(cv).sum(0) + 2 * d * (A + np.abs(o)))
        return out, tol

    def check(self, window=0, scale=None, rows=None):
        got = self.out.cpu().double().numpy()
        want, tol = self.expect(window, scale, rows)
        rows = range(self.B) if rows is None else rows
        for b in rows:
            assert np.isfinite(got[b]).all(), b
            e = np.abs(got[b] - want[b])
            assert (e <= tol[b]).all(), (b, float((e - tol[b]).max()), float(e.max()))
        assert pkv.pkv_read_error_word(self.err) == 0


def workspace(Hq, Hkv, D, dev):
    return torch.zeros(pkv.paged_decode_attn_q8_workspace(Hq, Hkv, D), dtype=torch.uint8,
                       device=dev)


@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("ps,G", [(64, 16), (16, 16), (8, 1), (128, 32), (32, 2), (256, 256)])
def test_small_shapes(dev, D, ps, G):
    rng = np.random.default_rng(D + ps + G)
    for Hq, Hkv in ((1, 1), (8, 1), (12, 4), (14, 2)):
        lens = rng.integers(1, 400, 5)
        c = Case(rng, 5, Hq, Hkv, D, ps, G, lens).device(dev)
        for window in (0, 1, 63, 129):
            c.run(window)
            c.check(window)


@pytest.mark.parametrize("L", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 300])
def test_every_tail(dev, L):
    rng = np.random.default_rng(L)
    c = Case(rng, 3, 4, 2, 128, 64, 16, [L, max(1, L - 1), L + 1]).device(dev)
    for window in (0, 16, 64, 100):
        c.run(window)
        c.check(window)


def test_rows_without_keys_are_zero(dev):
    """Length 0, negative and padding rows: exact zeros, whatever the cache holds."""
    rng = np.random.default_rng(20)
    c = Case(rng, 6, 8, 2, 128, 16, 4, [40, 0, 17, 5, 0, 70], slots=[3, 1, 0, 5, 0, 2]).device(dev)
    c.run()
    want, tol = c.expect()
    got = c.out.cpu().double().numpy()
    assert (np.abs(got - want) <= tol).all()
    for b in (1, 2, 4):
        assert not c.out[b].any()
    assert pkv.pkv_read_error_word(c.err) == 0
    all_empty = torch.zeros(6, dtype=torch.int32, device=dev)
    c.out.fill_(float("nan"))
    c.run(lens=all_empty)
    assert not c.out.any()


@pytest.mark.parametrize("Hq,Hkv,D,ps,G,L", [(32, 8, 128, 64, 16, 9000), (4, 1, 64, 16, 8, 70001),
                                             (8, 1, 512, 64, 64, 6001), (2, 2, 256, 128, 1, 5000)])
def test_long_rows_are_cut_and_joined(dev, Hq, Hkv, D, ps, G, L):
    rng = np.random.default_rng(L)
    c = Case(rng, 2, Hq, Hkv, D, ps, G, [L, 3], slots=[2, 1]).device(dev)
    for window in (0, 4000):
        c.run(window)
        c.check(window)


def test_large_batch_and_the_most_rows(dev):
    rng = np.random.default_rng(30)
    lens = rng.integers(0, 90, 512)
    c = Case(rng, 512, 4, 2, 64, 16, 16, lens, slots=rng.permutation(np.arange(1, 513))).device(dev)
    c.run()
    c.check()
    lens = np.rint(np.exp(rng.uniform(0, np.log(3000), 70))).astype(int)
    c = Case(rng, 70, 32, 8, 128, 64, 64, lens).device(dev)
    c.run()
    c.check(rows=rng.choice(70, 12, replace=False))


def test_rows_may_share_a_slot(dev):
    """Several queries of one sequence, each with its own length."""
    rng = np.random.default_rng(31)
    c = Case(rng, 4, 8, 2, 128, 64, 16, [200, 10, 10, 10])
    c.slots[1:] = 1
    c.lens[1:] = [199, 64, 1]
    c.device(dev).run()
    c.check()


@pytest.mark.parametrize("spread", [20, 60])
def test_scales_of_v_far_apart(dev, spread):
    """Blocks whose scales of v differ by 2^40 and 2^120: each output is as good as
    its largest contributions."""
    rng = np.random.default_rng(spread)
    c = Case(rng, 4, 8, 2, 128, 64, 16, [500, 64, 17, 130], v_spread=spread).device(dev)
    c.run()
    c.check()
    c = Case(rng, 4, 8, 2, 64, 16, 1, [500, 64, 17, 130], v_spread=spread, pow2=False).device(dev)
    c.run()
    c.check()


def test_scales_of_zero_and_sharp_scores(dev):
    """Scales of zero make keys even and values zero; a scale of 4 on the scores
    leaves one key of weight."""
    rng = np.random.default_rng(33)
    c = Case(rng, 3, 4, 2, 128, 64, 16, [200, 64, 33])
    c.s[0][:, ::3] *= 0
    c.s[1][:, ::2] *= 0
    c.device(dev).run()
    c.check()
    for a in (0, 1):
        c.s[a] = np.where(np.isnan(c.s[a]), np.nan, 0.0)
    c.device(dev).run()
    assert not c.out.any()
    c = Case(rng, 3, 4, 2, 128, 64, 16, [200, 64, 33]).device(dev)
    c.run(scale=4.0)
    c.check(scale=4.0)


def test_queries_of_every_size(dev):
    """q scaled by 2^-100 to 2^100 with the score scale the other way."""
    rng = np.random.default_rng(34)
    for e in (-100, -30, 30, 100):
        c = Case(rng, 2, 4, 1, 64, 16, 16, [90, 20])
        c.q = (c.q.float() * 2.0 ** e).bfloat16()
        c.device(dev).run(scale=2.0 ** -e / 8)
        c.check(scale=2.0 ** -e / 8)
    c = Case(rng, 2, 4, 1, 64, 16, 16, [90, 20])
    c.q.zero_()
    c.device(dev).run()
    c.check()


def test_bad_tables_and_lengths_are_reported(dev):
    """Entries outside the cache, slots outside the table, lengths past it: bits in
    the error word, no access through them, other rows as they were."""
    rng = np.random.default_rng(35)
    for ps in (16, 64, 128):
        c = Case(rng, 5, 8, 2, 128, ps, 8, [300, 200, 150, 90, 260], slots=[1, 2, 3, 4, 5])
        c.device(dev).run()
        good = c.out.clone()
        for row, col, val, bit in ((1, 1, -1, pkv.PKV_ERR_PAGE_NEG), (2, 0, c.P, pkv.PKV_ERR_PAGE_RANGE),
                                   (4, 0, 2**31 - 1, pkv.PKV_ERR_PAGE_RANGE),
                                   (5, 1, -2**31, pkv.PKV_ERR_PAGE_NEG)):
            keep = c.t["table"].clone()
            c.t["table"][row, col] = val
            c.err.zero_()
            c.run()
            assert pkv.pkv_read_error_word(c.err) == bit, (ps, row, col)
            others = [b for b in range(5) if b != row - 1]
            assert torch.equal(c.out[others], good[others])
            c.t["table"].copy_(keep)
        c.err.zero_()
        c.run()
        assert torch.equal(c.out, good) and pkv.pkv_read_error_word(c.err) == 0
        for slot, bit in ((-1, pkv.PKV_ERR_SLOT), (6, pkv.PKV_ERR_SLOT)):
            c.t["bidx"][2] = slot
            c.err.zero_()
            c.run()
            assert pkv.pkv_read_error_word(c.err) == bit
            assert not c.out[2].any()
            c.t["bidx"][2] = 3
        for L, bit in ((c.max_pages * ps + 1, pkv.PKV_ERR_POS), (2**31 - 1, pkv.PKV_ERR_POS),
                       (-3, pkv.PKV_ERR_POS)):
            c.t["lens"][3] = L
            c.err.zero_()
            c.run()
            # a length past the table also reaches entries that hold no page
            assert pkv.pkv_read_error_word(c.err) & bit
            want, tol = c.expect(rows=[0, 1, 2, 4])
            got = c.out.cpu().double().numpy()
            assert (np.abs(got - want) <= tol)[[0, 1, 2, 4]].all()
            c.t["lens"][3] = 90
        c.err.zero_()
        c.run()
        assert torch.equal(c.out, good) and pkv.pkv_read_error_word(c.err) == 0


def test_repeated_and_captured_calls_give_the_same_bits(dev):
    """The workspace is left ready; replays follow the lengths; two graphs with
    workspaces of their own run side by side."""
    rng = np.random.default_rng(36)
    c = Case(rng, 6, 32, 8, 128, 64, 16, [900, 20, 3000, 1, 128, 700]).device(dev)
    first = c.run().clone()
    for _ in range(20):
        assert torch.equal(c.run(), first)
    d = Case(rng, 3, 8, 1, 512, 64, 64, [2000, 64, 333]).device(dev)
    first_d = d.run().clone()
    graphs = []
    for x in (c, d):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            x.run()
        graphs.append(g)
    s2 = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        graphs[0].replay()
        with torch.cuda.stream(s2):
            graphs[1].replay()
    torch.cuda.synchronize()
    assert torch.equal(c.out, first) and torch.equal(d.out, first_d)
    c.lens = np.array([100, 20, 2500, 1, 0, 64])
    c.t["lens"].copy_(torch.from_numpy(c.lens.astype(np.int32)))
    graphs[0].replay()
    torch.cuda.synchronize()
    c.check()


def test_agrees_with_the_bf16_cache(dev):
    """The same values held in bf16 (codes times powers of two are exact there)
    through paged_decode_attn: both within their own bounds of each other."""
    rng = np.random.default_rng(37)
    c = Case(rng, 8, 32, 8, 128, 64, 16, rng.integers(64, 1025, 8)).device(dev)
    c.run()
    kc, vc = (torch.from_numpy(oracle.dequantise(a, np.where(np.isnan(s), 0, s), c.G)).bfloat16()
              .to(dev) for a, s in zip(c.c, c.s))
    out = torch.empty_like(c.out)
    n = pkv.paged_decode_attn_workspace(8, 32, 128, pkv.paged_decode_attn_splits(
        8, 8, 128, c.max_pages, 64))
    pkv.paged_decode_attn(c.t["q"], kc, vc, c.t["table"], c.n_slots, c.max_pages, 64, c.P,
                          c.t["bidx"], c.t["lens"], 0, 128 ** -0.5, 0,
                          torch.zeros(n, dtype=torch.uint8, device=dev), out)
    _, tol = c.expect()
    # the bf16 cache's own: weights in bf16 (2^-8 A at most), output in bf16
    want, _ = c.expect()
    A = tol / 2.0 ** -11            # an upper bound of A
    e = np.abs(out.cpu().double().numpy() - c.out.cpu().double().numpy())
    assert (e <= tol + 2.0 ** -8 * (A + np.abs(want))).all()


def test_past_32_bit_offsets(dev):
    """Pages behind 2^32 bytes of each cache, and of the second head."""
    H, D, ps, G = 2, 512, 128, 64
    P = (5 << 30) // (ps * D) // 1
    rows = P * ps
    kc = torch.empty((H, rows, D), dtype=torch.uint8, device=dev).view(FP8)
    vc = torch.empty((H, rows, D), dtype=torch.uint8, device=dev).view(FP8)
    ks = torch.empty((H, rows // G), dtype=torch.float32, device=dev)
    vs = torch.empty((H, rows // G), dtype=torch.float32, device=dev)
    rng = np.random.default_rng(38)
    pages = [P - 1, 5, P - 7]
    L = 2 * ps + 40
    table = torch.tensor([[0] * 3, pages], dtype=torch.int32, device=dev)
    x, y = tokens(rng, L, H, D), tokens(rng, L, H, D)
    i32 = dict(dtype=torch.int32, device=dev)
    err = torch.zeros(1, **i32)
    pkv.kv_append_q8(x.to(dev), y.to(dev), torch.ones(L, **i32), torch.arange(L, **i32), table, 2,
                     3, ps, P, kc, vc, ks, vs, err)
    small = [np.zeros((H, 4 * ps, D)), np.zeros((H, 4 * ps // G)), np.zeros((H, 4 * ps, D)),
             np.zeros((H, 4 * ps // G))]
    near = np.array([[0, 0, 0], [1, 2, 3]], np.int32)
    for a, z in ((0, x), (2, y)):
        oracle.kv_append_q8(small[a], small[a + 1], z.double().numpy(), near, np.ones(L, int),
                            np.arange(L), ps, 4, G)
    for i, p in enumerate(pages):
        n = min(ps, L - i * ps)
        for t, a in ((kc, 0), (vc, 2)):
            assert np.array_equal(codes_f64(t[:, p * ps:p * ps + n]),
                                  small[a][:, (i + 1) * ps:(i + 1) * ps + n])
    q = wl.randn_bf16(rng, (1, 4, D)).to(dev)

    def attend(kc, vc, ks, vs, table, n_pages):
        out = torch.empty((1, 4, D), dtype=torch.bfloat16, device=dev)
        pkv.paged_decode_attn_q8(q, kc, vc, ks, vs, table, 2, 3, ps, n_pages, torch.ones(1, **i32),
                                 torch.full((1,), L, **i32), 0, D ** -0.5,
                                 workspace(4, H, D, dev), out, err)
        return out

    got = attend(kc, vc, ks, vs, table, P)
    want = attend(to_codes(small[0], dev), to_codes(small[2], dev),
                  *(torch.from_numpy(small[a].astype(np.float32)).to(dev) for a in (1, 3)),
                  torch.from_numpy(near).to(dev), 4)
    assert torch.equal(got, want) and pkv.pkv_read_error_word(err) == 0
