"""Calls of the 8-bit cache's operators that the header allows beyond the plain ones:
shared and reused workspaces, scales at any address, no error word, no batch index,
side streams, graphs in turn, every way the append divides its tokens. The same call
gives the same bits however it is made, so most tests compare bits; the others use the
bounds and the oracle of test_gpu_q8."""
import numpy as np
import pytest
import torch

import oracle
from test_gpu_q8 import Cache, Case, dev, slot_table, tokens, workspace  # noqa: F401

pytestmark = pytest.mark.gpu
pkv = pytest.importorskip("paged_kv_decode_pagetable_gb300")


def call(c, ws=None, window=0, out=None, **kw):
    t = {**c.t, **kw}
    out = torch.full_like(c.out, float("nan")) if out is None else out
    pkv.paged_decode_attn_q8(t["q"], t["kc"], t["vc"], t["ks"], t["vs"], t["table"], c.n_slots,
                             c.max_pages, c.ps, c.P, t["bidx"], t["lens"], window, c.D ** -0.5,
                             c.ws if ws is None else ws, out, kw.get("err"))
    return out


def test_one_workspace_serves_every_shape(dev):
    """Records of G * D words begin elsewhere for each shape: a call must leave all of
    them zero for the next."""
    rng = np.random.default_rng(50)
    cases = [Case(rng, B, Hq, Hkv, D, ps, G, lens).device(dev) for B, Hq, Hkv, D, ps, G, lens in
             ((1, 8, 1, 512, 64, 64, [5000]), (3, 4, 4, 64, 8, 1, [3000, 1, 70]),
              (2, 32, 8, 128, 64, 16, [2500, 1900]), (1, 3, 1, 256, 32, 8, [4000]))]
    want = [c.run().clone() for c in cases]
    for c in cases:
        c.check()
    ws = torch.zeros(max(c.ws.nbytes for c in cases), dtype=torch.uint8, device=dev)
    for i in rng.integers(0, len(cases), 40):
        assert torch.equal(call(cases[i], ws), want[i]), i
    assert not ws.any()


def test_two_graphs_share_a_workspace(dev):
    """Captured calls of two shapes on one workspace, replayed in turn on one stream."""
    rng = np.random.default_rng(51)
    a = Case(rng, 2, 16, 2, 128, 64, 16, [3000, 700]).device(dev)
    b = Case(rng, 1, 8, 1, 512, 64, 64, [4100]).device(dev)
    want = [a.run().clone(), b.run().clone()]
    ws = torch.zeros(max(a.ws.nbytes, b.ws.nbytes), dtype=torch.uint8, device=dev)
    graphs = []
    for c in (a, b):
        c.out.fill_(float("nan"))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(c, ws, out=c.out)
        graphs.append(g)
    for i in (0, 1, 1, 0, 0, 1, 0):
        graphs[i].replay()
        assert torch.equal((a, b)[i].out, want[i])
        (a, b)[i].out.zero_()
    assert not ws.any()


@pytest.mark.parametrize("D,ps,G", [(64, 64, 16), (128, 16, 4), (512, 64, 1)])
def test_scales_at_any_address(dev, D, ps, G):
    """Scales a multiple of 4, not 16 bytes into a buffer."""
    rng = np.random.default_rng(52)
    c = Case(rng, 3, 8, 2, D, ps, G, [300, 65, 1000]).device(dev)
    want = c.run().clone()
    c.check()
    for off in (1, 2, 3):
        moved = {}
        for n in ("ks", "vs"):
            buf = torch.full((c.t[n].numel() + 8,), float("nan"), device=dev)
            moved[n] = buf[off:off + c.t[n].numel()].view_as(c.t[n]).copy_(c.t[n])
        assert torch.equal(call(c, **moved), want), off


def test_no_batch_index_no_error_word(dev):
    """Row b is slot b, row 0 the padding slot; bad lengths and pages without a word."""
    rng = np.random.default_rng(53)
    c = Case(rng, 4, 8, 2, 128, 64, 16, [0, 500, 3, 64], slots=[0, 1, 2, 3]).device(dev)
    want = c.run().clone()
    c.check()
    assert torch.equal(call(c, bidx=None), want) and not want[0].any()
    lens = torch.tensor([9, 10 ** 9, -1, 64], dtype=torch.int32, device=dev)
    got = call(c, bidx=None, lens=lens)    # clamped to the table, none, none, as before
    assert not got[0].any() and not got[2].any() and torch.equal(got[3], want[3])


@pytest.mark.parametrize("window", [1, 2, 63, 64, 65, 10 ** 9, -5])
def test_windows(dev, window):
    rng = np.random.default_rng(54)
    c = Case(rng, 6, 8, 2, 64, 16, 8, [1, 64, 65, 128, 1000, 66]).device(dev)
    c.run(window)
    c.check(window)


@pytest.mark.parametrize("B,Hq,Hkv,D,ps,G", [(512, 16, 16, 64, 8, 1), (400, 40, 40, 128, 16, 16),
                                             (130, 64, 64, 256, 16, 2), (1, 35, 5, 512, 8, 8)])
def test_many_short_rows_and_heads(dev, B, Hq, Hkv, D, ps, G):
    """Many (row, head)s of a tile or two a CTA, in every one of its stages."""
    rng = np.random.default_rng(B)
    lens = rng.integers(1, 60, B)
    lens[rng.integers(0, B, B // 9)] = 0
    c = Case(rng, B, Hq, Hkv, D, ps, G, lens, slots=rng.permutation(np.arange(1, B + 1)))
    c.device(dev).run()
    c.check(rows=rng.choice(B, min(B, 40), replace=False))
    assert torch.isfinite(c.out).all()


def test_calls_side_by_side_on_two_streams(dev):
    """Eager calls on two streams, each with its own workspace and output, over the
    same cache."""
    rng = np.random.default_rng(55)
    c = Case(rng, 5, 32, 8, 128, 64, 16, [4000, 20, 900, 1, 2100]).device(dev)
    want = c.run().clone()
    streams = [torch.cuda.Stream() for _ in range(2)]
    ws = [workspace(32, 8, 128, dev) for _ in streams]
    outs = [torch.full((20,) + c.out.shape, float("nan"), dtype=torch.bfloat16, device=dev)
            for _ in streams]
    torch.cuda.synchronize()
    for i in range(20):
        for s, w, o in zip(streams, ws, outs):
            with torch.cuda.stream(s):
                call(c, w, out=o[i])
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(x, want) for x in o)


# ------------------------------------------------------------------ append ---

@pytest.mark.parametrize("H,D,ps,G,lens", [
    (1, 64, 8, 1, [6001, 2]), (1, 64, 16, 2, [7000]), (2, 128, 64, 16, [3001, 5, 800]),
    (2, 256, 16, 16, [2500, 1]), (1, 512, 64, 64, [6100]), (4, 48, 32, 32, [1500, 33]),
    (3, 64, 12, 4, [1999, 12])])
@pytest.mark.parametrize("prefill", [False, True])
def test_prompts_larger_than_the_gpu(dev, H, D, ps, G, lens, prefill):
    """More tokens than warps, so that windows and groups of lanes share them, padding
    on slot 0 behind the last prompt, infinities among the values."""
    rng = np.random.default_rng(H * D + G)
    n = len(lens)
    max_pages = max(-(-x // ps) for x in lens) + 1
    P = n * max_pages + 1
    c = Cache(rng, dev, H, D, ps, P, G)
    table = slot_table(rng, n, max_pages, P)
    slots = np.concatenate([np.repeat(np.arange(1, n + 1), lens), np.zeros(37, int)])
    pos = np.concatenate([np.arange(x) for x in lens] + [np.zeros(37, int)])
    k, v = (tokens(rng, len(pos), H, D) for _ in range(2))
    k[rng.integers(0, len(pos), 50), 0, 3] = float("inf")
    v[rng.integers(0, len(pos), 50), H - 1, 0] = float("-inf")
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    assert c.append(k, v, table, slots, pos, err, prefill) == 0
    c.check()
    assert pkv.pkv_read_error_word(err) == 0


def test_a_step_of_more_rows_than_warps(dev):
    rng = np.random.default_rng(60)
    H, D, ps, G, n = 8, 64, 16, 16, 900
    c = Cache(rng, dev, H, D, ps, 2 * n + 1, G)
    table = slot_table(rng, n, 2, 2 * n + 1)
    at = rng.integers(0, 31, n)
    for step in range(2):
        order = rng.permutation(n)
        assert c.append(tokens(rng, n, H, D), tokens(rng, n, H, D), table, order + 1,
                        (at + step)[order]) == 0
        c.check()


def test_append_on_a_side_stream_without_batch_index(dev):
    """Token i on slot i (slot 0 is skipped), on another stream, no error word."""
    rng = np.random.default_rng(61)
    H, D, ps, G, n = 2, 128, 16, 8, 5
    c = Cache(rng, dev, H, D, ps, n + 2, G)
    table = slot_table(rng, n, 1, n + 2)
    k, v = tokens(rng, n + 1, H, D), tokens(rng, n + 1, H, D)
    s = torch.cuda.Stream()
    dk, dv = k.to(dev), v.to(dev)
    t = torch.from_numpy(table).to(dev)
    pos = torch.zeros(n + 1, dtype=torch.int32, device=dev)
    torch.cuda.synchronize()
    pkv.kv_append_q8(dk, dv, None, pos, t, n + 1, 1, ps, c.P, c.kc, c.vc, c.ks, c.vs, None, s)
    for x, (codes, scale) in zip((k, v), c.np):
        oracle.kv_append_q8(codes, scale, x.double().numpy(), table, np.arange(n + 1),
                            np.zeros(n + 1, int), ps, c.P, G)
    s.synchronize()
    c.check()


def test_ones_own_key_alone_is_its_value(dev):
    """One key a row: the output is that key's value, rounded once to bf16."""
    rng = np.random.default_rng(62)
    for D in (64, 128, 256, 512):
        c = Case(rng, 3, 4, 2, D, 8, 1, [1, 1, 1]).device(dev)
        got = c.run().cpu().double().numpy()
        for b in range(3):
            r = c.table[c.slots[b], 0] * 8
            want = np.repeat(c.c[1][:, r] * c.s[1][:, r][:, None], 2, 0)
            assert np.array_equal(got[b], want), (D, b)


@pytest.mark.parametrize("D", [64, 128, 256, 512])
def test_full_rings_are_read_before_they_are_refilled(dev, D):
    """Long rows keep every ring entry in use; a tile read after its entry was refilled
    shows as calls that differ (at D = 256, one in ten)."""
    rng = np.random.default_rng(63)
    c = Case(rng, 3, 24, 3, D, 64, 2, [29952, 28480, 29803]).device(dev)
    outs = torch.full((200,) + c.out.shape, float("nan"), dtype=torch.bfloat16, device=dev)
    for o in outs:
        call(c, out=o)
    assert torch.isfinite(outs).all()
    assert all(torch.equal(o, outs[0]) for o in outs[1:])
    c.out = outs[0]
    c.check(rows=[1])


def test_calls_beside_a_busy_stream(dev):
    """Other work holds SMs, so that not all CTAs of a call are resident at once: parts
    wait for ones that start later, and all finish."""
    rng = np.random.default_rng(64)
    cases = [Case(rng, 1, 32, 8, 128, 64, 16, [30000]).device(dev),
             Case(rng, 9, 8, 1, 512, 64, 64, rng.integers(500, 9000, 9)).device(dev)]
    want = [c.run().clone() for c in cases]
    a = torch.randn((4096, 4096), dtype=torch.bfloat16, device=dev)
    other, b = torch.cuda.Stream(), torch.empty_like(a)
    torch.cuda.synchronize()
    with torch.cuda.stream(other):
        for _ in range(200):
            torch.mm(a, a, out=b)
    outs = [[call(c) for _ in range(100)] for c in cases]
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert all(torch.equal(x, w) for x in o)
    assert all(not c.ws.any() for c in cases)
