"""Append, verification and move of drafted trees against the 64-bit oracle, and whole
speculative steps."""
import numpy as np
import pytest
import torch

import workloads as wl
from gpu_util import f64
from oracle import tree
from tree_util import BF16_STEP, TreeCase, random_tree

pytestmark = pytest.mark.gpu
pkv = pytest.importorskip("paged_kv_decode_pagetable_gb300")
EPS = 1e-6


def cuda(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x)) if not isinstance(x, torch.Tensor) else x
    return t.to("cuda", dtype) if dtype else t.cuda()


# ---------------------------------------------------------------- append ----

def append_case(rng, Hq, Hkv, D, ps, ctx, trees, strided=True, gains=True, k_eq_v=False, **kw):
    c = TreeCase(rng, Hq, Hkv, D, ps, ctx, trees, **kw)
    c.kc[:], c.vc[:] = 0, 0
    n = c.N + c.pad
    c.qkv = wl.randn_bf16(rng, (n, (Hq + 2 * Hkv) * D + (8 if strided else 0)))
    c.g = [(1 + 0.1 * torch.from_numpy(rng.standard_normal(D))).bfloat16() if gains else None
           for _ in range(2)]
    c.k_eq_v = k_eq_v
    return c


def parts(c, qkv):
    at, out = 0, []
    for h in (c.Hq, c.Hkv, c.Hkv):
        out.append(qkv[:, at:at + h * c.D].unflatten(1, (h, c.D)))
        at += h * c.D
    q, k, v = out
    return q, k, None if c.k_eq_v else v


def run_append(c, theta=1e4, rotary=None, v_norm=False, err_ok=False, contiguous=False):
    c.device(pkv)
    c.t["kc"].zero_(), c.t["vc"].zero_()
    q, k, v = parts(c, c.qkv.cuda())
    if contiguous:
        q, k, v = (x if x is None else x.contiguous() for x in (q, k, v))
    g = [None if x is None else x.cuda() for x in c.g]
    qo = torch.full((c.N + c.pad, c.Hq, c.D), 7.0, dtype=torch.bfloat16, device="cuda")
    pkv.tree_qkv_norm_rope_append(
        q, k, v, g[0], g[1], c.t["slots"], c.t["ctx"], c.t["row_start"], c.t["parents"], theta, EPS,
        rotary, v_norm, c.t["table"], c.n_slots, c.max_pages, c.ps, c.P, c.t["kc"], c.t["vc"], qo,
        c.err)
    torch.cuda.synchronize()
    if not err_ok:
        assert int(c.err) == 0
    return qo


def check_append(c, qo, theta=1e4, rotary=None, v_norm=False):
    """One rounding to bf16; in fp32 a norm's factor is off by less than D/32 + 8 roundings
    of 2^-24, a rotation factor by its angle, 2^-24 of a half turn, and 2 ulp."""
    q, k, v = (None if x is None else x.double().numpy() for x in parts(c, c.qkv))
    g = [None if x is None else x.double().numpy() for x in c.g]
    kc, vc = np.zeros(c.kc.shape), np.zeros(c.vc.shape)
    want = tree.tree_append(q, k, v, g[0], g[1], c.slots, c.ctx, c.row_start, c.parents, theta, EPS,
                            rotary, v_norm, c.table, c.ps, kc, vc)
    rel = 2.0 ** -24 * (c.D / 32 + 16) + np.pi * 2.0 ** -24

    def near(got, ref):
        half = c.D // 2
        size = np.hypot(ref[..., :half], ref[..., half:])
        size = np.concatenate([size, size], -1)     # the pair's length: what an angle moves
        bound = BF16_STEP * np.abs(ref) + 2 * rel * size * (1 + BF16_STEP) + 1e-30
        assert (np.abs(got - ref) <= bound).all(), float((np.abs(got - ref) / bound).max())

    near(f64(qo)[:c.N], want[:c.N])
    assert (f64(qo)[c.N:] == 7).all()
    near(f64(c.t["kc"]), kc)
    if v_norm:
        near(f64(c.t["vc"]), vc)
    else:
        assert np.array_equal(f64(c.t["vc"]), vc)


@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 1), (8, 8), (32, 8), (40, 5)])
def test_append(D, Hq, Hkv):
    rng = np.random.default_rng([21, D, Hq])
    c = append_case(rng, Hq, Hkv, D, 16, [0, 31, 4000],
                    [random_tree(rng, n, 3) for n in (7, 1, 20)])
    check_append(c, run_append(c))


@pytest.mark.parametrize("rotary,v_norm,k_eq_v,gains", [
    (0, False, False, True), (32, True, False, True), (128, True, True, True),
    (None, False, True, False), (2, False, False, False)])
def test_append_options(rotary, v_norm, k_eq_v, gains):
    rng = np.random.default_rng([22, rotary or 1])
    c = append_case(rng, 8, 2, 128, 8, [5, 700], [random_tree(rng, 9, 2)] * 2, gains=gains,
                    k_eq_v=k_eq_v, pad=3)
    check_append(c, run_append(c, 1e6, rotary, v_norm), 1e6, rotary, v_norm)


@pytest.mark.parametrize("theta", [0.5, 1.0, 1e4, 5e5, 1e9])
def test_far_positions(theta):
    """Angles stay exact at positions of millions: only the table's width bounds them."""
    rng = np.random.default_rng(23)
    c = append_case(rng, 2, 1, 64, 1024, [3], [random_tree(rng, 8, 2)])
    far = 4_000_000 // 1024
    c.table = np.concatenate([np.full((2, far), -1, np.int32), c.table[:, :1]], 1)
    c.table[0] = 0
    c.max_pages, c.ctx = far + 1, c.ctx + far * 1024
    check_append(c, run_append(c, theta), theta)


def test_append_of_contiguous_and_strided_tokens_and_in_place():
    rng = np.random.default_rng(24)
    c = append_case(rng, 4, 2, 128, 16, [10, 90], [random_tree(rng, 6, 2)] * 2)
    want = run_append(c).clone()
    kc, vc = c.t["kc"].clone(), c.t["vc"].clone()
    assert torch.equal(run_append(c, contiguous=True), want)
    assert torch.equal(c.t["kc"], kc) and torch.equal(c.t["vc"], vc)
    q, k, v = (x.contiguous() for x in parts(c, c.qkv.cuda()))
    pkv.tree_qkv_norm_rope_append(
        q, k, v, c.g[0].cuda(), c.g[1].cuda(), c.t["slots"], c.t["ctx"], c.t["row_start"],
        c.t["parents"], 1e4, EPS, None, False, c.t["table"], c.n_slots, c.max_pages, c.ps, c.P,
        c.t["kc"], c.t["vc"], q)
    assert torch.equal(q, want) and torch.equal(c.t["kc"], kc)


def test_append_faults_are_reported_and_skipped():
    rng = np.random.default_rng(25)
    trees = [random_tree(rng, 4, 2) for _ in range(4)]
    for what, bit in (("slot", pkv.PKV_ERR_SLOT), ("ctx", pkv.PKV_ERR_POS),
                      ("page", pkv.PKV_ERR_PAGE_NEG), ("page2", pkv.PKV_ERR_PAGE_RANGE),
                      ("start", pkv.PKV_ERR_TREE)):
        c = append_case(rng, 4, 2, 64, 16, [4, 5, 6, 7], trees)
        good = run_append(c).clone()
        kc = c.t["kc"].clone()
        if what == "slot":
            c.slots[2] = -1
        elif what == "ctx":
            c.ctx[2] = c.max_pages * 16 - 3
        elif what == "page":
            c.table[3, 0] = -1
        elif what == "page2":
            c.table[3, 0] = c.P
        else:
            c.row_start[4] = 100       # past the packed nodes
        got = run_append(c, err_ok=True)
        assert int(c.err) == bit, what
        row = 3 if what == "start" else 2
        rest = [n for n in range(16) if n // 4 != row]
        assert torch.equal(got[rest], good[rest])
        mine = [tree.cache_row(np.where(c.table < 0, 0, c.table) % c.P, b + 1, 4 + b + i, 16)
                for b in range(4) if b != row for i in range(4)]
        assert torch.equal(c.t["kc"][:, mine], kc[:, mine])


# ---------------------------------------------------------------- verify ----

def softmax_rows(rng, N, V, size=3.0):
    x = size * rng.standard_normal((N, V))
    x[np.arange(N), rng.integers(0, V, N)] += np.log(V) + size * size / 2
    x = np.exp(x - x.max(1, keepdims=True))
    return (x / x.sum(1, keepdims=True)).astype(np.float32)


def verify(p, q, tokens, row_start, parents, u, up, cols=64, err=None):
    B = len(row_start) - 1
    acc = torch.full((B,), -9, dtype=torch.int32, device="cuda")
    path = torch.full((B, cols), -9, dtype=torch.int32, device="cuda")
    nxt = torch.full((B,), -9, dtype=torch.int32, device="cuda")
    i32 = lambda x: cuda(np.asarray(x, np.int32))  # noqa: E731
    p, q = (x if x is None or isinstance(x, torch.Tensor) else cuda(x) for x in (p, q))
    pkv.tree_verify(p, q, i32(tokens), i32(row_start), i32(parents),
                    cuda(np.asarray(u, np.float32)), cuda(np.asarray(up, np.float32)), acc, path,
                    nxt, err)
    torch.cuda.synchronize()
    return acc.tolist(), path.tolist(), nxt.tolist()


def verify_case(rng, B, nodes, width, V, sampled):
    trees = [random_tree(rng, int(rng.integers(1, nodes + 1)), width) for _ in range(B)]
    start = np.concatenate([[0], np.cumsum([len(t) for t in trees])])
    N = int(start[-1])
    p = softmax_rows(rng, N, V)
    noisy = p.astype(np.float64) * np.exp(0.7 * rng.standard_normal((N, V)))
    q = (noisy / noisy.sum(1, keepdims=True)).astype(np.float32)
    parents = np.array([x for t in trees for x in t])
    base = np.repeat(start[:-1], np.diff(start))
    tokens = np.zeros(N, int)
    for n in range(N):
        if parents[n] >= 0:
            d = q[base[n] + parents[n]].astype(np.float64)
            rank = sum(parents[m] == parents[n] for m in range(base[n], n))
            tokens[n] = (rng.choice(V, p=d / d.sum()) if sampled
                         else np.argsort(-d)[min(rank, V - 1)])
    u = rng.random(N).astype(np.float32)
    return p, q if sampled else None, tokens, start, parents, u, rng.random(B).astype(np.float32)


@pytest.mark.parametrize("sampled", [True, False])
@pytest.mark.parametrize("width", [1, 3, 8])
@pytest.mark.parametrize("B,nodes,V", [(1, 4, 1), (3, 5, 2), (5, 64, 37), (2, 33, 128),
                                       (70, 12, 1001), (200, 6, 515), (3, 20, 32003),
                                       (1, 9, 100000)])
def test_verify(B, nodes, V, width, sampled):
    rng = np.random.default_rng([31, B, V, width, sampled])
    case = verify_case(rng, B, nodes, width, V, sampled)
    want = tree.tree_verify(*case, path_cols=64)
    got = verify(*case)
    assert got[0] == want[0].tolist() and got[1] == want[1].tolist()
    assert got[2] == want[2].tolist()


def exact_rows(rng, N, V):
    """Probabilities in whole units of 2^-20 that sum to 1: every sum is exact anywhere."""
    w = rng.multinomial(1 << 20, np.full(V, 1 / V), N)
    return (w / (1 << 20)).astype(np.float32)


@pytest.mark.parametrize("V", [1, 5, 128, 129, 4099, 70001])
def test_picks_on_the_borders(V):
    """u_pick on the very borders between tokens: the token whose share begins there."""
    rng = np.random.default_rng([32, V])
    B = 200
    p = exact_rows(rng, B, V)
    c = np.cumsum(p.astype(np.float64), 1)
    at = rng.integers(0, V, B)
    up = np.minimum([c[b, at[b] - 1] if at[b] else 0.0 for b in range(B)], 1 - 2.0 ** -24)
    want = [int(np.argmax(c[b] > up[b])) for b in range(B)]
    got = verify(p, None, np.zeros(B), np.arange(B + 1), np.full(B, -1), np.zeros(B), up)
    assert got[2] == want and got[0] == [0] * B


def test_tests_on_their_borders():
    """u q S equal to w refuses; the next fp32 number below accepts."""
    p = np.array([[0.25, 0.75], [0.5, 0.5]], np.float32)
    q = np.array([[0.5, 0.5], [0.5, 0.5]], np.float32)
    for u, good in ((0.5, 0), (np.nextafter(np.float32(0.5), np.float32(0)), 1), (0.0, 1)):
        assert verify(p, q, [0, 0], [0, 2], [-1, 0], [0, u], [0.5])[0] == [good]
        assert verify(p, None, [0, 0], [0, 2], [-1, 0], [0, u / 2], [0.5])[0] == [good]
    # a token that the target cannot say is refused even by u = 0
    p[0] = [0, 1]
    assert verify(p, q, [0, 0], [0, 2], [-1, 0], [0, 0.0], [0.5])[0] == [0]


def test_siblings_with_one_token():
    """The same token twice among certain drafts: the second is refused; among samples it is
    tried against what is left."""
    rng = np.random.default_rng(33)
    p, q = softmax_rows(rng, 4, 50), softmax_rows(rng, 4, 50)
    tokens = [0, 7, 7, 7]
    for u in np.linspace(0, 0.999, 23):
        case = ([0, 4], [-1, 0, 0, 0], [0, u, u / 2, u / 3], [u])
        for d in (None, q):
            want = tree.tree_verify(p, d, tokens, *case, path_cols=64)
            got = verify(p, d, tokens, *case)
            assert [list(x) for x in got] == [x.tolist() for x in want]


def test_nothing_left_falls_back_on_the_target():
    p = np.array([[0.5, 0.5, 0, 0], [1, 0, 0, 0]], np.float32)
    q = np.array([[0.5, 0.5, 0, 0], [1, 0, 0, 0]], np.float32)
    # p = q is always accepted for u < 1; u of 1 and more is refused and leaves nothing
    assert verify(p, q, [0, 1], [0, 2], [-1, 0], [0, 1.0], [0.75]) == ([0], [[0] + [-1] * 63], [1])


def test_probabilities_out_of_order():
    nan = float("nan")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    p = np.array([[nan, -1, 0.5, 0.5], [0] * 4, [nan] * 4], np.float32)
    got = verify(p, None, [0, 0, 0], [0, 1, 2, 3], [-1] * 3, [0] * 3, [0.0, 0.5, 0.5], err=err)
    assert got[2] == [2, -1, -1] and int(err) == pkv.PKV_ERR_PROB
    err.zero_()
    p = np.full((2, 4), 0.25, np.float32)
    got = verify(p, None, [0, 4], [0, 2], [-1, 0], [0, 0], [0.9], err=err)
    assert got[0] == [0] and got[2] == [3] and int(err) == pkv.PKV_ERR_PROB


def test_verify_rows_that_are_empty_or_wrong():
    rng = np.random.default_rng(34)
    p = softmax_rows(rng, 10, 99)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    parents = [-1, 0, 1, -1, 0, 0, -1, 0, 1, 2]
    case = (p, None, rng.integers(0, 99, 10), [0, 3, 3, 6, 10], parents, rng.random(10) * 0.02,
            rng.random(4))
    want = tree.tree_verify(*case, path_cols=5)
    got = verify(*case, cols=5, err=err)
    assert [list(x) for x in got] == [x.tolist() for x in want] and int(err) == 0
    got3 = verify(*case, cols=3, err=err)      # the last row's four nodes have no room
    assert int(err) == pkv.PKV_ERR_TREE
    assert got3[0][:3] == got[0][:3] and got3[2] == got[2][:3] + [-1] and got3[0][3] == 0
    err.zero_()
    bad = list(case)
    bad[3] = [0, 3, 2, 6, 11]
    got = verify(*bad, err=err)
    assert int(err) == pkv.PKV_ERR_TREE and got[2][1] == -1 and got[2][3] == -1
    assert got[2][0] == want[2][0]


@pytest.mark.parametrize("offset", [0, 1, 2, 3])
def test_verify_strided_and_unaligned_rows(offset):
    rng = np.random.default_rng([35, offset])
    case = list(verify_case(rng, 6, 9, 3, 1003, True))
    want = verify(*case)
    for k, (extra, off) in enumerate(((5, offset), (2, 3 - offset))):
        x = torch.full((case[k].shape[0], 1003 + extra), float("nan"), device="cuda")
        x[:, off if off <= extra else 0:][:, :1003] = cuda(case[k])
        case[k] = x[:, off if off <= extra else 0:][:, :1003]
    assert verify(*case) == want


def test_verify_is_the_same_however_rows_are_shared():
    """A row's result does not depend on how many CTAs share it (set by the batch)."""
    rng = np.random.default_rng(36)
    one = verify_case(rng, 1, 16, 4, 20011, True)
    alone = verify(*one)
    n = len(one[2])
    for copies in (2, 40, 80, 160, 400):
        p, q = (cuda(x).repeat(copies, 1) for x in one[:2])
        start = np.arange(copies + 1) * n
        got = verify(p, q, np.tile(one[2], copies), start, np.tile(one[4], copies),
                     np.tile(one[5], copies), np.tile(one[6], copies))
        assert got == tuple(x * copies for x in alone)


# ------------------------------------------------------------------ keep ----

@pytest.mark.parametrize("shape,dtype", [((128,), torch.bfloat16), ((64,), torch.float32),
                                         ((512,), torch.uint8), ((), torch.float32),
                                         ((3,), torch.uint8), ((5,), torch.bfloat16)])
@pytest.mark.parametrize("ps", [8, 64])
def test_keep_path(shape, dtype, ps):
    rng = np.random.default_rng([41, ps])
    trees = [random_tree(rng, n, w)
             for n, w in ((9, 3), (64, 5), (20, 1), (1, 1), (40, 8), (12, 4))]
    c = TreeCase(rng, 1, 1, 64, ps, [0, 100, 7, 64, 33, 5], trees,
                 slots=[3, 1, 2, 6, 4, 0]).device(pkv)
    path = np.full((6, 64), -1)
    acc = np.zeros(6, int)
    for b, t in enumerate(trees):
        leaf = int(np.argmax(tree.depths(t)))
        way = np.flatnonzero(tree.ancestors(t)[leaf])
        path[b, :len(way)] = way
        acc[b] = len(way) - 1
    caches = [torch.from_numpy(rng.integers(0, 255, (h, c.P * ps) + shape + (
        (torch.empty(0, dtype=dtype).element_size(),)), dtype=np.uint8)) for h in (1, 3, 2)]
    want = [x.numpy().copy() for x in caches]
    for w in want:
        tree.keep_path(w, c.table, c.slots, c.ctx, acc, path, ps)
    dev = [x.cuda().view(dtype).reshape(x.shape[:-1]) for x in caches]
    pkv.kv_keep_path(dev, c.t["table"], c.n_slots, c.max_pages, ps, c.P, c.t["slots"], c.t["ctx"],
                     cuda(acc, torch.int32), cuda(path, torch.int32), c.err)
    torch.cuda.synchronize()
    assert int(c.err) == 0
    for d, w in zip(dev, want):
        assert np.array_equal(d.cpu().contiguous().view(torch.uint8).numpy().reshape(w.shape), w)


def test_keep_path_of_many_caches_and_unaligned_ones():
    rng = np.random.default_rng(42)
    c = TreeCase(rng, 1, 1, 64, 16, [20, 3], [random_tree(rng, 12, 3)] * 2).device(pkv)
    path, acc = np.array([[0, 3, 5, 9, 11], [0, 2, 3, -1, -1]]), np.array([4, 2])
    base = torch.randint(0, 100, (150, 2 * c.P * 16 * 24 + 8), dtype=torch.uint8, device="cuda")
    caches = [base[i, i % 8:i % 8 + 2 * c.P * 16 * 24].view(2, c.P * 16, 24) for i in range(150)]
    want = base.cpu().numpy().copy()
    for i in range(150):
        tree.keep_path(want[i, i % 8:i % 8 + 2 * c.P * 16 * 24].reshape(2, c.P * 16, 24), c.table,
                       c.slots, c.ctx, acc, path, 16)
    pkv.kv_keep_path(caches, c.t["table"], c.n_slots, c.max_pages, 16, c.P, c.t["slots"],
                     c.t["ctx"], cuda(acc, torch.int32), cuda(path, torch.int32), c.err)
    assert int(c.err) == 0 and np.array_equal(base.cpu().numpy(), want)


@pytest.mark.parametrize("what,bit", [("order", pkv.PKV_ERR_TREE), ("count", pkv.PKV_ERR_TREE),
                                      ("low", pkv.PKV_ERR_TREE), ("slot", pkv.PKV_ERR_SLOT),
                                      ("ctx", pkv.PKV_ERR_POS), ("page", pkv.PKV_ERR_PAGE_NEG),
                                      ("range", pkv.PKV_ERR_PAGE_RANGE)])
def test_keep_path_leaves_faulty_rows_alone(what, bit):
    rng = np.random.default_rng(43)
    c = TreeCase(rng, 1, 1, 64, 8, [20, 30], [random_tree(rng, 12, 3)] * 2).device(pkv)
    path = np.array([[0, 3, 5, 9, 11], [0, 2, 3, 7, -1]])
    acc = np.array([4, 3])
    want = f64(c.t["kc"].nan_to_num_()).copy()
    tree.keep_path(want, c.table, c.slots, c.ctx, [4, 0], path, 8)
    if what == "order":
        path[1, 2] = 2
    elif what == "count":
        acc[1] = 5
    elif what == "low":
        path[1, :4] = [0, 1, 1, 1]
    elif what == "slot":
        c.t["slots"][1] = 3
    elif what == "ctx":
        c.t["ctx"][1] = c.max_pages * 8 - 6
    else:
        c.t["table"][2, 37 // 8] = -1 if what == "page" else c.P
    pkv.kv_keep_path([c.t["kc"]], c.t["table"], c.n_slots, c.max_pages, 8, c.P, c.t["slots"],
                     c.t["ctx"], cuda(acc, torch.int32), cuda(path, torch.int32), c.err)
    assert int(c.err) == bit
    assert np.array_equal(f64(c.t["kc"]), want)


# ------------------------------------------------------------ whole steps ----

def test_speculative_steps_against_single_ones():
    """Steps of the engine over trees, accepted as they come, leave the context that decode
    steps of the accepted tokens alone leave, and attend alike."""
    from paged_kv_decode_pagetable_gb300 import engine
    rng = np.random.default_rng(51)
    B, Hq, Hkv, D, ps, V, steps = 3, 8, 2, 64, 16, 40, 6
    spec = engine.LayerSpec(head_dim=D, theta=1e4, qk_norm=True)
    tokens = [int(x) for x in rng.integers(0, V, B)]      # the last committed ones
    emb = [wl.randn_bf16(rng, (V, h * D)).cuda() for h in (Hq, Hkv, Hkv)]
    gains = [(1 + 0.1 * torch.from_numpy(rng.standard_normal(D))).bfloat16().cuda()
             for _ in range(2)]
    pt, pt1 = (pkv.PageTable(B, ps, 80, 12, device="cuda") for _ in range(2))
    caches = [engine.alloc_cache(Hkv, 80, ps, D, "cuda") for _ in range(2)]
    slots = [pt.assign(1) for _ in range(B)]
    assert slots == [pt1.assign(1) for _ in range(B)]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    err = i32([0])
    ws = engine.TreeWorkspace(Hq, Hkv, D, "cuda")
    ws1 = engine.AttnWorkspace(B, Hq, Hkv, D, 12, ps, 0, "cuda")
    ctx = [0] * B
    for step in range(steps):
        trees = [random_tree(rng, int(rng.integers(1, 10)), 3) for _ in range(B)]
        start = np.concatenate([[0], np.cumsum([len(t) for t in trees])]).tolist()
        N = start[-1]
        tok = rng.integers(0, V, N)
        tok[start[:-1]] = tokens
        for b in range(B):
            pt.reserve(slots[b], ctx[b] + len(trees[b]))
        parents, rs, cl, bi = i32([p for t in trees for p in t]), i32(start), i32(ctx), i32(slots)
        qkv = [e[cuda(tok)].view(N, -1, D) for e in emb]
        qo, out = torch.empty_like(qkv[0]), torch.empty_like(qkv[0])
        engine.tree_layer_step(spec, pt, *caches[0], *qkv, bi, cl, rs, parents, qo, out, ws, *gains,
                               err=err)
        target = torch.softmax(
            torch.from_numpy(rng.standard_normal((N, V))).float() * 0.5, 1).cuda()
        # drafts that the target likes, so that some are accepted
        for n in range(N):
            row = max(b for b in range(B) if start[b] <= n)
            if trees[row][n - start[row]] >= 0:
                target[start[row] + trees[row][n - start[row]], tok[n]] += 1.0
        target /= target.sum(1, keepdim=True)
        acc, nxt = i32([0] * B), i32([0] * B)
        path = torch.zeros((B, 10), dtype=torch.int32, device="cuda")
        engine.accept_drafts(pt, list(caches[0]), target, None, cuda(tok, torch.int32), bi, cl, rs,
                             parents, torch.rand(N, device="cuda"), torch.rand(B, device="cuda"),
                             acc, path, nxt, err)
        assert int(err) == 0
        acc, path, nxt = acc.tolist(), path.tolist(), nxt.tolist()
        # the same tokens one by one
        for t in range(max(acc) + 1):
            rows = [b for b in range(B) if t <= acc[b]]
            nodes = [start[b] + path[b][t] for b in rows]
            pos = [ctx[b] + t for b in rows]
            for b in rows:
                pt1.reserve(slots[b], ctx[b] + t + 1)
            o1 = torch.empty((len(rows), Hq, D), dtype=torch.bfloat16, device="cuda")
            engine.decode_layer_step(spec, pt1, *caches[1], *[x[nodes] for x in qkv],
                                     i32([slots[b] for b in rows]), i32(pos),
                                     i32([p + 1 for p in pos]), o1, ws1, *gains, err=err)
            assert int(err) == 0
            # both round their weights and results to bf16 once, values are below 5
            assert (o1 - out[nodes]).abs().max() <= 4 * BF16_STEP * 5
        for b in range(B):
            ctx[b] += acc[b] + 1
            pt.truncate(slots[b], ctx[b])
            tokens[b] = nxt[b]
        for b in range(B):
            r = [[tree.cache_row(x.host_table().tolist(), slots[b], j, ps) for j in range(ctx[b])]
                 for x in (pt, pt1)]
            assert torch.equal(caches[0][1][:, r[0]], caches[1][1][:, r[1]])
            k = [f64(caches[i][0][:, r[i]]) for i in range(2)]
            assert np.abs(k[0] - k[1]).max() <= 2 * BF16_STEP * np.abs(k[0]).max()
    assert sum(ctx) > B * steps      # some drafts were accepted


def test_a_captured_step_serves_other_trees():
    from paged_kv_decode_pagetable_gb300 import engine
    rng = np.random.default_rng(52)
    spec = engine.LayerSpec(head_dim=128, theta=1e6)
    c = append_case(rng, 8, 2, 128, 16, [300, 40, 7], [random_tree(rng, n, 3) for n in (9, 12, 4)],
                    gains=False, pad=5).device(pkv)
    c.t["kc"].nan_to_num_(), c.t["vc"].nan_to_num_()
    pt = pkv.PageTable(3, 16, c.P, c.max_pages)       # geometry only
    q, k, v = parts(c, c.qkv.cuda())
    qo = torch.zeros((c.N + 5, 8, 128), dtype=torch.bfloat16, device="cuda")
    ws = engine.TreeWorkspace(8, 2, 128, "cuda")
    target = cuda(softmax_rows(rng, c.N + 5, 77))
    tok = cuda(rng.integers(0, 77, c.N + 5), torch.int32)
    u, up = torch.rand(c.N + 5, device="cuda"), torch.rand(3, device="cuda")
    acc, nxt = (torch.zeros(3, dtype=torch.int32, device="cuda") for _ in range(2))
    path = torch.zeros((3, 16), dtype=torch.int32, device="cuda")

    def step():
        engine.tree_layer_step(spec, pt, c.t["kc"], c.t["vc"], q, k, v, c.t["slots"], c.t["ctx"],
                               c.t["row_start"], c.t["parents"], qo, c.out, ws, err=c.err,
                               table=c.t["table"])
        engine.accept_drafts(pt, [c.t["kc"], c.t["vc"]], target, None, tok, c.t["slots"],
                             c.t["ctx"], c.t["row_start"], c.t["parents"], u, up, acc, path, nxt,
                             c.err, table=c.t["table"])

    saved = [x.clone() for x in (c.t["kc"], c.t["vc"])]
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for ns in ((9, 12, 4), (1, 0, 3), (10, 10, 5)):
        c.t["row_start"].copy_(cuda(np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)))
        c.t["parents"].zero_()
        c.t["parents"][:sum(ns)] = cuda(np.array(
            [p for n in ns for p in random_tree(rng, n, 3)], np.int32))
        results = []
        for run in (step, g.replay):
            c.t["kc"].copy_(saved[0]), c.t["vc"].copy_(saved[1])
            c.out.fill_(7), qo.fill_(7), u.fill_(0.02)
            run()
            torch.cuda.synchronize()
            assert int(c.err) == 0
            results.append([x.clone() for x in (qo, c.out, c.t["kc"], c.t["vc"], acc, path, nxt)])
        for a, b in zip(*results):
            assert torch.equal(a, b)
        assert (c.out[sum(ns):] == 7).all()
