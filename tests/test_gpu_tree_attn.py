"""paged_tree_attn against the 64-bit oracle, at the sizes, masks and orders where it can go
wrong."""
import numpy as np
import pytest
import torch

from gpu_util import NAN_BF16, f64
from oracle import tree
from tree_util import TreeCase, check_attn, random_tree

pytestmark = pytest.mark.gpu
pkv = pytest.importorskip("paged_kv_decode_pagetable_gb300")


def rng_of(*seed):
    return np.random.default_rng([abs(int(x)) for x in seed])


@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("G", [1, 2, 3, 5, 7, 8])
@pytest.mark.parametrize("width", [1, 4])
def test_heads(D, G, width):
    rng = rng_of(1, D, G, width)
    trees = [random_tree(rng, n, width) for n in (5, 1, 17)]
    TreeCase(rng, 2 * G, 2, D, 16, [70, 300, 3], trees).device(pkv).check(pkv)


@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("nodes", [1, 2, 3, 8, 15, 16, 17, 31, 32, 33, 63, 64])
def test_nodes(D, nodes):
    rng = rng_of(2, D, nodes)
    trees = [random_tree(rng, nodes, w) for w in (1, 3)]
    TreeCase(rng, 8, 1, D, 32, [129, 40], trees).device(pkv).check(pkv)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 6, 7, 8])
@pytest.mark.parametrize("window", [0, 40])
def test_more_columns_than_64(D, G, window):
    """Rows of many nodes take units of 128 columns (of 64 at D = 256); heads of a node may fall
    to both halves, rows of few nodes stand beside them."""
    rng = rng_of(20, D, G, window)
    ns = (64, 64, 61) if G <= 2 else (64, 30, 1, 41)
    trees = [random_tree(rng, n, w) for n, w in zip(ns, (4, 1, 8, 2))]
    c = TreeCase(rng, G, 1, D, 16, [300, 5, 131, 0][:len(ns)], trees, window=window)
    c.device(pkv).check(pkv)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_many_and_long_rows_of_many_nodes(D):
    rng = rng_of(21, D)
    trees = [random_tree(rng, int(rng.integers(15, 40)), 3) for _ in range(60)]
    TreeCase(rng, 8, 1, D, 32, rng.integers(0, 900, 60), trees).device(pkv).check(pkv)
    trees = [random_tree(rng, 20, 3), random_tree(rng, 33, 5)]
    TreeCase(rng, 16, 2, D, 64, [9000, 4001], trees).device(pkv).check(pkv)


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 4, 2), (128, 8, 2), (256, 3, 1), (512, 8, 1)])
@pytest.mark.parametrize("ctx", [0, 1, 2, 7, 8, 55, 63, 64, 65, 120, 126, 127, 128, 129, 191, 255,
                                 256, 257, 1000])
def test_context_lengths(D, Hq, Hkv, ctx):
    rng = rng_of(3, D, ctx)
    TreeCase(rng, Hq, Hkv, D, 8, [ctx, max(0, ctx - 5)],
             [random_tree(rng, 9, 3), random_tree(rng, 3, 1)]).device(pkv).check(pkv)


@pytest.mark.parametrize("ps", [8, 16, 32, 64, 128, 256, 1024])
@pytest.mark.parametrize("D", [64, 128, 256, 512])
def test_page_sizes(D, ps):
    rng = rng_of(4, D, ps)
    TreeCase(rng, 4, 1, D, ps, [515, 0, 130], [random_tree(rng, n, 2) for n in (12, 8, 30)]
             ).device(pkv).check(pkv)


@pytest.mark.parametrize("window", [1, 2, 5, 64, 100, 127, 128, 129, 200, 5000])
@pytest.mark.parametrize("D,G", [(128, 4), (256, 8), (512, 5)])
def test_windows(window, D, G):
    rng = rng_of(5, window, D)
    trees = [random_tree(rng, 20, 3), random_tree(rng, 40, 1), random_tree(rng, 6, 6), [-1]]
    TreeCase(rng, G, 1, D, 16, [300, 131, 0, 128], trees, window=window).device(pkv).check(pkv)


@pytest.mark.parametrize("window", [1, 300, 511, 512, 513])
@pytest.mark.parametrize("ns", [(9, 16, 20), (16, 16, 16), (17, 16, 16)])
def test_units_of_short_windows(window, ns):
    """Rows of up to and more than 128 columns in windows around a multiple of the tile."""
    rng = rng_of(24, window, *ns)
    trees = [random_tree(rng, n, 3) for n in ns]
    TreeCase(rng, 8, 1, 256, 64, [2000, 511, 90], trees, window=window).device(pkv).check(pkv)


def test_forests_and_empty_and_padding_rows():
    """Several roots, rows without nodes, rows on slot 0, nodes behind the last row."""
    rng = rng_of(6)
    trees = [random_tree(rng, 12, 3, roots=3), [], [-1] * 9, random_tree(rng, 4, 2), []]
    c = TreeCase(rng, 8, 2, 128, 16, [200, 77, 150, 5, 0], trees, slots=[5, 2, 1, 0, 3], pad=6)
    c.device(pkv).check(pkv)
    got = f64(c.out)
    assert (got[21:25] == 0).all() and (got[25:] == 7).all()


def test_no_rows_and_no_nodes():
    rng = rng_of(7)
    c = TreeCase(rng, 2, 1, 64, 16, [3, 4], [[], []], pad=2).device(pkv)
    c.call(pkv)
    torch.cuda.synchronize()
    assert (c.out == 7).all() and int(c.err) == 0


@pytest.mark.parametrize("B,ctx,nodes,D,Hq,Hkv", [
    (1, 20000, 4, 128, 32, 8), (1, 9000, 64, 64, 8, 8), (3, 7001, 13, 256, 8, 1),
    (1, 30000, 7, 512, 8, 1), (2, 4097, 64, 128, 16, 2), (1, 6000, 50, 512, 16, 2)])
def test_long_rows_are_cut(B, ctx, nodes, D, Hq, Hkv):
    rng = rng_of(8, ctx)
    TreeCase(rng, Hq, Hkv, D, 64, [ctx - 100 * b for b in range(B)],
             [random_tree(rng, nodes, 3) for _ in range(B)]).device(pkv).check(pkv)


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 2, 2), (128, 32, 8), (256, 8, 1), (512, 8, 1)])
def test_many_rows(D, Hq, Hkv):
    rng = rng_of(9, D)
    B = 200 if D <= 128 else 330
    trees = [random_tree(rng, int(rng.integers(1, 7)), 2) for _ in range(B)]
    TreeCase(rng, Hq, Hkv, D, 16, rng.integers(0, 150, B), trees).device(pkv).check(pkv)


def test_the_most_rows():
    rng = rng_of(10)
    trees = [random_tree(rng, int(rng.integers(0, 4)), 2) for _ in range(512)]
    TreeCase(rng, 3, 1, 64, 8, rng.integers(0, 60, 512), trees).device(pkv).check(pkv)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("more", [0, 20])
def test_values_of_other_branches_stay_out(value, D, more):
    """A node whose keys and values are not finite changes nothing for nodes that do not
    see it; the context behind a node's window likewise."""
    rng = rng_of(11, D)
    par = [-1, 0, 0, 1, 2, 3, 4, 1, 1] + [5] * more
    c = TreeCase(rng, 8, 1, D, 16, [100, 40], [par, par])
    bad = [tree.cache_row(c.table, s, ctx + 4, 16) for s, ctx in ((1, 100), (2, 40))]
    keep = c.kc[:, bad].copy(), c.vc[:, bad].copy()
    want = [x for x in c.want()]
    pattern = torch.tensor([value]).bfloat16().view(torch.int16).numpy()[0]
    for r in bad:
        c.kc[:, r], c.vc[:, r] = pattern, pattern
    c.device(pkv)
    got = f64(c.call(pkv))
    assert int(c.err) == 0
    sees = np.tile(tree.ancestors(par)[:, 4], 2)
    check_attn(got[~sees], want[0][~sees], want[1][~sees])
    assert keep[0].size
    # with only the values so, the nodes that see them have no finite result either
    c.kc[:, bad], c.vc[:, bad] = keep[0], pattern
    got = f64(c.device(pkv).call(pkv))
    check_attn(got[~sees], want[0][~sees], want[1][~sees])
    assert not np.isfinite(got[sees]).any()


@pytest.mark.parametrize("window", [3, 70])
def test_values_behind_a_window_stay_out(window):
    """A context token inside the root's window but not inside its deeper nodes'."""
    rng = rng_of(12, window)
    par = [-1, 0, 1, 2, 3, 0]
    c = TreeCase(rng, 4, 1, 128, 16, [150], [par], window=window)
    first = 150 - window + 1
    want = c.want()
    r = tree.cache_row(c.table, 1, first, 16)
    c.vc[:, r] = NAN_BF16
    got = f64(c.device(pkv).call(pkv))
    deep = np.array(tree.depths(par)) > 0
    check_attn(got[deep], want[0][deep], want[1][deep])
    assert np.isnan(got[0]).all()


def test_large_and_equal_scores():
    """Scores of hundreds, rising and falling along the row, and all alike."""
    rng = rng_of(13)
    for D in (128, 512):
        c = TreeCase(rng, 4, 1, D, 16, [400, 260], [random_tree(rng, 8, 2)] * 2,
                     scale=40 / D ** 0.5)
        c.device(pkv)
        got = f64(c.call(pkv))
        ref, mass = c.want()
        # scale sum |q k| < 600: fp32 products and sums move a weight by up to
        # 600 * 512 * 2^-24 < 2^-5
        assert (np.abs(got - ref) <= (2.0 ** -8 + 2.0 ** -5) * mass + 2.0 ** -8 * np.abs(ref)).all()
    c = TreeCase(rng, 4, 1, 128, 16, [400], [random_tree(rng, 8, 2)])
    c.kc[:] = 0
    c.device(pkv).check(pkv)
    for step in (-1, 1):    # every key outweighs all those before it by far, or none does
        c = TreeCase(rng, 2, 1, 64, 16, [600], [random_tree(rng, 5, 2)], scale=1.0)
        kc = torch.zeros(c.kc.shape)
        for j in range(605):
            kc[:, tree.cache_row(c.table, 1, j, 16), 0] = float(8 * step * (j // 8))
        c.kc = kc.bfloat16().view(torch.int16).numpy()
        c.q[:] = 0
        c.q[:, :, 0] = 1
        c.device(pkv).check(pkv)


def test_results_do_not_depend_on_the_run():
    rng = rng_of(14)
    c = TreeCase(rng, 32, 8, 128, 64, rng.integers(100, 1500, 24),
                 [random_tree(rng, 8, 2) for _ in range(24)]).device(pkv)
    first = c.call(pkv).clone()
    for _ in range(30):
        c.out.fill_(float("nan"))
        assert torch.equal(c.call(pkv), first)


def test_one_workspace_serves_every_shape():
    """Calls of all shapes in any order on one workspace: each finds its counts zero."""
    rng = rng_of(22)
    cases = [TreeCase(rng, Hq, Hkv, D, 64, ctx, [random_tree(rng, n, 2) for n in ns]).device(pkv)
             for Hq, Hkv, D, ctx, ns in (
                 (8, 1, 512, [20000], [6]), (32, 8, 128, [3000, 100, 900], [8, 4, 1]),
                 (8, 1, 256, [7000, 2000], [30, 20]), (2, 2, 64, [9000], [3]),
                 (8, 1, 128, [40000], [2]), (8, 8, 64, [700, 60], [64, 50]))]
    want = [c.call(pkv).clone() for c in cases]
    for c in cases:
        c.check(pkv)
    ws = torch.zeros(max(c.ws.nbytes for c in cases), dtype=torch.uint8, device="cuda")
    for i in rng.integers(0, len(cases), 60):
        assert torch.equal(cases[i].call(pkv, ws=ws, out=torch.full_like(cases[i].out, 7.0)),
                           want[i]), i


@pytest.mark.parametrize("D, G, ns", [(128, 4, [3, 1, 5]), (64, 1, [7, 2]), (128, 8, [11, 13]),
                                      (256, 8, [1, 9]), (512, 8, [3, 20])])
def test_unused_columns_change_nothing(D, G, ns):
    """Columns that a row does not fill hold what was there: results are the same whatever
    queries the calls before had."""
    rng = rng_of(23)
    c = TreeCase(rng, 2 * G, 2, D, 64, [500 + 300 * i for i in range(len(ns))],
                 [random_tree(rng, n, 2) for n in ns]).device(pkv)
    full = TreeCase(rng, 2 * G, 2, D, 64, [700] * 8,
                    [random_tree(rng, 64, 2) for _ in range(8)]).device(pkv)
    want = None
    for fill in (0.0, 1e3, -1e3, 3e38, float("inf"), float("nan")):
        full.t["q"].fill_(fill)
        full.call(pkv)
        got = c.call(pkv).clone()
        want = got if want is None else want
        assert torch.equal(got, want), fill


@pytest.mark.parametrize("D", [128, 256])
def test_lengths_and_trees_written_by_the_kernel_before(D):
    """What a call reads before the kernel ahead of it has ended may come from that kernel, if it
    is an ordinary one."""
    rng = rng_of(25, D)
    B, n = 24, 9
    c = TreeCase(rng, 8, 2, D, 32, rng.integers(400, 1500, B),
                 [random_tree(rng, n, 3) for _ in range(B)]).device(pkv)
    kinds = []
    for _ in range(3):
        ctx = torch.tensor(rng.integers(0, 400, B), dtype=torch.int32, device="cuda")
        cut = np.sort(rng.integers(0, B * n + 1, B - 1))
        start = np.concatenate([[0], cut, [B * n]])
        # rows out of the same packed nodes (one of more than 64 is left as it is), all of them roots
        start = np.minimum.accumulate(np.minimum(start, np.arange(B + 1) * 60)[::-1])[::-1]
        kinds.append((ctx, torch.tensor(start.copy(), dtype=torch.int32, device="cuda"),
                      torch.full((B * n,), -1, dtype=torch.int32, device="cuda")))
    ctx, start, parents = (x.clone() for x in kinds[0])
    want = []
    for k in kinds:
        torch.cuda.synchronize()
        out = torch.full_like(c.out, 7.0)
        want.append(c.call(pkv, ctx=k[0], row_start=k[1], parents=k[2], out=out).clone())
    outs = [torch.full_like(c.out, 7.0) for _ in range(60)]
    torch.cuda.synchronize()
    for i, out in enumerate(outs):
        for to, value in zip((ctx, start, parents), kinds[i % 3]):
            torch.add(value, 0, out=to)
        c.call(pkv, ctx=ctx, row_start=start, parents=parents, out=out)
    torch.cuda.synchronize()
    for i, out in enumerate(outs):
        assert torch.equal(out, want[i % 3]), i


def test_cache_beyond_32_bits():
    """Rows whose elements lie past 2^32: the last pages of a 9 GB cache."""
    D, ps, P, Hkv = 128, 128, 1 << 17, 2
    rng = rng_of(15)
    c = TreeCase(rng, 4, Hkv, D, ps, [500, 130], [random_tree(rng, 8, 2)] * 2)
    c.device(pkv)
    big = [torch.empty((Hkv, P * ps, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    shift = P - c.P
    for small, large in zip((c.t["kc"], c.t["vc"]), big):
        large[:, shift * ps:] = small
    table = c.t["table"].clone()
    table[table > 0] += shift
    small_P, c.P = c.P, P
    got = c.call(pkv, kc=big[0], vc=big[1], table=table)
    c.P = small_P
    c.check(pkv, out=got)


def test_no_batch_index_and_no_error_word():
    rng = rng_of(16)
    c = TreeCase(rng, 4, 2, 64, 16, [0, 33, 90], [[], random_tree(rng, 5, 2),
                                                  random_tree(rng, 7, 1)], slots=[0, 1, 2])
    c.device(pkv)
    c.err, want = None, c.call(pkv).clone()
    assert torch.equal(c.call(pkv, slots=None), want)
    check_attn(f64(want), *c.want())


@pytest.mark.parametrize("what,bit,rows", [
    ("parent", pkv.PKV_ERR_TREE, ()), ("slot", pkv.PKV_ERR_SLOT, (1,)),
    ("ctx", pkv.PKV_ERR_POS, (1,)), ("negative ctx", pkv.PKV_ERR_POS, (1,)),
    ("page", pkv.PKV_ERR_PAGE_NEG, (1,)), ("page range", pkv.PKV_ERR_PAGE_RANGE, (1,)),
    ("row_start", pkv.PKV_ERR_TREE, (2,)), ("too many", pkv.PKV_ERR_TREE, (1,))])
def test_faults_are_reported_and_stay_in_their_row(what, bit, rows):
    rng = rng_of(17)
    trees = [random_tree(rng, 6, 2), random_tree(rng, 7, 2), random_tree(rng, 5, 2)]
    c = TreeCase(rng, 4, 1, 128, 16, [90, 200, 40], trees).device(pkv)
    t = {k: v.clone() for k, v in c.t.items()}
    if what == "parent":
        t["parents"][8] = 5            # row 1's node 2 names a later node: it counts as a root
        c.parents[8] = -1
    elif what == "slot":
        t["slots"][1] = 99
    elif what == "ctx":
        t["ctx"][1] = c.max_pages * 16 - 3
    elif what == "negative ctx":
        t["ctx"][1] = -1
    elif what == "page":
        t["table"][2, 3] = -7
    elif what == "page range":
        t["table"][2, 3] = c.P
    elif what == "row_start":
        t["row_start"][3] = 19         # past the packed nodes
    else:                              # 65 nodes in one row, where the packed ones are enough
        trees = [random_tree(rng, 6, 2), random_tree(rng, 64, 2), random_tree(rng, 5, 2)]
        c = TreeCase(rng, 4, 1, 128, 16, [90, 200, 40], trees).device(pkv)
        t = {k: v.clone() for k, v in c.t.items()}
        t["row_start"][2] += 1
    got = f64(c.call(pkv, **t))
    assert int(c.err) & bit, int(c.err)
    want, mass = c.want()
    for b in range(3):
        if b in rows or (what == "too many" and b == 2):
            continue
        s = slice(int(c.row_start[b]), int(c.row_start[b + 1]))
        check_attn(got[s], want[s], mass[s])


def test_graph_replays_follow_the_trees():
    """One captured call serves other trees, lengths and batches of no more nodes and rows;
    two graphs share a workspace."""
    rng = rng_of(18)
    cases = [TreeCase(rng, 8, 2, 128, 16, ctx, [random_tree(rng, n, 3) for n in ns],
                      pad=40 - sum(ns), max_pages=80)
             for ctx, ns in (([700, 30, 0], [8, 9, 3]), ([5, 1200, 90], [20, 1, 4]),
                             ([0, 0, 0], [0, 1, 0]), ([900, 100, 333], [13, 13, 14]))]
    P = max(c.P for c in cases)
    for c in cases:
        pad = P - c.P
        c.kc, c.vc = (np.concatenate([x, np.zeros((2, pad * 16, 128), x.dtype)], 1)
                      for x in (c.kc, c.vc))
        c.P = P
    live = TreeCase(rng, 8, 2, 128, 16, [0, 0, 0], [[], [], []], pad=40, max_pages=80)
    live.kc, live.vc, live.P = cases[0].kc, cases[0].vc, P
    live.device(pkv)
    other = TreeCase(rng, 8, 1, 256, 16, [400], [random_tree(rng, 30, 3)]).device(pkv)
    ws = torch.zeros(max(live.ws.nbytes, other.ws.nbytes), dtype=torch.uint8, device="cuda")
    graphs = []
    for c in (live, other):
        c.call(pkv, ws=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.call(pkv, ws=ws)
        graphs.append(g)
    for c in cases + cases[:1]:
        c.device(pkv)
        for k in live.t:
            live.t[k].copy_(c.t[k])
        live.out.fill_(7.0)
        other.out.zero_()
        graphs[0].replay()
        graphs[1].replay()
        c.check(pkv, out=live.out)
        other.check(pkv, out=other.out)


def test_side_streams():
    rng = rng_of(19)
    c = TreeCase(rng, 16, 4, 128, 16, rng.integers(1, 900, 9),
                 [random_tree(rng, 6, 2) for _ in range(9)]).device(pkv)
    want = c.call(pkv).clone()
    torch.cuda.synchronize()
    outs = []
    for _ in range(3):
        s = torch.cuda.Stream()
        ws, out = torch.empty_like(c.ws), torch.empty_like(c.out)
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            for _ in range(5):
                c.call(pkv, ws=ws, out=out)
        outs.append((s, out))
    for s, out in outs:
        s.synchronize()
        assert torch.equal(out, want)
