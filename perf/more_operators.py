"""Cases of speculative decoding over the paged cache: the append of a row's drafted
tokens (a tree) with norm and rotation, the attention of such a tree, the verification of
the drafts against the target's probabilities, and the move of the accepted tokens' keys
and values to where they belong.

``own`` False runs each operator in its plain form (elementary torch operations); True
calls the library. ``exact`` gives the 64-bit value of the outputs.

A row b has ``ctx`` tokens in the cache and a tree of drafted tokens ("nodes") behind
them, node 0 the last token known for certain. Nodes are packed over the rows
(``row_start`` [B + 1]); ``parents`` names each node's parent inside its row, before it.
Node i sits at cache position ctx + i and at rotation position ctx + depth(i).
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

EPS = 1e-6


# ------------------------------------------------------------------ cases ----

def listed():
    return [
        # a chat batch drafting four tokens a row: launch and latency only
        append("append_chain_b8", B=8, nodes=5, width=1, Hq=32, Hkv=8, D=128, page=64, lo=64,
               hi=1024),
        # the rollout batch with trees: a thousand tokens a step
        append("append_tree_b64", B=64, nodes=24, width=4, Hq=32, Hkv=8, D=128, page=64, lo=100,
               hi=1024),
        # one short answer with three drafts: latency only; ratio 2, small pages
        attn("attn_one_chain", B=1, nodes=4, width=1, Hq=2, Hkv=1, D=64, page=16, lo=37, hi=37),
        # the rollout batch: 64 rows of 100 to 1024 tokens, trees of up to 8 nodes
        attn("attn_rollout_b64", B=64, nodes=8, width=3, Hq=32, Hkv=8, D=128, page=64, lo=100,
             hi=1024),
        # long prompts, few rows: the long axis is split
        attn("attn_long_b16", B=16, nodes=8, width=1, Hq=32, Hkv=8, D=128, page=64, lo=16384,
             hi=32768),
        # the sliding layer of the Gemma-4 workload
        attn("attn_window_d256", B=64, nodes=16, width=4, Hq=8, Hkv=1, D=256, page=64, lo=256,
             hi=2048, window=512),
        # its full layer under the widest trees
        attn("attn_wide_d512", B=16, nodes=64, width=8, Hq=8, Hkv=1, D=512, page=64, lo=256,
             hi=2048),
        # one answer, three drafts of a small model
        verify("verify_one_chain", B=1, nodes=4, width=1, V=32000, sampled=True),
        # the rollout batch, five sampled drafts a row
        verify("verify_chain_b64", B=64, nodes=6, width=1, V=151936, sampled=True),
        # trees of the draft's likeliest tokens over a large vocabulary
        verify("verify_tree_b16", B=16, nodes=32, width=4, V=262144, sampled=False),
        # one bf16 layer of a chat batch
        keep("keep_one_layer", B=8, nodes=16, width=4, caches=2, heads=8, D=128, page=64, lo=64,
             hi=256),
        # every layer of the rollout batch in one call
        keep("keep_all_layers", B=64, nodes=16, width=4, caches=48, heads=8, D=128, page=32, lo=20,
             hi=100),
    ]


def append(name, **kw):
    return dict(dict(op="append", rotary=0, v_norm=False, k_eq_v=False), **kw, name=name)


def attn(name, **kw):
    return dict(dict(op="attn", window=0), **kw, name=name)


def verify(name, **kw):
    return dict(dict(op="verify"), **kw, name=name)


def keep(name, **kw):
    return dict(dict(op="keep"), **kw, name=name)


def draw(rng):
    def logu(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(("append", "attn", "attn", "attn", "verify", "verify", "keep"))
    page = rng.choice((16, 32, 64, 128))
    nodes, width = logu(1, 64), rng.choice((1, 1, 2, 4, 8))
    if op == "append":
        D = rng.choice((64, 128, 128, 256, 512))
        Hkv = rng.choice((1, 2, 4, 8)) if D <= 128 else rng.choice((1, 2))
        B = logu(1, max(1, min(256, 1600 // nodes)))
        hi = logu(1, 1500)
        gemma = rng.random() < 0.4
        c = append("", B=B, nodes=nodes, width=width, Hq=Hkv * rng.randint(1, 8), Hkv=Hkv, D=D,
                   page=page, lo=rng.randint(0, hi), hi=hi,
                   rotary=rng.choice((0, D // 4, D // 2)) if gemma else 0, v_norm=gemma,
                   k_eq_v=gemma and rng.random() < 0.5)
    elif op == "attn":
        D = rng.choice((64, 128, 128, 256, 512))
        Hkv = rng.choice((1, 2, 4, 8)) if D <= 128 else rng.choice((1, 2))
        ratio = rng.randint(1, 8)
        B = logu(1, 256)
        top = min(32768, (180 << 20) // (B * Hkv * D), (9 << 30) // (B * Hkv * ratio * nodes * D))
        hi = logu(1, max(1, top))
        c = attn("", B=B, nodes=nodes, width=width, Hq=Hkv * ratio, Hkv=Hkv, D=D, page=page,
                 lo=rng.randint(0, hi), hi=hi, window=rng.choice((0, 0, 0, 129, 512, 1024)))
    elif op == "verify":
        V = logu(1000, 262144)
        B = logu(1, max(1, min(128, (100 << 20) // (V * nodes))))
        c = verify("", B=B, nodes=nodes, width=width, V=V, sampled=rng.random() < 0.6)
    else:
        D = rng.choice((64, 128, 256, 512))
        heads = rng.choice((1, 2, 4, 8))
        B, hi = logu(1, 128), logu(1, 300)
        size = B * (hi + nodes + page) * heads * D * 2
        c = keep("", B=B, nodes=nodes, width=width, heads=heads, D=D, page=page,
                 caches=logu(1, max(1, min(64, (800 << 20) // size))), lo=rng.randint(0, hi), hi=hi)
    c.pop("name")
    return c


def _spread(lo, hi, n):
    """n whole numbers evenly over [lo, hi]; the seed only decides which row has which."""
    return np.rint(np.linspace(lo, hi, n)).astype(np.int64)


def _sizes(case):
    """Nodes of the rows: from half the most up to the most."""
    return _spread((case["nodes"] + 1) // 2, case["nodes"], case["B"])


def work(case):
    B, n = case["B"], int(_sizes(case).sum())
    if case["op"] == "append":
        kv = (1 if case["k_eq_v"] else 2) + 2
        return {"bytes": 2 * n * case["D"] * (2 * case["Hq"] + kv * case["Hkv"]),
                "flops": 10 * n * case["D"] * (case["Hq"] + case["Hkv"])}
    if case["op"] == "attn":
        ctx = _spread(case["lo"], case["hi"], B)
        seen = np.minimum(ctx, case["window"]) if case["window"] > 0 else ctx
        q = n * case["Hq"] * case["D"] * 2
        # every node sees the context and, at the least, itself
        pairs = float(seen.mean() + 1) * n
        return {"bytes": 4 * (int(seen.sum()) + n) * case["Hkv"] * case["D"] + 2 * q,
                "flops": 4 * pairs * case["Hq"] * case["D"]}
    if case["op"] == "verify":
        # the target's row at the last accepted node, and the draft's (a long chain of
        # samples is nearly always cut short)
        return {"bytes": 4 * B * case["V"] * (2 if case["sampled"] else 1), "flops": B * case["V"]}
    # half the nodes of a path are taken to move
    each = case["caches"] * case["heads"] * case["D"] * 2
    return {"bytes": 2 * each * B, "flops": 0}


# ----------------------------------------------------------------- inputs ----

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)


def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


def _trees(rng, case):
    """Parents of every row's nodes: a chain (width 1), or each node under one of the
    ``width`` nodes before it."""
    sizes = rng.permutation(_sizes(case))
    parents = []
    for n in sizes:
        i = np.arange(1, n)
        back = rng.integers(1, np.minimum(i, case["width"]) + 1) if n > 1 else i
        parents.append(np.concatenate([[-1], i - back]))
    return sizes, np.concatenate([[0], np.cumsum(sizes)]), np.concatenate(parents)


def _paged(rng, case, sizes, ctx):
    """Pages for ctx + nodes tokens of every row, drawn from a permutation; slot 0 is the
    no-op slot."""
    B, ps = case["B"], case["page"]
    slot = rng.permutation(np.arange(1, B + 1))
    need = np.zeros(B + 1, np.int64)
    need[slot] = -(-(ctx + sizes) // ps)
    max_pages = -(-(case["hi"] + case["nodes"]) // ps)
    n_pages = B * max_pages + 3
    perm = rng.permutation(np.arange(1, n_pages))
    table = np.full((B + 1, max_pages), -1, np.int64)
    table[0] = 0
    at = np.cumsum(need) - need
    for s in range(1, B + 1):
        table[s, :need[s]] = perm[at[s]:at[s] + need[s]]
    return dict(batch_idx=_i32(slot), table=_i32(table), n_slots=B + 1, max_pages=max_pages,
                n_pages=n_pages)


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    g = _gen(seed)
    st = dict(case)
    sizes, start, parents = _trees(rng, case)
    N = int(start[-1])
    st.update(row_start=_i32(start), parents=_i32(parents), N=N)
    if case["op"] == "verify":
        return _prepare_verify(st, rng, g, start, parents)
    ctx = rng.permutation(_spread(case["lo"], case["hi"], case["B"]))
    st.update(_paged(rng, case, sizes, ctx), ctx_lens=_i32(ctx))
    rows = st["n_pages"] * case["page"]
    if case["op"] == "keep":
        pool = _randn(g, case["caches"], case["heads"], rows, case["D"])
        # a root-to-leaf walk cut at some depth, as verification leaves it
        path = np.full((case["B"], case["nodes"]), -1, np.int64)
        accepted = np.zeros(case["B"], np.int64)
        for b in range(case["B"]):
            par = parents[start[b]:start[b + 1]]
            walk = [int(rng.integers(0, len(par)))]
            while par[walk[-1]] >= 0:
                walk.append(int(par[walk[-1]]))
            path[b, :len(walk)] = walk[::-1]
            accepted[b] = len(walk) - 1
        st.update(pool=pool, kv=list(pool.unbind(0)), accepted=_i32(accepted), path=_i32(path))
        return st
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    st.update(k_cache=_randn(g, Hkv, rows, D), v_cache=_randn(g, Hkv, rows, D))
    if case["op"] == "attn":
        st.update(q=_randn(g, N, Hq, D), scale=D ** -0.5,
                  out=torch.empty((N, Hq, D), dtype=torch.bfloat16, device="cuda"))
        return st
    # q, k and v as the fused projection leaves them: parts of one row
    qkv = _randn(g, N, (Hq + 2 * Hkv) * D)
    q, k, v = qkv.split([Hq * D, Hkv * D, Hkv * D], 1)
    gain = [1 + 0.1 * torch.randn(D, generator=g, device="cuda") for _ in range(2)]
    st.update(q=q.unflatten(1, (Hq, D)), k=k.unflatten(1, (Hkv, D)),
              v=None if case["k_eq_v"] else v.unflatten(1, (Hkv, D)),
              gamma_q=gain[0].bfloat16(), gamma_k=gain[1].bfloat16(), theta=1e6,
              q_out=torch.empty((N, Hq, D), dtype=torch.bfloat16, device="cuda"))
    return st


def _prepare_verify(st, rng, g, start, parents):
    """Target and draft rows of many unlikely tokens and, mostly, one likely one; the drafts
    are samples of the draft's rows, or their likeliest tokens."""
    N, V = st["N"], st["V"]
    logits = 4 * torch.randn((N, V), generator=g, device="cuda")
    top = torch.randint(0, V, (N, 1), generator=g, device="cuda")
    lead = 4 * torch.rand((N, 1), generator=g, device="cuda") - 1
    logits.scatter_(1, top, torch.logsumexp(logits, 1, keepdim=True) + lead)
    draft = logits + 0.7 * torch.randn((N, V), generator=g, device="cuda")
    target, draft = torch.softmax(logits, 1), torch.softmax(draft, 1)
    del logits
    base = np.repeat(start[:-1], np.diff(start))
    parent = np.where(parents < 0, 0, parents) + base
    # rank of each node among its siblings
    order = np.argsort(parent + np.where(parents < 0, N, 0), kind="stable")
    rank = np.zeros(N, np.int64)
    key = (parent + np.where(parents < 0, N, 0))[order]
    first = np.concatenate([[0], np.flatnonzero(np.diff(key)) + 1])
    rank[order] = np.arange(N) - np.repeat(first, np.diff(np.append(first, N)))
    most = int(rank[parents >= 0].max()) + 1 if (parents >= 0).any() else 0
    at = torch.from_numpy(parent).cuda()
    if st["sampled"]:
        # the least of exponential times at rate q is a sample of q
        token = torch.empty(N, dtype=torch.long, device="cuda")
        for part in torch.arange(N, device="cuda").split(256):
            t = torch.empty((len(part), V), device="cuda").exponential_(generator=g)
            token[part] = (t / draft[at[part]]).argmin(1)
    else:
        best = draft.topk(max(most, 1), 1).indices
        token = best[at, torch.from_numpy(np.where(parents < 0, 0, rank)).cuda()]
    st.update(target=target, draft=draft if st["sampled"] else None, tokens=token.int(),
              most=most, u_accept=torch.rand(N, generator=g, device="cuda"),
              u_pick=torch.rand(st["B"], generator=g, device="cuda"),
              accepted=torch.empty(st["B"], dtype=torch.int32, device="cuda"),
              path=torch.empty((st["B"], st["nodes"]), dtype=torch.int32, device="cuda"),
              next_token=torch.empty(st["B"], dtype=torch.int32, device="cuda"))
    return st


# ------------------------------------------------------------------- runs ----

def run(st):
    if st["op"] == "append":
        return _own_append(st) if own else _plain_append(st)
    if st["op"] == "attn":
        return _own_attn(st) if own else _plain_attn(st)
    if st["op"] == "verify":
        return _own_verify(st) if own else _plain_verify(st)
    return _own_keep(st) if own else _plain_keep(st)


def _own_append(st):
    import paged_kv_decode_pagetable_gb300 as pkv
    pkv.tree_qkv_norm_rope_append(
        st["q"], st["k"], st["v"], st["gamma_q"], st["gamma_k"], st["batch_idx"], st["ctx_lens"],
        st["row_start"], st["parents"], st["theta"], EPS, st["rotary"] or None, st["v_norm"],
        st["table"], st["n_slots"], st["max_pages"], st["page"], st["n_pages"], st["k_cache"],
        st["v_cache"], st["q_out"])
    return st["q_out"], st["k_cache"], st["v_cache"]


def _own_attn(st):
    import paged_kv_decode_pagetable_gb300 as pkv
    if "workspace" not in st:     # a program keeps one for every step
        n = pkv.paged_tree_attn_workspace(st["Hq"], st["Hkv"], st["D"])
        st["workspace"] = torch.zeros(n, dtype=torch.uint8, device="cuda")
    pkv.paged_tree_attn(st["q"], st["k_cache"], st["v_cache"], st["table"], st["n_slots"],
                        st["max_pages"], st["page"], st["n_pages"], st["batch_idx"],
                        st["ctx_lens"], st["row_start"], st["parents"], st["window"], st["scale"],
                        st["workspace"], st["out"])
    return st["out"]


def _own_verify(st):
    import paged_kv_decode_pagetable_gb300 as pkv
    pkv.tree_verify(st["target"], st["draft"], st["tokens"], st["row_start"], st["parents"],
                    st["u_accept"], st["u_pick"], st["accepted"], st["path"], st["next_token"])
    return st["accepted"], st["path"], st["next_token"]


def _own_keep(st):
    import paged_kv_decode_pagetable_gb300 as pkv
    pkv.kv_keep_path(st["kv"], st["table"], st["n_slots"], st["max_pages"], st["page"],
                     st["n_pages"], st["batch_idx"], st["ctx_lens"], st["accepted"], st["path"])
    return st["pool"]


def _packed(st):
    """Row, index in the row, and padded ancestors-or-self [B][nodes][nodes] of the nodes."""
    start, parents = st["row_start"].long(), st["parents"].long()
    node = torch.arange(st["N"], device="cuda")
    row = torch.searchsorted(start, node, right=True) - 1
    at = node - start[row]
    step = torch.zeros((st["B"], st["nodes"], st["nodes"]), device="cuda")
    has = parents >= 0
    step[row[has], at[has], parents[has]] = 1
    # powers of (parent or self) by squaring: six cover a tree of 64 nodes
    seen = step + torch.eye(st["nodes"], device="cuda")
    return row, at, _squared(_squared(_squared(_squared(_squared(_squared(seen))))))


def _squared(m):
    return (m @ m > 0).float()


def _cache_rows(st, slot, pos):
    """Cache rows of the tokens `pos` of `slot`."""
    ps = st["page"]
    return st["table"][slot, pos // ps].long() * ps + pos % ps


def _norm(x, gain=None):
    x = x.float()
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    return x if gain is None else x * gain.float()


def _rotate(x, pos, theta, rotary):
    D = x.shape[-1]
    i = torch.arange(D // 2, device=x.device, dtype=torch.float64)
    freq = torch.where(i < rotary // 2, theta ** (-2 * i / D), 0.0)
    phi = (pos.double()[:, None] * freq)[:, None]
    c, s = torch.cos(phi).float(), torch.sin(phi).float()
    a, b = x[..., :D // 2], x[..., D // 2:]
    return torch.cat([a * c - b * s, b * c + a * s], -1)


def _plain_append(st):
    row, at, seen = _packed(st)
    ctx = st["ctx_lens"].long()[row]
    pos = ctx + seen.sum(-1).long()[row, at] - 1
    rotary = st["rotary"] or st["D"]
    st["q_out"].copy_(_rotate(_norm(st["q"], st["gamma_q"]), pos, st["theta"], rotary))
    k = _rotate(_norm(st["k"], st["gamma_k"]), pos, st["theta"], rotary)
    v = st["k"] if st["v"] is None else st["v"]
    v = _norm(v) if st["v_norm"] else v
    to = _cache_rows(st, st["batch_idx"].long()[row], ctx + at)
    st["k_cache"][:, to] = k.bfloat16().transpose(0, 1)
    st["v_cache"][:, to] = v.bfloat16().transpose(0, 1)
    return st["q_out"], st["k_cache"], st["v_cache"]


def _plain_attn(st):
    B, T, H, W = st["B"], st["nodes"], st["Hkv"], st["window"]
    row, at, seen = _packed(st)
    D, G = st["D"], st["Hq"] // st["Hkv"]
    q = torch.zeros((B, T, H, G, D), device="cuda")
    q[row, at] = st["q"].float().view(-1, H, G, D)
    ctx = st["ctx_lens"].long()
    j = torch.arange(st["max_pages"] * st["page"], device="cuda")
    depth = seen.sum(-1).long() - 1                              # [B][T]
    tree = (j[None] - ctx[:, None]).clamp(0, T - 1)              # node of a key, if it is one
    is_ctx = j[None] < ctx[:, None]
    is_node = ~is_ctx & (j[None] < ctx[:, None] + T)
    keep = torch.where(is_ctx[:, None], True,
                       is_node[:, None] & (seen.gather(2, tree[:, None].expand(-1, T, -1)) > 0))
    if W > 0:
        key = torch.where(is_ctx, j[None], ctx[:, None] + depth.gather(1, tree))
        keep &= (ctx[:, None] + depth)[:, :, None] - key[:, None] < W
    r = _cache_rows(st, st["batch_idx"].long()[:, None], j[None].expand(B, -1)).clamp(min=0)
    k = st["k_cache"][:, r].float()                              # [H][B][keys][D]
    s = torch.einsum("bthgd,hbjd->bhgtj", q, k) * st["scale"]
    del k
    s = torch.where(keep[:, None, None], s, -math.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True))
    total = p.sum(-1, keepdim=True)
    v = st["v_cache"][:, r].float()
    o = torch.einsum("bhgtj,hbjd->bhgtd", p, v) / total
    st["out"].copy_(o.permute(0, 3, 1, 2, 4)[row, at].reshape(-1, st["Hq"], D))
    return st["out"]


def _plain_verify(st):
    row, at, seen = _packed(st)
    N, B, V = st["N"], st["B"], st["V"]
    start = st["row_start"].long()
    parents = st["parents"].long()
    child = parents >= 0
    up = start[row] + parents.clamp(min=0)                       # the parent among all nodes
    tok = st["tokens"].long()
    u = st["u_accept"].double()
    p = st["target"][up, tok].double()
    node = torch.arange(N, device="cuda")
    sibling = (up[:, None] == up[None]) & (node[:, None] > node[None])
    sibling &= child[:, None] & child[None]
    rank = sibling.sum(1)
    kids = torch.zeros(N, dtype=torch.long, device="cuda").index_add_(0, up, child.long())
    if st["draft"] is None:
        twice = (sibling & (tok[:, None] == tok[None])).any(1)
        p = torch.where(twice, 0.0, p)
        left = 1 - sibling.double() @ p
        good = u * left < p
    else:
        q = st["draft"][up, tok].double()
        # a and S of every node after so many rejections
        a, S = [torch.zeros(N, device="cuda").double()], [torch.ones(N, device="cuda").double()]
        for _ in range(st["most"]):
            a.append(a[-1] + S[-1])
            S.append(_residual(st["target"], st["draft"], a[-1]).sum(1) if len(a) <= st["most"]
                     else S[-1])
        a, S = torch.stack(a), torch.stack(S)
        good = u * q * S[rank, up] < (p - a[rank, up] * q).clamp(min=0)
    # the first good child of every node, then the nodes whose ancestors are all such
    earlier = sibling.double() @ good.double() > 0
    taken = (good & ~earlier & child) | (at == 0)
    bad = torch.zeros((B, st["nodes"]), device="cuda")
    bad[row, at] = (~taken).float()
    alive = (seen @ bad[:, :, None])[:, :, 0] == 0
    alive &= torch.arange(st["nodes"], device="cuda")[None] < (start[1:] - start[:-1])[:, None]
    count = alive.sum(1)
    st["accepted"].copy_(count - 1)
    t = torch.arange(st["nodes"], device="cuda")
    order = torch.where(alive, t[None], st["nodes"]).sort(1).values
    st["path"].copy_(torch.where(order < st["nodes"], order, -1))
    last = start[:-1] + order.gather(1, (count - 1)[:, None])[:, 0]
    w = st["target"][last].double()
    if st["draft"] is None:
        gone = (up == last[row]) & child
        w[row[gone], tok[gone]] = 0
    else:
        w = _residual(w, st["draft"][last], a[kids[last], last])
    total = w.cumsum(1)
    pick = (total > st["u_pick"].double()[:, None] * total[:, -1:]).int().argmax(1)
    st["next_token"].copy_(pick)
    return st["accepted"], st["path"], st["next_token"]


def _residual(p, q, a):
    return (p.double() - a[:, None] * q.double()).clamp(min=0)


def _plain_keep(st):
    t = torch.arange(st["nodes"], device="cuda")
    moves = (t[None] >= 1) & (t[None] <= st["accepted"].long()[:, None])
    b, i = moves.nonzero(as_tuple=True)
    slot, ctx = st["batch_idx"].long()[b], st["ctx_lens"].long()[b]
    src = _cache_rows(st, slot, ctx + st["path"].long()[b, i])
    dst = _cache_rows(st, slot, ctx + i)
    st["pool"][:, :, dst] = st["pool"][:, :, src]
    return st["pool"]


# ------------------------------------------------------------------ exact ----

def exact(case, seed):
    if case["op"] == "keep":
        return None          # copies: nothing is computed
    st = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(st)
    if case["op"] == "attn":
        return _exact_attn(st)
    return _exact_verify(st)


def _rows_of(st):
    """(row, first node, parents of its nodes, depths, slot, ctx) of every row."""
    start, parents = st["row_start"].tolist(), st["parents"].tolist()
    for b in range(st["B"]):
        par = parents[start[b]:start[b + 1]]
        depth = []
        for i in par:
            depth.append(0 if i < 0 else depth[i] + 1)
        yield b, start[b], par, depth


def _exact_append(st):
    D, ps = st["D"], st["page"]
    rotary = st["rotary"] or D
    freq = st["theta"] ** (-2 * np.arange(D // 2) / D) * (np.arange(D // 2) < rotary // 2)
    table, ctx = st["table"].tolist(), st["ctx_lens"].tolist()
    slots = st["batch_idx"].tolist()

    def unit(x):
        return x / np.sqrt((x * x).mean(-1, keepdims=True) + EPS)

    def host(x):
        return x.double().cpu().numpy()

    q, k = host(st["q"]), host(st["k"])
    v = k if st["v"] is None else host(st["v"])
    q, key = unit(q) * host(st["gamma_q"]), unit(k) * host(st["gamma_k"])
    v = unit(v) if st["v_norm"] else v
    caches = [host(st["k_cache"]), host(st["v_cache"])]
    for b, n0, par, depth in _rows_of(st):
        for i in range(len(par)):
            phi = (ctx[b] + depth[i]) * freq
            z = np.exp(1j * phi)
            for x in (q, key):
                y = (x[n0 + i, :, :D // 2] + 1j * x[n0 + i, :, D // 2:]) * z
                x[n0 + i] = np.concatenate([y.real, y.imag], -1)
            at = ctx[b] + i
            r = table[slots[b]][at // ps] * ps + at % ps
            caches[0][:, r] = key[n0 + i]
            caches[1][:, r] = v[n0 + i]
    return torch.from_numpy(q), torch.from_numpy(caches[0]), torch.from_numpy(caches[1])


def _exact_attn(st):
    """Row by row in 64 bits, every node against the list of its keys' masks."""
    H, D, ps, W = st["Hkv"], st["D"], st["page"], st["window"]
    out = torch.zeros((st["N"], st["Hq"], D), dtype=torch.float64, device="cuda")
    ctx, slots = st["ctx_lens"].tolist(), st["batch_idx"].tolist()
    for b, n0, par, depth in _rows_of(st):
        n, c = len(par), ctx[b]
        mask = np.zeros((n, c + n), bool)
        mask[:, :c] = True
        for i in range(n):
            s = i
            while s >= 0:
                mask[i, c + s] = True
                s = par[s]
        if W > 0:
            key = np.concatenate([np.arange(c), c + np.array(depth)])
            mask &= (c + np.array(depth))[:, None] - key[None] < W
        t = torch.arange(c + n, device="cuda")
        r = st["table"][slots[b]].long()[t // ps] * ps + t % ps
        k, v = st["k_cache"][:, r].double(), st["v_cache"][:, r].double()
        q = st["q"][n0:n0 + n].double().view(n, H, -1, D).permute(1, 2, 0, 3) * float(st["scale"])
        s = torch.einsum("hgtd,hjd->hgtj", q, k)
        s.masked_fill_(~torch.from_numpy(mask).cuda(), -math.inf)
        p = torch.softmax(s, -1)
        out[n0:n0 + n] = torch.einsum("hgtj,hjd->tghd", p, v).transpose(1, 2).reshape(n, -1, D)
    return out


def _exact_verify(st):
    """Row by row: the textbook's walk with its residual distribution kept normalised."""
    accepted, paths, picks = [], [], []
    tok, u = st["tokens"].tolist(), st["u_accept"].double().tolist()
    pick = st["u_pick"].double().tolist()
    for b, n0, par, _ in _rows_of(st):
        cur, path = 0, [0]
        dist = st["target"][n0].double()
        whole = True                          # dist is the target's own row
        for i in range(1, len(par)):
            if par[i] != cur:
                continue
            x, p = tok[n0 + i], float(dist[tok[n0 + i]])
            q = float(st["draft"][n0 + cur, x].double()) if st["sampled"] else 1.0
            if u[n0 + i] * q < p:
                cur, whole = i, True
                path.append(i)
                dist = st["target"][n0 + i].double()
                continue
            if st["sampled"]:
                dist = (dist - st["draft"][n0 + cur].double()).clamp(min=0)
            else:
                if whole:
                    dist, whole = dist.clone(), False
                left = 1 - float(dist[x]) if p > 0 else 1.0
                dist[x] = 0
                dist /= left
                continue
            dist = dist / dist.sum()
        c = torch.cumsum(dist, 0)
        picks.append(int((c > pick[b] * c[-1]).int().argmax()))
        accepted.append(len(path) - 1)
        paths.append(path + [-1] * (st["nodes"] - len(path)))
    return (torch.tensor(accepted, dtype=torch.int32), torch.tensor(paths, dtype=torch.int32),
            torch.tensor(picks, dtype=torch.int32))
