"""Cases of the 8-bit paged cache's operators: the quantising append, the decode
attention that reads the cache, and the copy of pages between places.

``own`` False runs each operator in its plain form (elementary torch operations in
32 bits); True calls the library. ``exact`` gives the 64-bit value of the outputs.

The 8-bit cache: per layer k_cache and v_cache are float8_e4m3fn
[Hkv][n_pages * page_size][D], with one fp32 power-of-two scale for each kv head and
block of ``block`` consecutive rows of a page: value = code * scale.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

FP8 = torch.float8_e4m3fn
E4M3_MAX = 448.0
MIN_EXP = -126          # smallest scale 2^-126, the smallest normal fp32


# ------------------------------------------------------------------ cases ----

def listed():
    return [
        # one short answer in flight: launch and latency only; ratio 2, small pages
        attn("attn_one_short", B=1, Hq=2, Hkv=1, D=64, page=16, block=16, lo=37, hi=37),
        # an interactive batch on the Qwen3-4B heads of the workloads
        attn("attn_chat_b8", B=8, Hq=32, Hkv=8, D=128, page=64, block=16, lo=64, hi=1024),
        # the rollout batch: 64 slots of up to 1024 tokens
        attn("attn_rollout_b64", B=64, Hq=32, Hkv=8, D=128, page=64, block=64, lo=100, hi=1024),
        # long prompts, few rows: the long axis is split
        attn("attn_long_b16", B=16, Hq=32, Hkv=8, D=128, page=64, block=32, lo=16384, hi=32768),
        # the sliding layer (window 512) and the full layer of the Gemma-4 workload
        attn("attn_window_d256", B=64, Hq=8, Hkv=1, D=256, page=64, block=16, lo=256, hi=2048,
             window=512),
        attn("attn_full_d512", B=64, Hq=8, Hkv=1, D=512, page=64, block=1, lo=256, hi=2048),
        # a decode step's new tokens; many of them land inside a block begun before
        append("append_step_b8", N=8, Hkv=8, D=128, page=64, block=16, prefill=False),
        append("append_step_b512", N=512, Hkv=4, D=256, page=32, block=32, prefill=False),
        # packed prompts, 16 documents of uneven length
        append("append_prompts_16k", N=16411, Hkv=8, D=128, page=64, block=16, prefill=True,
               docs=16),
        # one prompt forked once: the last, partly filled page of one bf16 layer
        copy("copy_fork_one", caches=2, heads=8, page=64, D=128, bits=16, pages=136, pairs=1,
             kind="fork"),
        # 64 prompts forked into groups of 8 on four 8-bit layers
        copy("copy_fork_groups", caches=8, heads=8, page=64, D=128, bits=8, pages=1025, pairs=448,
             kind="fork"),
        # moving the used pages of a fragmented bf16 cache to its front
        copy("copy_compact", caches=4, heads=8, page=64, D=128, bits=16, pages=2881, pairs=1311,
             kind="compact"),
    ]


def attn(name, **kw):
    return dict(dict(op="attn", window=0), **kw, name=name)


def append(name, **kw):
    return dict(dict(op="append", docs=1), **kw, name=name)


def copy(name, **kw):
    return dict(dict(op="copy"), **kw, name=name)


def draw(rng):
    def logu(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(("attn", "attn", "append", "copy"))
    if op == "copy":
        bits = rng.choice((8, 16))
        heads, D, page = rng.choice((1, 2, 4, 8)), rng.choice((64, 128, 256)), \
            rng.choice((16, 32, 64, 128))
        caches = rng.choice((1, 2, 3, 4, 8))
        page_bytes = caches * heads * page * D * bits // 8
        pairs = logu(1, max(1, min(2000, (600 << 20) // page_bytes)))
        kind = rng.choice(("fork", "compact"))
        c = copy("", caches=caches, heads=heads, page=page, D=D, bits=bits,
                 pages=2 * pairs + rng.randint(2, 40), pairs=pairs, kind=kind)
    elif op == "append":
        page = rng.choice((16, 32, 64, 128))
        block = rng.choice([b for b in (1, 8, 16, 32, 64) if b <= page])
        Hkv, D = rng.choice((1, 2, 4, 8)), rng.choice((64, 128, 256, 512))
        prefill = rng.random() < 0.5
        N = logu(2, (1 << 24) // (Hkv * D)) if prefill else logu(1, 512)
        c = append("", N=N, Hkv=Hkv, D=D, page=page, block=block, prefill=prefill,
                   docs=min(N, rng.randint(1, 24)) if prefill else 1)
    else:
        D = rng.choice((64, 128, 128, 256, 512))
        Hkv = rng.choice((1, 2, 4, 8)) if D <= 128 else rng.choice((1, 2))
        page = rng.choice((16, 32, 64, 128))
        block = rng.choice([b for b in (1, 8, 16, 32, 64) if b <= page])
        B = logu(1, 256)
        top = min(32768, (380 << 20) // (B * Hkv * D))
        hi = logu(2, max(2, top))
        lo = rng.randint(max(1, hi // 4), hi)
        window = rng.choice((0, 0, 0, 129, 512, 1024))
        c = attn("", B=B, Hq=Hkv * rng.randint(1, 8), Hkv=Hkv, D=D, page=page, block=block, lo=lo,
                 hi=hi, window=window)
    c.pop("name")
    return c


def _lengths(case):
    """Evenly spread over [lo, hi]; the seed only decides which row has which."""
    return np.rint(np.linspace(case["lo"], case["hi"], case["B"])).astype(np.int64)


def _splits(case):
    """Lengths of the documents of a packed prompt: uneven, summing to N."""
    n, d = case["N"], case["docs"]
    w = np.arange(1, d + 1, dtype=np.float64)
    cut = np.concatenate([[0], np.rint(np.cumsum(w) / w.sum() * n)]).astype(np.int64)
    return np.diff(cut)


def work(case):
    if case["op"] == "attn":
        L = _lengths(case)
        keys = int((np.minimum(L, case["window"]) if case["window"] > 0 else L).sum())
        n = keys * case["Hkv"]
        q = case["B"] * case["Hq"] * case["D"] * 2
        return {"bytes": 2 * n * case["D"] + 2 * 4 * n / case["block"] + 2 * q,
                "flops": 4 * keys * case["Hq"] * case["D"]}
    if case["op"] == "append":
        n = case["N"] * case["Hkv"]
        blocks = n / case["block"] if case["prefill"] else n
        return {"bytes": 2 * n * case["D"] * 3 + 2 * 4 * blocks, "flops": 4 * n * case["D"]}
    b = case["caches"] * case["heads"] * case["page"] * case["D"] * case["bits"] // 8
    return {"bytes": 2 * b * case["pairs"], "flops": 0}


# ----------------------------------------------------------------- inputs ----

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)


def _pow2_scale(amax):
    """Smallest power of two s >= 2^-126 with amax / s <= 448, for finite amax >= 0."""
    m, e = torch.frexp(amax.float())              # amax = m 2^e, m in [0.5, 1)
    k = e - 9 + (m > 0.875).to(e.dtype)           # 448 = 0.875 * 2^9
    k = torch.where(amax == 0, torch.full_like(k, MIN_EXP), k).clamp(min=MIN_EXP)
    return torch.ldexp(torch.ones_like(m), k)


def _fill(g, heads, rows, D, block):
    """A cache of `rows` rows in use: tokens of uneven size, quantised block by block."""
    codes = torch.empty((heads, rows, D), dtype=FP8, device="cuda")
    scale = torch.empty((heads, rows // block), dtype=torch.float32, device="cuda")
    for h in range(heads):
        size = torch.exp(0.7 * torch.randn((rows, 1), generator=g, device="cuda"))
        x = _randn(g, rows, D).float() * size
        s = _pow2_scale(x.abs().view(rows // block, block * D).amax(1))
        codes[h] = (x.view(rows // block, block, D) / s[:, None, None]).view(rows, D).to(FP8)
        scale[h] = s
    return codes, scale


def _table(rng, n_slots, max_pages, need, n_pages):
    """Pages of every slot drawn from a permutation; slot 0 is the no-op slot."""
    perm = rng.permutation(np.arange(1, n_pages))
    t = np.full((n_slots, max_pages), -1, np.int32)
    t[0] = 0
    at = 0
    for s, n in enumerate(need):
        t[s + 1, :n] = perm[at:at + n]
        at += n
    return torch.from_numpy(t).cuda()


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    g = _gen(seed)
    i32 = dict(dtype=torch.int32, device="cuda")
    st = dict(case)
    if case["op"] == "copy":
        P, n = case["pages"], case["pairs"]
        if case["bits"] == 16:
            pool = _randn(g, case["caches"], case["heads"], P, case["page"] * case["D"])
        else:
            pool = torch.randint(0, 120, (case["caches"], case["heads"], P,
                                          case["page"] * case["D"]), generator=g, device="cuda",
                                 dtype=torch.uint8).view(FP8)
        perm = rng.permutation(np.arange(1, P))
        if case["kind"] == "fork":        # several copies of few pages
            few = max(1, n // 7)
            src, dst = perm[np.arange(n) % few], perm[few:few + n]
        else:                             # used pages move to free ones nearer the front
            src, dst = np.sort(perm[:n])[::-1], np.sort(perm[n:2 * n])
        st.update(pool=pool, caches=list(pool.unbind(0)),
                  pairs=torch.from_numpy(np.stack([src, dst], 1).astype(np.int32)))
        return st
    H, D, ps, blk = case["Hkv"], case["D"], case["page"], case["block"]
    if case["op"] == "append":
        if case["prefill"]:
            lens = _splits(case)
            start = np.zeros(len(lens), np.int64)
            order = rng.permutation(len(lens))
            lens = lens[order]
            slot = np.repeat(np.arange(1, len(lens) + 1), lens)
            pos = np.concatenate([np.arange(n) for n in lens])
            need = -(-lens // ps)
        else:                             # one new token behind what each slot holds
            start = rng.integers(0, 4 * ps, case["N"])
            slot, pos = rng.permutation(np.arange(1, case["N"] + 1)), start
            lens = np.empty(case["N"], np.int64)
            lens[slot - 1] = start + 1
            need = -(-lens // ps)
        P = (int(need.sum()) if case["prefill"] else 4 * case["N"]) + 3
        k_cache, k_scale = _fill(g, H, P * ps, D, blk)
        v_cache, v_scale = _fill(g, H, P * ps, D, blk)
        shape = (H, case["N"], D) if case["prefill"] else (case["N"], H, D)
        size = torch.exp(0.7 * torch.randn((case["N"], 1), generator=g, device="cuda"))
        size = size if case["prefill"] else size[:, None]
        st.update(k=(_randn(g, *shape) * size).bfloat16(), v=(_randn(g, *shape) * size).bfloat16(),
                  batch_idx=torch.tensor(slot, **i32), input_pos=torch.tensor(pos, **i32))
        n_slots = len(need) + 1
    else:
        lens = rng.permutation(_lengths(case))
        need = -(-lens // ps)
        P = int(need.sum()) + 3
        k_cache, k_scale = _fill(g, H, P * ps, D, blk)
        v_cache, v_scale = _fill(g, H, P * ps, D, blk)
        n_slots = case["B"] + 1
        slot = rng.permutation(np.arange(1, n_slots))
        by_slot = np.empty(case["B"], np.int64)
        by_slot[slot - 1] = need
        need = by_slot
        st.update(q=_randn(g, case["B"], case["Hq"], D), scale=D ** -0.5,
                  batch_idx=torch.tensor(slot, **i32), seq_lens=torch.tensor(lens, **i32),
                  out=torch.empty((case["B"], case["Hq"], D), dtype=torch.bfloat16, device="cuda"))
    max_pages = int(need.max())
    st.update(k_cache=k_cache, v_cache=v_cache, k_scale=k_scale, v_scale=v_scale, n_pages=P,
              n_slots=n_slots, max_pages=max_pages,
              table=_table(rng, n_slots, max_pages, need, P))
    return st


# ------------------------------------------------------------------- runs ----

def run(st):
    if st["op"] == "copy":
        return _own_copy(st) if own else _plain_copy(st)
    if st["op"] == "append":
        return _own_append(st) if own else _plain_append(st)
    return _own_attn(st) if own else _plain_attn(st)


def _own_copy(st):
    import paged_kv_decode_pagetable_gb300 as pkv
    pkv.kv_copy_pages(st["caches"], st["pages"], st["pairs"])
    return st["pool"]


def _own_append(st):
    import paged_kv_decode_pagetable_gb300 as pkv
    call = pkv.kv_append_prefill_q8 if st["prefill"] else pkv.kv_append_q8
    call(st["k"], st["v"], st["batch_idx"], st["input_pos"], st["table"], st["n_slots"],
         st["max_pages"], st["page"], st["n_pages"], st["k_cache"], st["v_cache"], st["k_scale"],
         st["v_scale"])
    return st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"]


def _own_attn(st):
    import paged_kv_decode_pagetable_gb300 as pkv
    if "workspace" not in st:     # a program keeps one for every step
        n = pkv.paged_decode_attn_q8_workspace(st["Hq"], st["Hkv"], st["D"])
        st["workspace"] = torch.zeros(n, dtype=torch.uint8, device="cuda")
    pkv.paged_decode_attn_q8(st["q"], st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"],
                             st["table"], st["n_slots"], st["max_pages"], st["page"],
                             st["n_pages"], st["batch_idx"], st["seq_lens"], st["window"],
                             st["scale"], st["workspace"], st["out"])
    return st["out"]


def _plain_copy(st):
    pairs = st["pairs"].cuda().long()
    st["pool"].view(torch.int8)[:, :, pairs[:, 1]] = st["pool"].view(torch.int8)[:, :, pairs[:, 0]]
    return st["pool"]


def _rows(st, slot, pos):
    """Cache rows of the tokens `pos` of `slot`."""
    ps = st["page"]
    return st["table"][slot, pos // ps].long() * ps + pos % ps


def _plain_append(st):
    row = _rows(st, st["batch_idx"].long(), st["input_pos"].long())
    _append_one(st, st["k"], st["k_cache"], st["k_scale"], row)
    _append_one(st, st["v"], st["v_cache"], st["v_scale"], row)
    return st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"]


def _append_one(st, x, cache, scale, row):
    H, G = scale.shape[0], st["block"]
    x = (x if st["prefill"] else x.transpose(0, 1)).float()          # [H][N][D]
    blk, off = row // G, row % G
    first = torch.full((scale.shape[1],), G, device=x.device).scatter_reduce(0, blk, off, "amin")
    lead = blk[off == first[blk]]                                    # one entry a block
    r0 = first[lead]
    a = torch.where(x.isfinite(), x, 0.0).abs().amax(2)
    need = torch.zeros_like(scale).scatter_reduce(1, blk.expand(H, -1), a, "amax")[:, lead]
    s_old = torch.where(r0 == 0, 0.0, scale[:, lead])
    s_new = torch.maximum(_pow2_scale(need), s_old)      # the scales held are powers of two
    ratio = s_old / s_new
    codes = cache.view(H, -1, G, cache.shape[2])
    old = codes.view(torch.uint8)[:, lead].view(FP8).float()
    keep = torch.arange(G, device=x.device)[None, :, None] < r0[:, None, None]
    old = torch.where(keep, old * ratio[:, :, None, None], old)
    codes.view(torch.uint8)[:, lead] = old.to(FP8).view(torch.uint8)
    scale[:, lead] = s_new
    q = (x / scale[:, blk][:, :, None]).clamp(-E4M3_MAX, E4M3_MAX)
    cache.view(torch.uint8)[:, row] = q.to(FP8).view(torch.uint8)


def _plain_attn(st):
    q, L, W = st["q"].float(), st["seq_lens"].long(), st["window"]
    B, Hq, D = q.shape
    H = st["Hkv"]
    ps = st["page"]
    j = torch.arange(st["max_pages"] * ps, device=q.device)
    keep = j[None] < L[:, None]
    if W > 0:
        keep &= j[None] >= L[:, None] - W
    row = _rows(st, st["batch_idx"].long()[:, None], j[None].expand(B, -1)).clamp(min=0)
    sk = st["k_scale"][:, row // st["block"]]                        # [H][B][T]
    sv = st["v_scale"][:, row // st["block"]]
    k = st["k_cache"].view(torch.uint8)[:, row].view(FP8).float()    # [H][B][T][D]
    s = torch.einsum("hbgd,hbtd->hbgt", q.view(B, H, -1, D).permute(1, 0, 2, 3), k)
    del k
    s = s * (sk * st["scale"])[:, :, None]
    s = torch.where(keep[None, :, None], s, -math.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True))
    total = p.sum(-1, keepdim=True)
    v = st["v_cache"].view(torch.uint8)[:, row].view(FP8).float()
    p = torch.where(keep[None, :, None], p * sv[:, :, None], 0.0)
    o = torch.einsum("hbgt,hbtd->hbgd", p, v) / total
    st["out"].copy_(o.permute(1, 0, 2, 3).reshape(B, Hq, D))
    return st["out"]


# ------------------------------------------------------------------ exact ----

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "copy":
        pool, pairs = st["pool"].view(torch.uint8), st["pairs"].tolist()
        src = pool[:, :, [a for a, _ in pairs]].clone()
        pool[:, :, [b for _, b in pairs]] = src
        return st["pool"]
    if case["op"] == "append":
        return _exact_append(st)
    return _exact_attn(st)


def _exact_attn(st):
    """Row by row and kv head by kv head, in 64 bits."""
    B, Hq, D = st["q"].shape
    H, ps, G = st["Hkv"], st["page"], st["block"]
    out = torch.zeros((B, Hq, D), dtype=torch.float64, device="cuda")
    slots, lens = st["batch_idx"].tolist(), st["seq_lens"].tolist()
    for b in range(B):
        L = lens[b]
        lo = max(0, L - st["window"]) if st["window"] > 0 else 0
        t = torch.arange(lo, L, device="cuda")
        r = st["table"][slots[b]].long()[t // ps] * ps + t % ps
        k = st["k_cache"].view(torch.uint8)[:, r].view(FP8).double()
        v = st["v_cache"].view(torch.uint8)[:, r].view(FP8).double()
        k *= st["k_scale"][:, r // G].double()[:, :, None]
        v *= st["v_scale"][:, r // G].double()[:, :, None]
        q = st["q"][b].double().view(H, Hq // H, D) * float(st["scale"])
        p = torch.softmax(q @ k.transpose(1, 2), -1)
        out[b] = (p @ v).view(Hq, D)
    return out


def _round_e4m3(x):
    """Nearest e4m3 value (ties to even) of 64-bit values within +-448."""
    e = np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -6)))
    step = np.exp2(e - 3)
    return np.rint(x / step) * step


def _exact_append(st):
    """Block by block in 64 bits, from the definition: the block's scale grows to fit
    its largest value, earlier tokens follow it."""
    tbl = st["table"].cpu().numpy().astype(np.int64)
    slot, pos = st["batch_idx"].cpu().numpy(), st["input_pos"].cpu().numpy()
    ps, G = st["page"], st["block"]
    row = tbl[slot, pos // ps] * ps + pos % ps
    order = np.argsort(row, kind="stable")
    cuts = np.flatnonzero(np.diff(row[order] // G)) + 1
    out = []
    for x, cache, scale in ((st["k"], st["k_cache"], st["k_scale"]),
                            (st["v"], st["v_cache"], st["v_scale"])):
        x = x.double().cpu().numpy()
        x = x if st["prefill"] else x.transpose(1, 0, 2)
        codes = cache.double().cpu().numpy()
        s = scale.double().cpu().numpy()
        for idx in np.split(order, cuts):
            r = row[idx]
            b, r0 = r[0] // G, r.min()
            new = x[:, idx]
            amax = np.abs(new).max((1, 2))
            with np.errstate(divide="ignore"):
                need = np.exp2(np.maximum(np.ceil(np.log2(amax / E4M3_MAX)), MIN_EXP))
            held = np.zeros_like(need) if r0 % G == 0 else s[:, b]
            now = np.maximum(need, held)
            if r0 % G:
                codes[:, b * G:r0] = _round_e4m3(codes[:, b * G:r0] * (held / now)[:, None, None])
            s[:, b] = now
            codes[:, r] = _round_e4m3(new / now[:, None, None])
        out += [codes, s]
    return torch.from_numpy(out[0]), torch.from_numpy(out[2]), torch.from_numpy(out[1]), \
        torch.from_numpy(out[3])
