"""Seeded drafted trees over a paged cache, and the bounds their results are held to."""
from __future__ import annotations

import numpy as np
import torch

import workloads as wl
from gpu_util import NAN_BF16, bits_to_f64, f64
from oracle import tree

BF16_STEP = 2.0 ** -8      # half a step of bf16, relative to the value


def random_tree(rng, n, width, roots=1):
    """Parents of n nodes: a chain (width 1), or each under one of the `width` before it."""
    par = [-1] * min(n, roots)
    while len(par) < n:
        i = len(par)
        par.append(i - int(rng.integers(1, min(i, width) + 1)))
    return par


class TreeCase:
    """B rows of ctx[b] tokens and a tree each, on pages drawn from a permutation; every
    cache row that no node can read holds NaN."""

    def __init__(self, rng, Hq, Hkv, D, ps, ctx, trees, window=0, slots=None, pad=0, scale=None,
                 max_pages=None):
        self.Hq, self.Hkv, self.D, self.ps, self.window = Hq, Hkv, D, ps, window
        self.B = len(ctx)
        self.ctx = np.array(ctx, np.int32)
        self.row_start = np.concatenate([[0], np.cumsum([len(t) for t in trees])]).astype(np.int32)
        self.N = int(self.row_start[-1])
        self.parents = np.array([p for t in trees for p in t] + [-1] * pad, np.int32)
        self.pad = pad
        self.slots = np.arange(1, self.B + 1, dtype=np.int32) if slots is None else np.array(
            slots, np.int32)
        self.n_slots = int(max([self.B, *self.slots])) + 1
        self.scale = D ** -0.5 if scale is None else scale
        need = [-(-(int(c) + len(t)) // ps) for c, t in zip(ctx, trees)]
        self.max_pages = max_pages or max(need + [1])
        self.P = sum(need) + 4
        self.table = np.full((self.n_slots, self.max_pages), -1, np.int32)
        self.table[0] = 0
        perm = iter(rng.permutation(np.arange(1, self.P)))
        readable = np.zeros(self.P * ps, bool)
        for b in range(self.B):
            if self.slots[b] == 0:
                continue
            for j in range(need[b]):
                self.table[self.slots[b], j] = next(perm)
            lo = 0 if window <= 0 else max(0, int(ctx[b]) - window + 1) if trees[b] else 0
            for j in range(lo, int(ctx[b]) + len(trees[b])):
                readable[tree.cache_row(self.table, self.slots[b], j, ps)] = True
        kc, vc = (wl.randn_bf16(rng, (Hkv, self.P * ps, D)).view(torch.int16).numpy().copy()
                  for _ in range(2))
        kc[:, ~readable], vc[:, ~readable] = NAN_BF16, NAN_BF16
        self.kc, self.vc = kc, vc
        self.q = wl.randn_bf16(rng, (self.N + pad, Hq, D))
        self.err = None

    def device(self, pkv, dev="cuda"):
        i32 = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(dev)  # noqa: E731
        self.t = dict(q=self.q.to(dev),
                      kc=torch.from_numpy(self.kc).view(torch.bfloat16).to(dev),
                      vc=torch.from_numpy(self.vc).view(torch.bfloat16).to(dev),
                      table=i32(self.table), slots=i32(self.slots), ctx=i32(self.ctx),
                      row_start=i32(self.row_start), parents=i32(self.parents))
        n = pkv.paged_tree_attn_workspace(self.Hq, self.Hkv, self.D)
        self.ws = torch.zeros(n, dtype=torch.uint8, device=dev)
        self.out = torch.full((self.N + self.pad, self.Hq, self.D), 7.0, dtype=torch.bfloat16,
                              device=dev)
        self.err = torch.zeros(1, dtype=torch.int32, device=dev)
        return self

    def call(self, pkv, ws=None, out=None, **kw):
        t = {**self.t, **kw}
        out = self.out if out is None else out
        pkv.paged_tree_attn(t["q"], t["kc"], t["vc"], t["table"], self.n_slots, self.max_pages,
                            self.ps, self.P, t["slots"], t["ctx"], t["row_start"], t["parents"],
                            self.window, self.scale, self.ws if ws is None else ws, out, self.err)
        return out

    def want(self):
        return tree.tree_attention(self.q.double().numpy(), bits_to_f64(self.kc),
                                   bits_to_f64(self.vc), self.table, self.slots, self.ctx,
                                   self.row_start, self.parents, self.window, self.scale, self.ps,
                                   weight_of=True)

    def check(self, pkv, out=None):
        out = self.call(pkv) if out is None else out
        torch.cuda.synchronize()
        assert int(self.err) == 0
        got = f64(out)
        check_attn(got[:self.N], *[x[:self.N] for x in self.want()])
        assert (got[self.N:] == 7.0).all()          # nodes of no row are left alone


def check_attn(got, ref, mass):
    """Each weight is rounded to bf16 once (half a step of its value), the result once; fp32
    scores and sums move a weight by less than 2^-13: |s| stays below 60, so D + 1 roundings
    of 2^-24 of it add up to less than 60 * 513 * 2^-24 < 2^-9 only if all fell the same way;
    the products' sum is kept in fp32 with relative error D 2^-24 of sum |q k| / sqrt(D) < 16,
    hence exp moves by < 16 * 512 * 2^-24 = 2^-11 at worst and is taken as that."""
    bound = BF16_STEP * (mass + np.abs(ref)) + 2.0 ** -11 * mass + 1e-30
    assert np.isfinite(got).all(), "non-finite output"
    bad = np.abs(got - ref) > bound
    assert not bad.any(), (int(bad.sum()), float((np.abs(got - ref) / bound).max()))
