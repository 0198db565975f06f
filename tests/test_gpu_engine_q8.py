"""The layer step over an 8-bit cache (GPU): graph buckets equal the eager chain, and
a run of a group of samples as it is used: prompt appended, samples forked, decoded,
the cache compacted, decoded on, against the oracle fed the same tokens."""
import numpy as np
import pytest
import torch

import oracle
import workloads as wl

pytestmark = pytest.mark.gpu
pkv = pytest.importorskip("paged_kv_decode_pagetable_gb300")
from paged_kv_decode_pagetable_gb300 import engine  # noqa: E402


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pkv.load_library()
    return torch.device("cuda:0")


def same(a, b):
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("spec", [
    engine.LayerSpec(128, 1e6, 0, True, True),
    engine.LayerSpec(256, 1e4, 512, True, True, v_norm=True),
    engine.LayerSpec(512, 1e6, 0, True, True, rotary_dims=128, v_norm=True, k_eq_v=True),
    engine.LayerSpec(64, 1e4, 0, False, False)])
def test_bucketed_graph_replay_equals_eager(dev, spec):
    rng = np.random.default_rng(91)
    max_bs, Hq, Hkv, D, ps, P, mp = 8, 8, 2, spec.head_dim, 64, 120, 16
    pt = pkv.PageTable(max_bs, ps, P, mp, device=dev)
    caches = engine.alloc_cache_q8(Hkv, P, ps, D, dev, scale_block=16)
    gq, gk = wl.gamma_bf16(rng, D).to(dev), wl.gamma_bf16(rng, D).to(dev)
    lens = rng.integers(30, 700, size=7)
    slots = [pt.assign(int(L) + 4) for L in lens]
    i32 = dict(dtype=torch.int32, device=dev)
    for s, L in zip(slots, lens):                # the prompts
        k, v = (wl.randn_bf16(rng, (Hkv, int(L), D)).to(dev) for _ in range(2))
        pkv.kv_append_prefill_q8(k, v, torch.full((int(L),), s, **i32), torch.arange(int(L), **i32),
                                 pt.dev_table, pt.n_slots, mp, ps, P, *caches)
    graphs = engine.DecodeGraphs(spec, pt, caches[0], caches[1], Hq, max_bs, dev, gq, gk,
                                 k_scale=caches[2], v_scale=caches[3])
    for rows in ([0, 3, 4], [1, 2, 6, 5, 0], [6]):
        B = len(rows)
        q, k, v = (wl.randn_bf16(rng, (B, h, D)).to(dev) for h in (Hq, Hkv, Hkv))
        bidx = torch.tensor([slots[r] for r in rows], **i32)
        pos = torch.tensor([int(lens[r]) for r in rows], **i32)
        eager = [c.clone() for c in caches]
        out = torch.empty((B, Hq, D), dtype=torch.bfloat16, device=dev)
        err = torch.zeros(1, **i32)
        engine.decode_layer_step(spec, pt, eager[0], eager[1], q.clone(), k.clone(), v.clone(),
                                 bidx, pos, pos + 1, out, engine.AttnWorkspaceQ8(Hq, Hkv, D, dev),
                                 gq, gk, err=err, k_scale=eager[2], v_scale=eager[3])
        got = graphs.step(q, k, v, bidx, pos)
        torch.cuda.synchronize()
        assert pkv.pkv_read_error_word(err) == 0 and pkv.pkv_read_error_word(graphs.err) == 0
        # a bucket with padding rows cuts the work elsewhere: same sums, other order
        if B in graphs.ladder:
            assert same(got, out)
        else:
            assert (got.float() - out.float()).abs().max() <= 2 ** -8 * max(1.0, out.abs().max())
        assert all(same(a, b) for a, b in zip(caches, eager))
        for r in rows:
            lens[r] += 1


def test_a_group_of_samples_end_to_end(dev):
    rng = np.random.default_rng(92)
    Hq, Hkv, D, ps, G, P, mp = 8, 2, 128, 16, 8, 40, 8
    spec = engine.LayerSpec(D, 1e4, 0, False, False)       # no norm, no rotation
    pt = pkv.PageTable(5, ps, P, mp, device=dev)
    kc, vc, ks, vs = engine.alloc_cache_q8(Hkv, P, ps, D, dev, scale_block=G)
    caches = [kc, vc, ks, vs]
    i32 = dict(dtype=torch.int32, device=dev)
    err = torch.zeros(1, **i32)
    ws = engine.AttnWorkspaceQ8(Hq, Hkv, D, dev)
    kv = {}                                                # rid -> tokens [n][2][Hkv][D]
    filler = pt.assign(7 * ps)

    def prefill(batch):
        for s in batch:
            x = wl.randn_bf16(rng, (2, Hkv, s.prompt_len, D))
            kv[s.rid] = [x[:, :, t] for t in range(s.prompt_len)]
            n = s.prompt_len
            pkv.kv_append_prefill_q8(x[0].to(dev), x[1].to(dev), torch.full((n,), s.slot, **i32),
                                     torch.arange(n, **i32), pt.dev_table, pt.n_slots, mp, ps, P,
                                     kc, vc, ks, vs, err)

    worst = 0.0

    def decode(batch):
        nonlocal worst
        B = len(batch)
        x = wl.randn_bf16(rng, (2, B, Hkv, D)) * 2
        q = wl.randn_bf16(rng, (B, Hq, D))
        for b, s in enumerate(batch):
            kv[s.rid].append(x[:, b])
            assert len(kv[s.rid]) == s.total_length
        slots = torch.tensor([s.slot for s in batch], **i32)
        pos = torch.tensor([s.total_length - 1 for s in batch], **i32)
        out = torch.empty((B, Hq, D), dtype=torch.bfloat16, device=dev)
        engine.decode_layer_step(spec, pt, kc, vc, q.to(dev), x[0].to(dev), x[1].to(dev), slots,
                                 pos, pos + 1, out, ws, err=err, k_scale=ks, v_scale=vs)
        got = out.cpu().double().numpy()
        for b, s in enumerate(batch):
            n = s.total_length
            dense = []
            for a in (0, 1):                # the sequence alone, in a cache of its own
                codes, scale = np.zeros((Hkv, mp * ps, D)), np.zeros((Hkv, mp * ps // G))
                t = torch.stack([y[a] for y in kv[s.rid]]).double().numpy()
                own = np.arange(mp)[None].repeat(2, 0)
                for i in ([(0, s.prompt_len)] + [(j, j + 1) for j in range(s.prompt_len, n)]):
                    oracle.kv_append_q8(codes, scale, t[i[0]:i[1]], own, np.ones(i[1] - i[0], int),
                                        np.arange(*i), ps, mp, G)
                dense.append(oracle.dequantise(codes, scale, G)[:, :n])
            for h in range(Hq):
                k, v = dense[0][h // (Hq // Hkv)], dense[1][h // (Hq // Hkv)]
                o, _ = oracle.decode_attention_row(q[b, h].double().numpy(), k, v, D ** -0.5)
                # output 2^-8, weights 2^-11 of the weighted |v| <= max |v|, scores to 2^-14
                bound = 2.0 ** -8 * np.abs(o) + 2.0 ** -10 * np.abs(v).max()
                e = np.abs(got[b, h] - o)
                assert (e <= bound).all(), (s.rid, h, e.max())
                worst = max(worst, float((e / bound).max()))

    cb = engine.ContinuousBatcher(pt, [engine.Sequence(0, 45, 30)], prefill, decode)
    cb.step()
    new = cb.fork(cb.running[0], [1, 2, 3], caches)
    assert all(f.slot > 0 for f in new)
    for f in new:
        kv[f.rid] = list(kv[0])
    pt.free(filler)
    for i in range(12):
        cb.step()
    assert engine.compact_cache(pt, caches) > 0
    cb.run()
    assert len(cb.done) == 4 and pkv.pkv_read_error_word(err) == 0 and worst > 0
