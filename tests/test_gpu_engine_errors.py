"""DecodeGraphs.errors (GPU): what the steps reported, once, and workspaces that are ready
again after a step whose waits gave up."""
import numpy as np
import pytest
import torch

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


@pytest.mark.parametrize("q8", [False, True])
def test_errors_are_told_once_and_workspaces_reset(dev, q8):
    rng = np.random.default_rng(5)
    Hq, Hkv, D, ps, P, mp = 8, 2, 128, 64, 300, 64
    spec = engine.LayerSpec(D, 1e6)
    pt = pkv.PageTable(4, ps, P, mp, device=dev)
    if q8:
        kc, vc, ks, vs = engine.alloc_cache_q8(Hkv, P, ps, D, dev)
    else:
        (kc, vc), ks, vs = engine.alloc_cache(Hkv, P, ps, D, dev), None, None
    lens = [4000, 700, 30]
    slots = [pt.assign(L + 1) for L in lens]
    i32 = dict(dtype=torch.int32, device=dev)
    for s, L in zip(slots, lens):
        k, v = (wl.randn_bf16(rng, (Hkv, L, D)).to(dev) for _ in range(2))
        args = (k, v, torch.full((L,), s, **i32), torch.arange(L, **i32), pt.dev_table,
                pt.n_slots, mp, ps, P, kc, vc)
        pkv.kv_append_prefill_q8(*args, ks, vs) if q8 else pkv.kv_append_prefill(*args)
    graphs = engine.DecodeGraphs(spec, pt, kc, vc, Hq, 4, dev, k_scale=ks, v_scale=vs)
    q, k, v = (wl.randn_bf16(rng, (3, h, D)).to(dev) for h in (Hq, Hkv, Hkv))
    bidx, pos = torch.tensor(slots, **i32), torch.tensor(lens, **i32)
    step = lambda: graphs.step(q, k, v, bidx, pos).clone()
    want = step()
    assert graphs.errors() == 0 and torch.equal(step(), want)
    # what a step whose waits gave up leaves: the bit, and words of its parts
    graphs.err.fill_(pkv.PKV_ERR_TIMEOUT)
    for w in graphs.ws.values():
        w.buf.random_(1, 255)
    assert graphs.errors() == pkv.PKV_ERR_TIMEOUT
    assert not any(w.buf.any() for w in graphs.ws.values())
    assert torch.equal(step(), want) and graphs.errors() == 0
    # an entry that names no page: told once
    row = pt.dev_table[slots[1], 2].clone()
    pt.dev_table[slots[1], 2] = -1
    step()
    assert graphs.errors() == pkv.PKV_ERR_PAGE_NEG and graphs.errors() == 0
    pt.dev_table[slots[1], 2] = row
    assert torch.equal(step(), want) and graphs.errors() == 0


def test_reset_of_a_workspace_of_its_own(dev):
    for w in (engine.AttnWorkspaceQ8(8, 2, 64, dev),
              engine.AttnWorkspace(2, 8, 2, 64, 40, 64, 0, dev),
              engine.AttnWorkspace(2, 8, 2, 64, 1, 64, 0, dev)):
        if w.buf is not None:
            w.buf.fill_(3)
        w.reset()
        assert w.buf is None or not w.buf.any()
