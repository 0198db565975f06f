"""The bf16 decode kernels over rings in full use (GPU): a tile read after its ring entry
was refilled would show as calls that differ. Repeated attention calls and fused steps over
long rows agree bit for bit, and with a 64-bit computation."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
pkv = pytest.importorskip("paged_kv_decode_pagetable_gb300")


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pkv.load_library()
    return torch.device("cuda:0")


class Rows:
    def __init__(self, dev, D, ps, Hq, Hkv, lens):
        g = torch.Generator(device=dev).manual_seed(D + ps)
        rnd = lambda *s: torch.randn(s, generator=g, device=dev).bfloat16()
        i32 = lambda a: torch.from_numpy(np.asarray(a, np.int32)).to(dev)
        self.B, self.D, self.ps, self.Hq, self.Hkv, self.L = len(lens), D, ps, Hq, Hkv, lens
        nb = -(-np.asarray(lens) // ps)
        self.P, self.max_pages, self.n_slots = int(nb.sum()) + 2, int(nb.max()), len(lens) + 1
        table = np.full((self.n_slots, self.max_pages), -1, np.int32)
        table[0] = 0
        pages = np.split(np.random.default_rng(0).permutation(np.arange(1, self.P)),
                         np.cumsum(nb))
        for b in range(self.B):
            table[b + 1, :nb[b]] = pages[b]
        self.table, self.bidx, self.lens = i32(table), i32(np.arange(1, self.B + 1)), i32(lens)
        self.kc, self.vc = rnd(Hkv, self.P * ps, D), rnd(Hkv, self.P * ps, D)
        self.q, self.k, self.v = rnd(self.B, Hq, D), rnd(self.B, Hkv, D), rnd(self.B, Hkv, D)
        self.gq, self.gk = rnd(D), rnd(D)
        n = pkv.paged_decode_attn_workspace(self.B, Hq, D, pkv.paged_decode_attn_splits(
            self.B, Hkv, D, self.max_pages, ps))
        self.ws = torch.zeros(max(n, 16), dtype=torch.uint8, device=dev)
        self.geometry = (self.n_slots, self.max_pages, ps, self.P)

    def attend(self, out, q=None):
        pkv.paged_decode_attn(self.q if q is None else q, self.kc, self.vc, self.table,
                              *self.geometry, self.bidx, self.lens, 0, self.D ** -0.5, 0, self.ws,
                              out)

    def step(self, out):
        pkv.paged_decode_step(self.q, self.k, self.v, self.gq, self.gk, self.bidx, self.lens - 1,
                              1e6, 1e-6, self.table, *self.geometry, self.kc, self.vc, 0,
                              self.D ** -0.5, 0, self.ws, out)

    def row(self, b, q):
        """Row b in 64 bits, and a bound: the weights and the output are rounded to bf16
        (2^-8 relative each), the scores' fp32 error is far below that."""
        t = torch.arange(self.L[b], device=q.device)
        r = self.table[b + 1].long()[t // self.ps] * self.ps + t % self.ps
        k, v = self.kc[:, r].double(), self.vc[:, r].double()
        p = torch.softmax(q[b].double().view(self.Hkv, -1, self.D) * self.D ** -0.5
                          @ k.transpose(1, 2), -1)
        o, A = p @ v, p @ v.abs()
        return o.view(self.Hq, self.D), (2 ** -8 * o.abs() + 2 ** -7 * A).view(self.Hq, self.D)


@pytest.mark.parametrize("D,ps,G", [(64, 64, 8), (128, 64, 8), (128, 16, 4), (256, 64, 8),
                                    (256, 128, 4), (512, 64, 8)])
def test_repeated_calls_over_full_rings(dev, D, ps, G):
    r = Rows(dev, D, ps, 3 * G, 3, [29952, 28480, 29803])
    outs = torch.full((200,) + r.q.shape, float("nan"), dtype=torch.bfloat16, device=dev)
    for o in outs:
        r.attend(o)
    assert torch.isfinite(outs).all()
    assert all(torch.equal(o, outs[0]) for o in outs[1:])
    want, tol = r.row(1, r.q)
    assert ((outs[0][1].double() - want).abs() <= tol).all()
    assert not r.ws.any()


@pytest.mark.parametrize("D,ps,G", [(64, 64, 8), (128, 64, 4), (256, 64, 8), (512, 64, 8)])
def test_repeated_steps_over_full_rings(dev, D, ps, G):
    """A step appends the same token again and again, so all calls are alike; the chain of
    separate calls gives the same bits."""
    r = Rows(dev, D, ps, 3 * G, 3, [29952, 28480, 29803])
    outs = torch.full((100,) + r.q.shape, float("nan"), dtype=torch.bfloat16, device=dev)
    for o in outs:
        r.step(o)
    assert torch.isfinite(outs).all()
    assert all(torch.equal(o, outs[0]) for o in outs[1:])
    q, k, chain = r.q.clone(), r.k.clone(), torch.empty_like(outs[0])
    pkv.qk_norm_rope(q, k, r.gq, r.gk, r.lens - 1, 1e6, 1e-6)
    pkv.kv_append(k, r.v, r.bidx, r.lens - 1, r.table, *r.geometry, r.kc, r.vc)
    r.attend(chain, q)
    assert torch.equal(chain, outs[0])


@pytest.mark.parametrize("D", [64, 128, 256, 512])
def test_repeated_calls_over_many_rows(dev, D):
    """Units of every length one behind another: query stages are refilled as fast as
    entries."""
    lens = np.random.default_rng(D).integers(1, 1500, 120)
    r = Rows(dev, D, 64, 16, 2, [int(x) for x in lens])
    outs = torch.full((60,) + r.q.shape, float("nan"), dtype=torch.bfloat16, device=dev)
    for o in outs:
        r.attend(o)
    assert torch.isfinite(outs).all()
    assert all(torch.equal(o, outs[0]) for o in outs[1:])
    for b in (0, 57, 119):
        want, tol = r.row(b, r.q)
        assert ((outs[0][b].double() - want).abs() <= tol).all()
