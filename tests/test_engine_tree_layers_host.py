"""engine.tree_layer_step asks for the norm and rotation that decode_layer_step gives the same
layer: keys of both lie in one cache. No GPU: the library's calls are recorded."""
import itertools

import pytest
import torch

pkv = pytest.importorskip("paged_kv_decode_pagetable_gb300")
from paged_kv_decode_pagetable_gb300 import engine  # noqa: E402

I32 = torch.int32
D = 64


def bf16(*s):
    return torch.zeros(s, dtype=torch.bfloat16)


@pytest.mark.parametrize("qk_norm,rope,gains", list(itertools.product([0, 1], [0, 1], [0, 1])))
def test_norm_and_rotation(qk_norm, rope, gains, monkeypatch):
    spec = engine.LayerSpec(head_dim=D, theta=1e4, qk_norm=bool(qk_norm), rope=bool(rope))
    pt = type("Geometry", (), dict(dev_table=torch.zeros((3, 2), dtype=I32), n_slots=3,
                                   max_pages_per_seq=2, page_size=16, n_pages=4))
    g = (bf16(D), bf16(D)) if gains else (None, None)
    caches, i32 = (bf16(2, 64, D), bf16(2, 64, D)), torch.zeros(2, dtype=I32)
    decode = {}
    for name in ("qk_norm_rope", "kv_append", "paged_decode_attn"):
        monkeypatch.setattr(engine, name, lambda *a, name=name, **k: decode.update({name: a}))
    ws = type("Workspace", (), dict(splits=0, buf=None))
    engine.decode_layer_step(spec, pt, *caches, bf16(2, 4, D), bf16(2, 2, D), bf16(2, 2, D), i32,
                             i32, i32, bf16(2, 4, D), ws, *g, fused=False)
    tree = {}

    class Recorder:
        def __getattr__(self, name):
            def call(record):
                tree[name] = pkv._RECORDS[name.removesuffix("_args")].unpack(record)
                return pkv.PKV_OK
            return call
    monkeypatch.setattr(pkv, "_lib", Recorder())
    monkeypatch.setattr(pkv, "_on_device", lambda *t: None)
    tws = type("Workspace", (), dict(buf=torch.zeros(1, dtype=torch.uint8)))
    engine.tree_layer_step(spec, pt, *caches, bf16(5, 4, D), bf16(5, 2, D), bf16(5, 2, D), i32, i32,
                           torch.zeros(3, dtype=I32), torch.zeros(5, dtype=I32), bf16(5, 4, D),
                           bf16(5, 4, D), tws, *g)
    record = tree["tree_qkv_norm_rope_append_args"]
    gq, gk, rotary = record[6], record[7], record[14]
    norm = "qk_norm_rope" in decode and decode["qk_norm_rope"][2] is not None
    assert (gq != 0, gk != 0) == (norm, norm)
    assert rotary == (D if "qk_norm_rope" in decode else 0)


@pytest.mark.parametrize("theta", [0.0, float("inf"), -1.0])
def test_a_layer_without_rotation_needs_no_theta(theta, monkeypatch):
    spec = engine.LayerSpec(head_dim=D, theta=theta, rope=False)
    got = {}
    monkeypatch.setattr(engine, "tree_qkv_norm_rope_append", lambda *a, **k: got.update(a=a))
    monkeypatch.setattr(engine, "paged_tree_attn", lambda *a, **k: None)
    pt = type("Geometry", (), dict(dev_table=None, n_slots=3, max_pages_per_seq=2, page_size=16,
                                   n_pages=4))
    engine.tree_layer_step(spec, pt, *[None] * 11, type("Workspace", (), dict(buf=None)))
    theta, rotary = got["a"][9], got["a"][11]
    assert rotary == 0 and 2.0 ** -56 <= theta < float("inf")
