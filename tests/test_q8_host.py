"""Refusals of the 8-bit cache's calls, none of which needs a GPU: the binding's checks
of tensors, and the library's own checks on pointers that are never followed."""
import ctypes

import pytest
import torch

pkv = pytest.importorskip("paged_kv_decode_pagetable_gb300")
FP8 = torch.float8_e4m3fn
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    return pkv.load_library()


def append_args(**kw):
    H, D, ps, P, G, B = (kw.get(k, d) for k, d in (("H", 2), ("D", 64), ("ps", 16), ("P", 4),
                                                   ("G", 8), ("B", 3)))
    return dict(k=torch.zeros((B, H, D), dtype=BF16), v=torch.zeros((B, H, D), dtype=BF16),
                batch_idx=torch.ones(B, dtype=torch.int32),
                input_pos=torch.zeros(B, dtype=torch.int32),
                dev_table=torch.zeros((3, 2), dtype=torch.int32), n_slots=3, max_pages_per_seq=2,
                page_size=ps, n_pages=P, k_cache=torch.zeros((H, P * ps, D), dtype=FP8),
                v_cache=torch.zeros((H, P * ps, D), dtype=FP8),
                k_scale=torch.zeros((H, P * ps // G)), v_scale=torch.zeros((H, P * ps // G)))


@pytest.mark.parametrize("change,match", [
    (dict(k=torch.zeros((3, 2, 64))), "k must be a contiguous bfloat16"),
    (dict(k=torch.zeros((3, 64, 2), dtype=BF16).transpose(1, 2)), "k must be a contiguous"),
    (dict(v=torch.zeros((3, 1, 64), dtype=BF16)), "one shape"),
    (dict(k=torch.zeros((6, 64), dtype=BF16), v=torch.zeros((6, 64), dtype=BF16)), "one shape"),
    (dict(k_cache=torch.zeros((2, 64, 64))), "k_cache must be a contiguous float8"),
    (dict(k_cache=torch.zeros((2, 64, 64), dtype=torch.uint8)), "k_cache must be"),
    (dict(v_cache=torch.zeros((2, 64, 64), dtype=torch.float8_e5m2)), "v_cache must be"),
    (dict(v_cache=torch.zeros((2, 32, 64), dtype=FP8)), "must both hold"),
    (dict(k_cache=torch.zeros((1, 64, 64), dtype=FP8)), "must both hold"),
    (dict(k_scale=torch.zeros((2, 8), dtype=torch.float64)), "k_scale must be"),
    (dict(v_scale=torch.zeros((2, 4))), "k_scale and v_scale"),
    (dict(k_scale=torch.zeros((1, 8)), v_scale=torch.zeros((1, 8))), "k_scale and v_scale"),
    (dict(k_scale=torch.zeros((2, 7)), v_scale=torch.zeros((2, 7))), "k_scale and v_scale"),
    (dict(k_scale=torch.zeros((2, 0)), v_scale=torch.zeros((2, 0))), "k_scale and v_scale"),
    (dict(input_pos=torch.zeros(3, dtype=torch.int64)), "input_pos must be"),
    (dict(batch_idx=torch.ones(3)), "batch_idx must be"),
    (dict(input_pos=torch.zeros(2, dtype=torch.int32)), "for every token"),
    (dict(batch_idx=torch.zeros(2, dtype=torch.int32)), "for every token"),
    (dict(input_pos=None), "for every token"), (dict(dev_table=None), "dev_table must be"),
    (dict(n_slots=4), "dev_table must be"), (dict(max_pages_per_seq=3), "dev_table must be"),
    (dict(n_pages=5), "must both hold"),
    (dict(), "current CUDA device")])
def test_append_binding_refusals(lib, change, match):
    with pytest.raises(pkv.BadArgError, match=match):
        pkv.kv_append_q8(**{**append_args(), **change})


def test_prefill_layout_is_told_apart(lib):
    with pytest.raises(pkv.BadArgError, match="heads or head dim"):
        pkv.kv_append_prefill_q8(**append_args())
    a = append_args()
    a["k"] = a["v"] = torch.zeros((2, 3, 64), dtype=BF16)
    with pytest.raises(pkv.BadArgError, match="heads or head dim"):
        pkv.kv_append_q8(**a)
    with pytest.raises(pkv.BadArgError, match="current CUDA device"):
        pkv.kv_append_prefill_q8(**a)


A = 1 << 20        # a 16-byte aligned address that nothing follows
APPEND = dict(k=A, v=A, batch_idx=A, input_pos=A, B=3, dev_table=A, n_slots=3, max_pages=2,
              page_size=16, n_pages=4, scale_block=8, k_cache=A, v_cache=A, k_scale=A, v_scale=A,
              Hkv=2, D=64, err=None, stream=None)


@pytest.mark.parametrize("change", [
    dict(B=-1), dict(Hkv=0), dict(D=0), dict(D=8), dict(D=24), dict(page_size=0), dict(n_pages=0),
    dict(n_slots=0), dict(max_pages=0), dict(scale_block=0), dict(scale_block=3),
    dict(scale_block=32), dict(page_size=12, scale_block=8), dict(scale_block=-8), dict(k=None),
    dict(v=None), dict(input_pos=None), dict(dev_table=None), dict(k_cache=None),
    dict(v_cache=None), dict(k_scale=None), dict(v_scale=None), dict(k=A + 2), dict(v=A + 8),
    dict(k_cache=A + 1), dict(v_cache=A + 8), dict(D=1 << 28, page_size=64, scale_block=64)])
def test_append_library_refusals(lib, change):
    for fn in (lib.kv_append_q8, lib.kv_append_prefill_q8):
        assert fn(*{**APPEND, **change}.values()) == pkv.PKV_E_BAD_ARG
        assert b"kv_append" in lib.pkv_last_error()
    assert lib.kv_append_q8(*{**APPEND, "B": 0}.values()) == pkv.PKV_OK


def attn_args(B=2, Hq=4, Hkv=2, D=64, ps=16, P=4, G=8):
    n = pkv.paged_decode_attn_q8_workspace(Hq, Hkv, D)
    return dict(q=torch.zeros((B, Hq, D), dtype=BF16),
                k_cache=torch.zeros((Hkv, P * ps, D), dtype=FP8),
                v_cache=torch.zeros((Hkv, P * ps, D), dtype=FP8),
                k_scale=torch.zeros((Hkv, P * ps // G)), v_scale=torch.zeros((Hkv, P * ps // G)),
                dev_table=torch.zeros((3, 2), dtype=torch.int32), n_slots=3, max_pages_per_seq=2,
                page_size=ps, n_pages=P, batch_idx=torch.ones(B, dtype=torch.int32),
                seq_lens=torch.ones(B, dtype=torch.int32), window=0, scale=0.125,
                workspace=torch.zeros(n, dtype=torch.uint8),
                out=torch.zeros((B, Hq, D), dtype=BF16))


@pytest.mark.parametrize("change,match", [
    (dict(q=torch.zeros((2, 4, 64))), "q must be"),
    (dict(out=torch.zeros((2, 4, 32), dtype=BF16)), "differ in shape"),
    (dict(out=torch.zeros((1, 4, 64), dtype=BF16)), "differ in shape"),
    (dict(q=torch.zeros((2, 4, 32), dtype=BF16), out=torch.zeros((2, 4, 32), dtype=BF16)),
     "differ in shape"),
    (dict(workspace=None), "workspace is missing"), (dict(seq_lens=None), "for every row"),
    (dict(seq_lens=torch.ones(2, dtype=torch.int64)), "seq_lens must be"),
    (dict(seq_lens=torch.ones(1, dtype=torch.int32)), "for every row"),
    (dict(batch_idx=torch.ones(1, dtype=torch.int32)), "for every row"),
    (dict(dev_table=None), "dev_table must be"), (dict(n_slots=4), "dev_table must be"),
    (dict(n_pages=3), "must both hold"),
    (dict(k_cache=torch.zeros((2, 64, 64), dtype=torch.uint8)), "k_cache must be"),
    (dict(), "current CUDA device")])
def test_attn_binding_refusals(lib, change, match):
    with pytest.raises(pkv.BadArgError, match=match):
        pkv.paged_decode_attn_q8(**{**attn_args(), **change})


ATTN = dict(q=A, k_cache=A, v_cache=A, k_scale=A, v_scale=A, dev_table=A, n_slots=3, max_pages=2,
            page_size=16, n_pages=4, scale_block=8, batch_idx=A, seq_lens=A, window=0,
            scale=0.125, B=2, Hq=4, Hkv=2, D=64, workspace=A, workspace_bytes=1 << 40, out=A,
            err=None, stream=None)


@pytest.mark.parametrize("change", [
    dict(D=32), dict(D=96), dict(D=0), dict(Hq=3), dict(Hq=18), dict(Hq=1), dict(Hkv=0),
    dict(page_size=4, scale_block=4), dict(page_size=24), dict(page_size=0), dict(scale_block=0),
    dict(scale_block=3), dict(scale_block=32), dict(B=-1), dict(B=513), dict(n_slots=0),
    dict(n_pages=0), dict(max_pages=0), dict(max_pages=1 << 27), dict(n_pages=1 << 27),
    dict(max_pages=1 << 26, Hkv=64, Hq=64), dict(scale=0.0), dict(scale=-1.0),
    dict(scale=float("nan")), dict(scale=float("inf")), dict(q=None), dict(k_cache=None),
    dict(v_cache=None), dict(k_scale=None), dict(v_scale=None), dict(dev_table=None),
    dict(seq_lens=None), dict(out=None), dict(q=A + 8), dict(out=A + 2), dict(k_cache=A + 4),
    dict(v_cache=A + 8), dict(workspace=None), dict(workspace=A + 8), dict(workspace_bytes=64)])
def test_attn_library_refusals(lib, change):
    a = {**ATTN, **change}
    a["workspace_bytes"] = ctypes.c_size_t(a["workspace_bytes"])
    assert lib.paged_decode_attn_q8(*a.values()) == pkv.PKV_E_BAD_ARG
    assert b"paged_decode_attn_q8" in lib.pkv_last_error()


def test_workspace_size(lib):
    assert pkv.paged_decode_attn_q8_workspace(8, 2, 96) == 0
    assert pkv.paged_decode_attn_q8_workspace(9, 2, 64) == 0
    assert pkv.paged_decode_attn_q8_workspace(18, 2, 64) == 0
    for D in (64, 128, 256, 512):
        a, b = (pkv.paged_decode_attn_q8_workspace(h, 1, D) for h in (1, 8))
        assert 0 < a < b and a % 4 == 0
        assert b == pkv.paged_decode_attn_q8_workspace(64, 8, D)   # by the group alone
    assert lib.paged_decode_attn_q8(*{**ATTN, "B": 0}.values()) == pkv.PKV_OK


def test_more_heads_than_a_call_takes(lib):
    assert pkv.paged_decode_attn_q8_workspace(65535, 65535, 64) > 0
    assert pkv.paged_decode_attn_q8_workspace(65536, 65536, 64) == 0
