"""Refusals of the 8-bit cache's calls: each is an error on the host, before any
launch (no GPU needed: the tensors are never reached)."""
import pytest
import torch

pkv = pytest.importorskip("paged_kv_decode_pagetable_gb300")
FP8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def lib():
    pkv.load_library()


def aligned(shape, dtype):
    """A zeroed tensor whose data starts on a 16-byte boundary."""
    size = torch.empty(0, dtype=dtype).element_size()
    n = 1
    for s in shape:
        n *= s
    buf = torch.zeros(n * size + 32, dtype=torch.uint8)
    off = -buf.data_ptr() % 16
    return buf[off:off + n * size].view(dtype).view(shape)


def append_args(**kw):
    H, D, ps, P, G, B = (kw.get(k, d) for k, d in (("H", 2), ("D", 64), ("ps", 16), ("P", 4),
                                                   ("G", 8), ("B", 3)))
    a = dict(k=aligned((B, H, D), torch.bfloat16), v=aligned((B, H, D), torch.bfloat16),
             batch_idx=torch.ones(B, dtype=torch.int32), input_pos=torch.zeros(B, dtype=torch.int32),
             dev_table=torch.zeros((3, 2), dtype=torch.int32), n_slots=3, max_pages_per_seq=2,
             page_size=ps, n_pages=P, k_cache=aligned((H, P * ps, D), FP8),
             v_cache=aligned((H, P * ps, D), FP8), k_scale=torch.zeros((H, P * ps // G)),
             v_scale=torch.zeros((H, P * ps // G)))
    return a


@pytest.mark.parametrize("change", [
    dict(k=torch.zeros((3, 2, 64))), dict(k=aligned((3, 64, 2), torch.bfloat16).transpose(1, 2)),
    dict(v=aligned((3, 1, 64), torch.bfloat16)), dict(k_cache=torch.zeros((2, 64, 64))),
    dict(v_cache=aligned((2, 32, 64), FP8)), dict(k_cache=aligned((1, 64, 64), FP8)),
    dict(k_scale=torch.zeros((2, 8), dtype=torch.float64)), dict(v_scale=torch.zeros((2, 4))),
    dict(k_scale=torch.zeros((1, 8)), v_scale=torch.zeros((1, 8))),
    dict(k_scale=torch.zeros((2, 7)), v_scale=torch.zeros((2, 7))),
    dict(k_scale=torch.zeros((2, 0)), v_scale=torch.zeros((2, 0))),
    dict(k_scale=torch.zeros((2, 2)), v_scale=torch.zeros((2, 2))),      # 32 rows > a page
    dict(input_pos=torch.zeros(3, dtype=torch.int64)), dict(batch_idx=torch.ones(3)),
    dict(n_pages=5), dict(n_slots=0), dict(max_pages_per_seq=0), dict(page_size=0),
    dict(dev_table=None), dict(input_pos=None)])
def test_append_refusals(change):
    a = {**append_args(), **change}
    with pytest.raises(pkv.BadArgError):
        pkv.kv_append_q8(**a)


def test_append_refuses_odd_sizes_and_alignment():
    with pytest.raises(pkv.BadArgError):
        pkv.kv_append_q8(**append_args(D=24))
    with pytest.raises(pkv.BadArgError):
        pkv.kv_append_q8(**append_args(ps=12, G=3))        # not a power of two
    a = append_args()
    buf = aligned((2 * 64 * 64 + 16,), FP8)
    a["k_cache"] = buf[8:8 + 2 * 64 * 64].view(2, 64, 64)
    with pytest.raises(pkv.BadArgError):
        pkv.kv_append_q8(**a)
    with pytest.raises(pkv.BadArgError):                    # head-major shape expected
        pkv.kv_append_prefill_q8(**append_args())
    a = append_args(B=0)
    pkv.kv_append_q8(**a)                                   # no rows: nothing to do


def attn_args(B=2, Hq=4, Hkv=2, D=64, ps=16, P=4, G=8):
    n = pkv.paged_decode_attn_q8_workspace(Hq, Hkv, D)
    return dict(q=aligned((B, Hq, D), torch.bfloat16), k_cache=aligned((Hkv, P * ps, D), FP8),
                v_cache=aligned((Hkv, P * ps, D), FP8), k_scale=torch.zeros((Hkv, P * ps // G)),
                v_scale=torch.zeros((Hkv, P * ps // G)),
                dev_table=torch.zeros((3, 2), dtype=torch.int32), n_slots=3, max_pages_per_seq=2,
                page_size=ps, n_pages=P, batch_idx=torch.ones(B, dtype=torch.int32),
                seq_lens=torch.ones(B, dtype=torch.int32), window=0, scale=0.125,
                workspace=aligned((max(n, 16),), torch.uint8),
                out=aligned((B, Hq, D), torch.bfloat16))


@pytest.mark.parametrize("change", [
    dict(q=torch.zeros((2, 4, 64))), dict(out=aligned((2, 4, 32), torch.bfloat16)),
    dict(out=aligned((1, 4, 64), torch.bfloat16)), dict(scale=0.0), dict(scale=-1.0),
    dict(scale=float("nan")), dict(scale=float("inf")), dict(workspace=None),
    dict(workspace=aligned((64,), torch.uint8)), dict(seq_lens=None),
    dict(seq_lens=torch.ones(2, dtype=torch.int64)), dict(dev_table=None), dict(n_slots=0),
    dict(n_pages=3), dict(max_pages_per_seq=1 << 27),
    dict(k_scale=torch.zeros((2, 2)), v_scale=torch.zeros((2, 2))),
    dict(k_cache=aligned((2, 64, 64), FP8).view(torch.uint8))])
def test_attn_refusals(change):
    with pytest.raises(pkv.BadArgError):
        pkv.paged_decode_attn_q8(**{**attn_args(), **change})


@pytest.mark.parametrize("shape", [dict(D=32), dict(D=96), dict(Hq=3), dict(Hq=18), dict(Hq=1),
                                   dict(ps=4, G=4), dict(ps=24, G=8), dict(B=513)])
def test_attn_refuses_unsupported_shapes(shape):
    with pytest.raises(pkv.BadArgError):
        pkv.paged_decode_attn_q8(**attn_args(**shape))


def test_workspace_size():
    assert pkv.paged_decode_attn_q8_workspace(8, 2, 96) == 0
    assert pkv.paged_decode_attn_q8_workspace(9, 2, 64) == 0
    assert pkv.paged_decode_attn_q8_workspace(18, 2, 64) == 0
    for D in (64, 128, 256, 512):
        a, b = (pkv.paged_decode_attn_q8_workspace(h, 1, D) for h in (1, 8))
        assert 0 < a < b and a % 4 == 0
        assert b == pkv.paged_decode_attn_q8_workspace(64, 8, D)   # by the group alone
    pkv.paged_decode_attn_q8(**attn_args(B=0))                     # no rows: nothing to do
