"""Arguments that the 8-bit cache's bindings refuse as bad arguments, whatever is wrong
with them (no GPU needed)."""
import pytest
import torch

from test_q8_host import BF16, append_args, attn_args

pkv = pytest.importorskip("paged_kv_decode_pagetable_gb300")


@pytest.fixture(scope="module", autouse=True)
def lib():
    pkv.load_library()


APPEND = [dict([(n, x)]) for n in ("k", "v", "k_cache", "v_cache", "k_scale", "v_scale")
          for x in (None, 1 << 20, [1.0])] + [
    dict(input_pos=1 << 20), dict(batch_idx=1 << 20), dict(dev_table=1 << 20),
    dict(k=torch.zeros(6, dtype=BF16), v=torch.zeros(6, dtype=BF16)),
    dict(err_word=torch.zeros(1, dtype=torch.int64)), dict(err_word=torch.zeros(1)),
    dict(err_word=torch.zeros(0, dtype=torch.int32)), dict(err_word=[0])]


@pytest.mark.parametrize("change", APPEND)
def test_append(change):
    for call in (pkv.kv_append_q8, pkv.kv_append_prefill_q8):
        a = append_args()
        if call is pkv.kv_append_prefill_q8:
            a["k"], a["v"] = (x.transpose(0, 1).contiguous() for x in (a["k"], a["v"]))
        with pytest.raises(pkv.BadArgError) as e:
            call(**{**a, **change})
        assert "CUDA device" not in str(e.value)  # refused for what it is


ATTN = [dict([(n, x)]) for n in ("q", "out", "k_cache", "v_cache", "k_scale", "v_scale",
                                 "workspace") for x in (None, 1 << 20, [1.0])] + [
    dict(q=torch.zeros((2, 256), dtype=BF16)), dict(q=torch.zeros((2, 4, 64, 1), dtype=BF16)),
    dict(q=torch.zeros(8, dtype=BF16)), dict(out=torch.zeros((2, 256), dtype=BF16)),
    dict(seq_lens=1 << 20), dict(batch_idx=1 << 20), dict(dev_table=1 << 20),
    dict(err_word=torch.zeros(1, dtype=torch.int64)), dict(err_word=torch.zeros(1)),
    dict(err_word=torch.zeros(0, dtype=torch.int32)), dict(err_word=[0]),
    dict(workspace=torch.zeros(1, dtype=torch.uint8).expand(1 << 24)),
    dict(workspace=torch.zeros(1 << 22, dtype=torch.uint8)[::2])]


@pytest.mark.parametrize("change", ATTN)
def test_attention(change):
    with pytest.raises(pkv.BadArgError) as e:
        pkv.paged_decode_attn_q8(**{**attn_args(), **change})
    assert "CUDA device" not in str(e.value)
