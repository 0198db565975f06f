"""Refusals of the speculative calls, none of which needs a GPU: the binding's checks of
tensors, and the library's own checks on pointers that are never followed."""
import ctypes

import pytest
import torch

pkv = pytest.importorskip("paged_kv_decode_pagetable_gb300")
BF16, I32 = torch.bfloat16, torch.int32


@pytest.fixture(scope="module", autouse=True)
def lib():
    return pkv.load_library()


def i32(*shape):
    return torch.zeros(shape, dtype=I32)


def bf16(*shape):
    return torch.zeros(shape, dtype=BF16)


GEOMETRY = dict(dev_table=i32(3, 2), n_slots=3, max_pages_per_seq=2, page_size=16, n_pages=4)
ROWS = dict(batch_idx=i32(2), ctx_lens=i32(2), row_start=i32(3), parents=i32(5))


def append_args():
    return dict(q=bf16(5, 4, 64), k=bf16(5, 2, 64), v=bf16(5, 2, 64), gamma_q=bf16(64),
                gamma_k=bf16(64), **ROWS, theta=1e4, eps=1e-6, rotary_dims=None, v_norm=False,
                **GEOMETRY, k_cache=bf16(2, 64, 64), v_cache=bf16(2, 64, 64), q_out=bf16(5, 4, 64))


def attn_args():
    return dict(q=bf16(5, 4, 64), k_cache=bf16(2, 64, 64), v_cache=bf16(2, 64, 64), **GEOMETRY,
                **ROWS, window=0, scale=0.1, workspace=torch.zeros(1 << 20, dtype=torch.uint8),
                out=bf16(5, 4, 64))


def verify_args():
    f32 = torch.zeros
    return dict(target_probs=f32(5, 9), draft_probs=f32(5, 9), tokens=i32(5), row_start=i32(3),
                parents=i32(5), u_accept=f32(5), u_pick=f32(2), accepted=i32(2), path=i32(2, 4),
                next_token=i32(2))


def keep_args():
    return dict(caches=[bf16(2, 64, 64)], **GEOMETRY, batch_idx=i32(2), ctx_lens=i32(2),
                accepted=i32(2), path=i32(2, 4))


def refused(call, args, change):
    with pytest.raises(pkv.BadArgError) as e:
        call(**{**args, **change})
    assert "CUDA device" not in str(e.value)     # refused for what it is


TABLE = [dict(dev_table=None), dict(dev_table=torch.zeros(3, 2)), dict(n_slots=4),
         dict(max_pages_per_seq=3)]
TREES = [dict(row_start=None), dict(row_start=i32(0)), dict(row_start=torch.zeros(3)),
         dict(parents=None), dict(parents=i32(4)), dict(parents=i32(10)[::2]),
         dict(err_word=torch.zeros(1)), dict(err_word=i32(0)), dict(err_word=[0])]
CTX = [dict(ctx_lens=None), dict(ctx_lens=i32(1)), dict(batch_idx=i32(1)), dict(batch_idx=[1, 2]),
       dict(row_start=i32(4))]
CACHE = [dict(k_cache=None), dict(v_cache=torch.zeros(2, 64, 64)), dict(v_cache=bf16(2, 32, 64)),
         dict(k_cache=bf16(64, 64)), dict(n_pages=5), dict(page_size=8)]


@pytest.mark.parametrize("change", TABLE + TREES + CTX + CACHE + [
    dict(q=None), dict(q=bf16(5, 256)), dict(q=bf16(5, 4, 32)), dict(q=torch.zeros(5, 4, 64)),
    dict(q=bf16(5, 64, 4).transpose(1, 2)), dict(k=None), dict(k=bf16(5, 3, 64)),
    dict(k=bf16(4, 2, 64)), dict(v=bf16(6, 2, 64)), dict(v=[0.0]), dict(q_out=None),
    dict(q_out=bf16(5, 2, 64)), dict(q_out=bf16(5, 4, 128)[:, :, :64]), dict(gamma_q=bf16(32)),
    dict(gamma_k=torch.ones(64)), dict(gamma_q=None), dict(theta=0.0), dict(theta=float("inf")),
    dict(theta=float("nan")), dict(eps=-1.0), dict(rotary_dims=3), dict(rotary_dims=66),
    dict(q=torch.zeros(5 * 4 * 64 + 8 * 5, dtype=BF16).as_strided((5, 4, 64), (260, 64, 1)))],
    ids=lambda c: "-".join(c))
def test_append(change, monkeypatch):
    monkeypatch.setattr(pkv, "_on_device", lambda *t: None)   # the library refuses before it runs
    refused(pkv.tree_qkv_norm_rope_append, append_args(), change)


@pytest.mark.parametrize("change", TABLE + TREES + CTX + CACHE + [
    dict(q=None), dict(q=bf16(5, 256)), dict(q=bf16(5, 4, 32)), dict(q=bf16(5, 8, 64)[:, ::2]),
    dict(out=None), dict(out=bf16(4, 4, 64)), dict(out=torch.zeros(5, 4, 64)),
    dict(workspace=None), dict(workspace=torch.zeros(4, dtype=torch.uint8)),
    dict(workspace=torch.zeros(1 << 21, dtype=torch.uint8)[::2]), dict(window=-1),
    dict(scale=0.0), dict(scale=float("inf")), dict(scale=float("nan")),
    dict(q=bf16(5, 3, 64), out=bf16(5, 3, 64)), dict(q=bf16(5, 18, 64), out=bf16(5, 18, 64))],
    ids=lambda c: "-".join(c))
def test_attention(change, monkeypatch):
    monkeypatch.setattr(pkv, "_on_device", lambda *t: None)
    refused(pkv.paged_tree_attn, attn_args(), change)


@pytest.mark.parametrize("change", TREES + [
    dict(target_probs=None), dict(target_probs=torch.zeros(4, 9)),
    dict(target_probs=torch.zeros(45)), dict(target_probs=bf16(5, 9)),
    dict(target_probs=torch.zeros(9, 5).t()), dict(draft_probs=torch.zeros(5, 8)),
    dict(draft_probs=torch.zeros(4, 9)), dict(draft_probs=torch.zeros(5, 9, dtype=torch.float64)),
    dict(target_probs=torch.zeros(5, 0), draft_probs=None), dict(tokens=None),
    dict(tokens=torch.zeros(5, dtype=torch.int64)), dict(u_accept=None), dict(u_accept=i32(5)),
    dict(u_accept=torch.zeros(4)), dict(u_pick=torch.zeros(1)), dict(u_pick=torch.zeros(4)[::2]),
    dict(accepted=i32(1)), dict(accepted=torch.zeros(2)), dict(next_token=i32(1)),
    dict(next_token=None), dict(path=None), dict(path=i32(4)), dict(path=i32(1, 4)),
    dict(path=i32(2, 0)), dict(path=i32(2, 8)[:, ::2])], ids=lambda c: "-".join(c))
def test_verify(change, monkeypatch):
    monkeypatch.setattr(pkv, "_on_device", lambda *t: None)
    refused(pkv.tree_verify, verify_args(), change)


@pytest.mark.parametrize("change", TABLE + [
    dict(caches=None), dict(caches=bf16(2, 64, 64)), dict(caches=[None]),
    dict(caches=[bf16(2, 32, 64)]), dict(caches=[bf16(128)]),
    dict(caches=[bf16(2, 64, 128)[:, :, ::2]]), dict(caches=[bf16(2, 64, 64), bf16(0, 64, 64)]),
    dict(accepted=None), dict(accepted=i32(1)), dict(ctx_lens=i32(1)), dict(batch_idx=i32(1)),
    dict(path=None), dict(path=i32(8)), dict(path=torch.zeros(2, 4)), dict(path=i32(2, 0)),
    dict(err_word=torch.zeros(1)), dict(n_pages=8)], ids=lambda c: "-".join(c))
def test_keep_path(change, monkeypatch):
    monkeypatch.setattr(pkv, "_on_device", lambda *t: None)
    refused(pkv.kv_keep_path, keep_args(), change)


@pytest.mark.parametrize("call,args", [
    (pkv.tree_qkv_norm_rope_append, append_args), (pkv.paged_tree_attn, attn_args),
    (pkv.tree_verify, verify_args), (pkv.kv_keep_path, keep_args)])
def test_tensors_on_the_host_are_refused(call, args):
    with pytest.raises(pkv.BadArgError, match="current CUDA device"):
        call(**args())


A = 1 << 20        # a 16-byte aligned address that nothing follows


def raw(fn, order, base, change):
    """The library's answer, the same to the arguments one by one and in a record."""
    lib, args = pkv.load_library(), [{**base, **change}[k] for k in order]
    status, said = getattr(lib, fn)(*args), lib.pkv_last_error()
    record = pkv._RECORDS[fn].pack(*[0 if a is None else a for a in args])
    assert getattr(lib, fn + "_args")(record) == status
    assert lib.pkv_last_error() == said
    return status


ATTN = dict(q=A, k=A, v=A, table=A, n_slots=3, max_pages=2, page_size=16, n_pages=4, slots=A,
            ctx=A, row_start=A, parents=A, window=0, scale=1.0, B=2, N=5, Hq=4, Hkv=2, D=64, ws=A,
            ws_bytes=1 << 40, out=A, err=None, stream=None)


@pytest.mark.parametrize("change", [
    dict(D=96), dict(D=0), dict(B=-1), dict(B=513), dict(N=-1), dict(Hkv=0), dict(Hq=3),
    dict(Hq=18), dict(page_size=12), dict(page_size=4), dict(n_pages=0), dict(n_slots=0),
    dict(max_pages=0), dict(n_pages=1 << 28), dict(max_pages=1 << 27), dict(q=None), dict(k=None),
    dict(v=None), dict(table=None), dict(ctx=None), dict(row_start=None), dict(parents=None),
    dict(out=None), dict(ws=None), dict(q=A + 2), dict(out=A + 8), dict(k=A + 4), dict(ws=A + 8),
    dict(ws_bytes=8)], ids=lambda c: "-".join(c))
def test_attention_of_the_library(change):
    assert raw("paged_tree_attn", list(ATTN), ATTN, change) == pkv.PKV_E_BAD_ARG
    assert pkv.pkv_last_error()


def test_nothing_to_do_is_fine():
    for change in (dict(B=0), dict(N=0)):
        assert raw("paged_tree_attn", list(ATTN), ATTN, {**change, "q": None}) == pkv.PKV_OK
    assert pkv.paged_tree_attn_workspace(8, 3, 64) == 0
    assert pkv.paged_tree_attn_workspace(8, 1, 96) == 0
    assert pkv.paged_tree_attn_workspace(18, 2, 64) == 0
    assert pkv.paged_tree_attn_workspace(8, 1, 512) > 0


APPEND = dict(q=A, k=A, v=A, sq=256, sk=128, sv=128, gq=A, gk=A, slots=A, ctx=A, row_start=A,
              parents=A, theta=1e4, eps=1e-6, rotary=64, v_norm=0, B=2, N=5, Hq=4, Hkv=2, D=64,
              table=A, n_slots=3, max_pages=2, page_size=16, n_pages=4, kc=A, vc=A, qo=A, err=None,
              stream=None)


@pytest.mark.parametrize("change", [
    dict(D=96), dict(B=513), dict(B=-1), dict(N=-1), dict(Hq=0), dict(Hkv=0), dict(page_size=0),
    dict(rotary=-2), dict(rotary=65), dict(rotary=66), dict(theta=-1.0), dict(eps=float("nan")),
    dict(gq=None), dict(q=None), dict(k=None), dict(kc=None), dict(qo=None), dict(ctx=None),
    dict(q=A + 2), dict(vc=A + 8), dict(gk=A + 2), dict(sq=252), dict(sk=-8),
    dict(sv=1 << 41)], ids=lambda c: "-".join(c))
def test_append_of_the_library(change):
    assert raw("tree_qkv_norm_rope_append", list(APPEND), APPEND, change) == pkv.PKV_E_BAD_ARG


VERIFY = dict(p=A, sp=9, q=A, sq=9, tokens=A, row_start=A, parents=A, u=A, up=A, B=2, N=5, V=9,
              cols=4, acc=A, path=A, nxt=A, err=None, stream=None)


@pytest.mark.parametrize("change", [
    dict(B=-1), dict(B=65536), dict(N=-1), dict(V=0), dict(V=(1 << 22) + 1), dict(cols=0),
    dict(sp=8), dict(sq=8), dict(p=None), dict(tokens=None), dict(row_start=None), dict(u=None),
    dict(up=None), dict(acc=None), dict(path=None), dict(nxt=None), dict(parents=None),
    dict(sp=1 << 41)], ids=lambda c: "-".join(c))
def test_verify_of_the_library(change):
    assert raw("tree_verify", list(VERIFY), VERIFY, change) == pkv.PKV_E_BAD_ARG


@pytest.mark.parametrize("change", [
    dict(n=-1), dict(B=-1), dict(B=65536), dict(cols=0), dict(page_size=0), dict(n_pages=1 << 28),
    dict(heads=0), dict(heads=70000), dict(bytes=0), dict(bytes=(1 << 20) + 1), dict(cache=None),
    dict(table=None), dict(acc=None), dict(path=None), dict(ctx=None)], ids=lambda c: "-".join(c))
def test_keep_path_of_the_library(change):
    a = {**dict(cache=A, heads=2, bytes=128, n=1, table=A, n_slots=3, max_pages=2, page_size=16,
                n_pages=4, slots=A, ctx=A, acc=A, path=A, cols=4, B=2), **change}
    caches = ((ctypes.c_void_p * 1)(a["cache"]), (ctypes.c_int * 1)(a["heads"]),
              (ctypes.c_int64 * 1)(a["bytes"]))
    rest = dict(n=a["n"], table=a["table"], n_slots=a["n_slots"], max_pages=a["max_pages"],
                page_size=a["page_size"], n_pages=a["n_pages"], slots=a["slots"], ctx=a["ctx"],
                acc=a["acc"], path=a["path"], cols=a["cols"], B=a["B"], err=None, stream=None)
    base = {**{i: ctypes.addressof(c) for i, c in enumerate(caches)}, **rest}
    assert raw("kv_keep_path", list(base), base, {}) == pkv.PKV_E_BAD_ARG


@pytest.mark.parametrize("fn", list(pkv._RECORDS))
def test_a_record_is_needed(fn):
    assert getattr(pkv.load_library(), fn + "_args")(None) == pkv.PKV_E_BAD_ARG


@pytest.mark.parametrize("call,args,change", [
    (pkv.tree_qkv_norm_rope_append, append_args, dict(rotary_dims=1 << 40)),
    (pkv.tree_qkv_norm_rope_append, append_args, dict(theta=1e300)),
    (pkv.paged_tree_attn, attn_args, dict(window=1 << 40)),
    (pkv.paged_tree_attn, attn_args, dict(window=-(1 << 40))),
    (pkv.paged_tree_attn, attn_args, dict(scale=1e300))])
def test_numbers_that_no_argument_holds(call, args, change, monkeypatch):
    monkeypatch.setattr(pkv, "_on_device", lambda *t: None)
    refused(call, args(), change)
