"""Python binding of libpkv — paged-KV single-token decode attention on GB300.

Thin ctypes marshalling over the C ABI declared in include/pkv.h: the
functions below have the C names, take torch tensors (or raw integers for
pointers), pass their data pointers and the current CUDA stream, and turn a
negative status into an exception. Every step of the hot path runs in the
library's CUDA kernels; there is no fallback of any kind. Build the library
with ``python -c "import __graft_entry__ as g; g.build()"`` (or
``python paged_kv_decode_pagetable_gb300/_build.py``).
"""
from __future__ import annotations

import array
import ctypes
import operator
import os
import struct

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpkv.so")

# status codes (include/pkv.h)
PKV_OK = 0
PKV_E_NO_SLOT = -1
PKV_E_NO_PAGES = -2
PKV_E_BAD_SLOT = -3
PKV_E_BAD_ARG = -4
PKV_E_CUDA = -5
# device error-word bits
PKV_ERR_POS = 1
PKV_ERR_PAGE_RANGE = 2
PKV_ERR_PAGE_NEG = 4
PKV_ERR_SLOT = 8
PKV_ERR_TIMEOUT = 16
PKV_ERR_ORDER = 32
PKV_ERR_TREE = 64
PKV_ERR_PROB = 128


class PkvError(RuntimeError):
    code = None


class NoSlotError(PkvError):
    code = PKV_E_NO_SLOT


class NoPagesError(PkvError):
    code = PKV_E_NO_PAGES


class BadSlotError(PkvError):
    code = PKV_E_BAD_SLOT


class BadArgError(PkvError):
    code = PKV_E_BAD_ARG


class CudaError(PkvError):
    code = PKV_E_CUDA


_ERRORS = {c.code: c for c in (NoSlotError, NoPagesError, BadSlotError, BadArgError, CudaError)}

_c_int, _c_p, _c_f, _c_sz = ctypes.c_int, ctypes.c_void_p, ctypes.c_float, ctypes.c_size_t
_c_i64 = ctypes.c_int64
_c_ip = ctypes.POINTER(ctypes.c_int32)

_SIGS = {
    "pt_create": (_c_int, [_c_int, _c_int, _c_int, _c_int, _c_p, _c_p, ctypes.POINTER(_c_p)]),
    "pt_destroy": (_c_int, [_c_p]),
    "pt_set_stream": (_c_int, [_c_p, _c_p]),
    "pt_get_stream": (_c_int, [_c_p, ctypes.POINTER(_c_p)]),
    "pt_can_reserve": (_c_int, [_c_p, _c_int, _c_int, ctypes.POINTER(_c_int)]),
    "pt_assign": (_c_int, [_c_p, _c_int, ctypes.POINTER(_c_int)]),
    "pt_reserve": (_c_int, [_c_p, _c_int, _c_int]),
    "pt_free": (_c_int, [_c_p, _c_int]),
    "pt_fork": (_c_int, [_c_p, _c_int, _c_int, _c_int, ctypes.POINTER(_c_int), _c_ip, _c_int,
                         ctypes.POINTER(_c_int)]),
    "pt_unshare": (_c_int, [_c_p, _c_int, _c_int, _c_int, _c_ip, _c_int,
                            ctypes.POINTER(_c_int)]),
    "pt_truncate": (_c_int, [_c_p, _c_int, _c_int]),
    "pt_compact": (_c_int, [_c_p, _c_ip, _c_int, ctypes.POINTER(_c_int)]),
    "pt_page_refs": (_c_int, [_c_p, _c_int, ctypes.POINTER(_c_int)]),
    "kv_copy_pages": (_c_int, [_c_p, _c_p, _c_p, _c_int, _c_int, _c_p, _c_int, _c_p]),
    "pt_capacity": (_c_int, [_c_p, _c_int, ctypes.POINTER(_c_int)]),
    "pt_pages": (_c_int, [_c_p, _c_int, _c_ip, _c_int, ctypes.POINTER(_c_int)]),
    "pt_free_pages": (_c_int, [_c_p, ctypes.POINTER(_c_int)]),
    "pt_free_page_list": (_c_int, [_c_p, _c_ip, _c_int, ctypes.POINTER(_c_int)]),
    "pt_host_table": (_c_int, [_c_p, _c_ip, _c_int]),
    "kv_append": (_c_int, [_c_p, _c_p, _c_p, _c_p, _c_int, _c_p, _c_int, _c_int, _c_int,
                           _c_int, _c_p, _c_p, _c_int, _c_int, _c_p, _c_p]),
    "kv_append_prefill": (_c_int, [_c_p, _c_p, _c_p, _c_p, _c_int, _c_p, _c_int, _c_int, _c_int,
                                   _c_int, _c_p, _c_p, _c_int, _c_int, _c_p, _c_p]),
    "kv_append_q8": (_c_int, [_c_p, _c_p, _c_p, _c_p, _c_int, _c_p, _c_int, _c_int, _c_int, _c_int,
                              _c_int, _c_p, _c_p, _c_p, _c_p, _c_int, _c_int, _c_p, _c_p]),
    "kv_append_prefill_q8": (_c_int, [_c_p, _c_p, _c_p, _c_p, _c_int, _c_p, _c_int, _c_int, _c_int,
                                      _c_int, _c_int, _c_p, _c_p, _c_p, _c_p, _c_int, _c_int,
                                      _c_p, _c_p]),
    "paged_decode_attn_q8": (_c_int, [_c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_int, _c_int, _c_int,
                                      _c_int, _c_int, _c_p, _c_p, _c_int, _c_f, _c_int, _c_int,
                                      _c_int, _c_int, _c_p, _c_sz, _c_p, _c_p, _c_p]),
    "paged_decode_attn_q8_workspace": (_c_sz, [_c_int, _c_int, _c_int]),
    "prefill_block_mask": (_c_int, [_c_p, _c_int, _c_int, _c_p, _c_p, _c_p, _c_p, _c_p]),
    "convert_logical_block_mask": (_c_int, [_c_p, _c_int, _c_int, _c_p, _c_int, _c_int, _c_int,
                                            _c_int, _c_p, _c_int, _c_p, _c_p, _c_p]),
    "prefill_attn": (_c_int, [_c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_int, _c_int,
                              _c_int, _c_int, _c_int, _c_f, _c_p, _c_p]),
    "qk_norm_rope": (_c_int, [_c_p, _c_p, _c_p, _c_p, _c_p, _c_f, _c_f, _c_int, _c_int,
                              _c_int, _c_int, _c_p]),
    "qk_norm_rope_append": (_c_int, [_c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_f, _c_f,
                                     _c_int, _c_int, _c_int, _c_int, _c_p, _c_int, _c_int,
                                     _c_int, _c_int, _c_p, _c_p, _c_p, _c_p]),
    "paged_decode_attn": (_c_int, [_c_p, _c_p, _c_p, _c_p, _c_int, _c_int, _c_int, _c_int,
                                   _c_p, _c_p, _c_int, _c_f, _c_int, _c_int, _c_int, _c_int,
                                   _c_int, _c_p, _c_sz, _c_p, _c_p, _c_p]),
    "paged_decode_attn_noalloc": (_c_int, [_c_p, _c_p, _c_p, _c_p, _c_int, _c_int, _c_int,
                                           _c_int, _c_p, _c_p, _c_int, _c_f, _c_int, _c_int,
                                           _c_int, _c_int, _c_int, _c_p, _c_p, _c_p]),
    "paged_decode_attn_splits": (_c_int, [_c_int, _c_int, _c_int, _c_int, _c_int, _c_int,
                                          ctypes.POINTER(_c_int)]),
    "paged_decode_attn_workspace": (_c_sz, [_c_int, _c_int, _c_int, _c_int]),
    "qkv_norm_rope": (_c_int, [_c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_f, _c_f, _c_int, _c_int,
                               _c_int, _c_int, _c_int, _c_p]),
    "paged_decode_step_ex": (_c_int, [_c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_f, _c_f,
                                      _c_int, _c_int, _c_int, _c_p, _c_int, _c_int, _c_int,
                                      _c_int, _c_p, _c_p, _c_int, _c_f, _c_int, _c_int, _c_int,
                                      _c_int, _c_int, _c_p, _c_sz, _c_p, _c_p, _c_p]),
    "paged_decode_step": (_c_int, [_c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_f, _c_f, _c_p,
                                   _c_int, _c_int, _c_int, _c_int, _c_p, _c_p, _c_int, _c_f,
                                   _c_int, _c_int, _c_int, _c_int, _c_int, _c_p, _c_sz, _c_p,
                                   _c_p, _c_p]),
    "tree_qkv_norm_rope_append": (_c_int, [_c_p, _c_p, _c_p, _c_i64, _c_i64, _c_i64, _c_p, _c_p,
                                           _c_p, _c_p, _c_p, _c_p, _c_f, _c_f, _c_int, _c_int,
                                           _c_int, _c_int, _c_int, _c_int, _c_int, _c_p, _c_int,
                                           _c_int, _c_int, _c_int, _c_p, _c_p, _c_p, _c_p, _c_p]),
    "paged_tree_attn": (_c_int, [_c_p, _c_p, _c_p, _c_p, _c_int, _c_int, _c_int, _c_int, _c_p,
                                 _c_p, _c_p, _c_p, _c_int, _c_f, _c_int, _c_int, _c_int, _c_int,
                                 _c_int, _c_p, _c_sz, _c_p, _c_p, _c_p]),
    "paged_tree_attn_workspace": (_c_sz, [_c_int, _c_int, _c_int]),
    "tree_verify": (_c_int, [_c_p, _c_i64, _c_p, _c_i64, _c_p, _c_p, _c_p, _c_p, _c_p, _c_int,
                             _c_int, _c_int, _c_int, _c_p, _c_p, _c_p, _c_p, _c_p]),
    "kv_keep_path": (_c_int, [_c_p, _c_p, _c_p, _c_int, _c_p, _c_int, _c_int, _c_int, _c_int,
                              _c_p, _c_p, _c_p, _c_p, _c_int, _c_int, _c_p, _c_p]),
    "tree_qkv_norm_rope_append_args": (_c_int, [ctypes.c_char_p]),
    "paged_tree_attn_args": (_c_int, [ctypes.c_char_p]),
    "tree_verify_args": (_c_int, [ctypes.c_char_p]),
    "kv_keep_path_args": (_c_int, [ctypes.c_char_p]),
    "pkv_read_error_word": (_c_int, [_c_p, _c_p, _c_ip]),
    "pkv_last_error": (ctypes.c_char_p, []),
}

EXPORTS = tuple(_SIGS)
_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Loads libpkv.so; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(
            f"libpkv.so not found at {path}; build it first "
            "(python -c 'import __graft_entry__ as g; g.build()')")
    lib = ctypes.CDLL(path)
    for name, (res, args) in _SIGS.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _check(status: int, what: str) -> None:
    if status != PKV_OK:
        msg = load_library().pkv_last_error().decode(errors="replace")
        raise _ERRORS.get(status, PkvError)(f"{what}: {msg} (status {status})")


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


# the current stream's handle without building a torch.cuda.Stream (about 4 us), and the
# current device without torch.cuda's own look at its initialisation
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_raw_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(stream) -> int | None:
    if stream is None:
        if torch.cuda.is_initialized():
            if _raw_stream is not None:
                return _raw_stream(_raw_device())
            return torch.cuda.current_stream().cuda_stream
        return None
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


_E4M3, _F32, _BF16, _I32 = torch.float8_e4m3fn, torch.float32, torch.bfloat16, torch.int32


def _bf16(t, name):
    if t is not None and not isinstance(t, int):
        try:
            good = t.dtype is _BF16 and t.is_contiguous()
        except AttributeError:
            good = False
        if not good:
            raise BadArgError(f"{name} must be a contiguous bfloat16 tensor")
    return t


def _i32(t, name):
    if t is not None and not isinstance(t, int):
        try:
            good = t.dtype is _I32 and t.is_contiguous()
        except AttributeError:
            good = False
        if not good:
            raise BadArgError(f"{name} must be a contiguous int32 tensor")
    return t


def _on_device(*tensors) -> None:
    """Refuses tensors that are not on the current CUDA device (None passes)."""
    dev = _raw_device() if torch.cuda.is_initialized() else None
    for t in tensors:
        if t is not None and type(t) is not int and t.get_device() != dev:
            raise BadArgError("every tensor must be on the current CUDA device")


# --------------------------------------------------------------------------
# PageTable allocator
# --------------------------------------------------------------------------

def pt_create(max_batch_size: int, page_size: int, n_pages: int, max_pages_per_seq: int,
              dev_table=None, stream=None) -> int:
    lib = load_library()
    h = _c_p()
    _check(lib.pt_create(max_batch_size, page_size, n_pages, max_pages_per_seq,
                         _ptr(_i32(dev_table, "dev_table")), _stream(stream) if dev_table is not None else None,
                         ctypes.byref(h)), "pt_create")
    return h.value


def pt_destroy(h: int) -> None:
    _check(load_library().pt_destroy(h), "pt_destroy")


def pt_set_stream(h: int, stream=None) -> None:
    _check(load_library().pt_set_stream(h, _stream(stream)), "pt_set_stream")


def pt_get_stream(h: int) -> int:
    """The handle's stream (0: the default stream)."""
    s = _c_p()
    _check(load_library().pt_get_stream(h, ctypes.byref(s)), "pt_get_stream")
    return s.value or 0


def pt_can_reserve(h: int, seq_len: int, slot: int = -1) -> bool:
    ok = _c_int()
    _check(load_library().pt_can_reserve(h, seq_len, slot, ctypes.byref(ok)), "pt_can_reserve")
    return bool(ok.value)


def pt_assign(h: int, seq_len: int) -> int:
    slot = _c_int()
    _check(load_library().pt_assign(h, seq_len, ctypes.byref(slot)), "pt_assign")
    return slot.value


def pt_reserve(h: int, slot: int, seq_len: int) -> None:
    _check(load_library().pt_reserve(h, slot, seq_len), "pt_reserve")


def pt_free(h: int, slot: int) -> None:
    _check(load_library().pt_free(h, slot), "pt_free")


def _pairs(n: int) -> torch.Tensor:
    return torch.empty((n, 2), dtype=torch.int32)


def pt_fork(h: int, src_slot: int, seq_len: int, count: int = 1):
    """`count` new slots holding the first seq_len tokens of src_slot; returns
    (slots, pairs): the pages to copy with kv_copy_pages (CPU int32 [n][2])."""
    slots = (_c_int * max(count, 1))()
    pairs = _pairs(max(count, 1))
    n = _c_int()
    _check(load_library().pt_fork(h, src_slot, seq_len, count, slots,
                                  ctypes.cast(pairs.data_ptr(), _c_ip), pairs.shape[0],
                                  ctypes.byref(n)), "pt_fork")
    return list(slots), pairs[:n.value]


def pt_unshare(h: int, slot: int, begin: int, end: int) -> torch.Tensor:
    """Pages of the slot's own under tokens [begin, end); returns the pairs."""
    pairs = _pairs(len(pt_pages(h, slot)))
    n = _c_int()
    _check(load_library().pt_unshare(h, slot, begin, end,
                                     ctypes.cast(pairs.data_ptr(), _c_ip), pairs.shape[0],
                                     ctypes.byref(n)), "pt_unshare")
    return pairs[:n.value]


def pt_truncate(h: int, slot: int, seq_len: int) -> None:
    _check(load_library().pt_truncate(h, slot, seq_len), "pt_truncate")


def pt_compact(h: int) -> torch.Tensor:
    """Moves the used pages to the lowest numbers; returns the pairs."""
    lib = load_library()
    n = _c_int()
    _check(lib.pt_compact(h, None, 0, ctypes.byref(n)), "pt_compact")
    pairs = _pairs(max(n.value, 1))
    _check(lib.pt_compact(h, ctypes.cast(pairs.data_ptr(), _c_ip), pairs.shape[0],
                          ctypes.byref(n)), "pt_compact")
    return pairs[:n.value]


def pt_page_refs(h: int, page: int) -> int:
    n = _c_int()
    _check(load_library().pt_page_refs(h, page, ctypes.byref(n)), "pt_page_refs")
    return n.value


def pt_capacity(h: int, slot: int) -> int:
    n = _c_int()
    _check(load_library().pt_capacity(h, slot, ctypes.byref(n)), "pt_capacity")
    return n.value


def pt_pages(h: int, slot: int) -> list[int]:
    lib = load_library()
    n = _c_int()
    _check(lib.pt_pages(h, slot, None, 0, ctypes.byref(n)), "pt_pages")
    buf = (ctypes.c_int32 * max(n.value, 1))()
    _check(lib.pt_pages(h, slot, buf, n.value, ctypes.byref(n)), "pt_pages")
    return list(buf[:n.value])


def pt_free_pages(h: int) -> int:
    n = _c_int()
    _check(load_library().pt_free_pages(h, ctypes.byref(n)), "pt_free_pages")
    return n.value


def pt_free_page_list(h: int) -> list[int]:
    lib = load_library()
    n = _c_int()
    _check(lib.pt_free_page_list(h, None, 0, ctypes.byref(n)), "pt_free_page_list")
    buf = (ctypes.c_int32 * max(n.value, 1))()
    _check(lib.pt_free_page_list(h, buf, n.value, ctypes.byref(n)), "pt_free_page_list")
    return list(buf[:n.value])


def pt_host_table(h: int, n_slots: int, max_pages_per_seq: int) -> torch.Tensor:
    out = torch.empty((n_slots, max_pages_per_seq), dtype=torch.int32)
    _check(load_library().pt_host_table(h, ctypes.cast(out.data_ptr(), _c_ip), out.numel()),
           "pt_host_table")
    return out


class PageTable:
    """Owns one pt_* handle and its caller-side device table tensor."""

    def __init__(self, max_batch_size: int, page_size: int, n_pages: int,
                 max_pages_per_seq: int, device=None, stream=None):
        self.max_batch_size = max_batch_size
        self.n_slots = max_batch_size + 1
        self.page_size = page_size
        self.n_pages = n_pages
        self.max_pages_per_seq = max_pages_per_seq
        self.dev_table = None
        if device is not None:
            self.dev_table = torch.empty((self.n_slots, max_pages_per_seq),
                                         dtype=torch.int32, device=device)
        self.handle = pt_create(max_batch_size, page_size, n_pages, max_pages_per_seq,
                                self.dev_table, stream)

    def __del__(self):
        h = getattr(self, "handle", None)
        if h and _lib is not None:
            _lib.pt_destroy(h)
            self.handle = None

    def can_reserve(self, seq_len, slot=-1):
        return pt_can_reserve(self.handle, seq_len, slot)

    def assign(self, seq_len):
        return pt_assign(self.handle, seq_len)

    def reserve(self, slot, seq_len):
        pt_reserve(self.handle, slot, seq_len)

    def free(self, slot):
        pt_free(self.handle, slot)

    def fork(self, slot, seq_len, count=1):
        return pt_fork(self.handle, slot, seq_len, count)

    def unshare(self, slot, begin, end):
        return pt_unshare(self.handle, slot, begin, end)

    def truncate(self, slot, seq_len):
        pt_truncate(self.handle, slot, seq_len)

    def compact(self):
        return pt_compact(self.handle)

    def page_refs(self, page):
        return pt_page_refs(self.handle, page)

    def capacity(self, slot):
        return pt_capacity(self.handle, slot)

    def pages(self, slot):
        return pt_pages(self.handle, slot)

    def free_page_list(self):
        return pt_free_page_list(self.handle)

    def host_table(self):
        return pt_host_table(self.handle, self.n_slots, self.max_pages_per_seq)


# --------------------------------------------------------------------------
# kernels
# --------------------------------------------------------------------------

def kv_append(k, v, batch_idx, input_pos, dev_table, n_slots, max_pages_per_seq,
              page_size, n_pages, k_cache, v_cache, err_word=None, stream=None) -> None:
    _bf16(k, "k"), _bf16(v, "v"), _bf16(k_cache, "k_cache"), _bf16(v_cache, "v_cache")
    _i32(batch_idx, "batch_idx"), _i32(input_pos, "input_pos"), _i32(dev_table, "dev_table")
    B, Hkv, D = k.shape
    _check(load_library().kv_append(
        _ptr(k), _ptr(v), _ptr(batch_idx), _ptr(input_pos), B, _ptr(dev_table), n_slots,
        max_pages_per_seq, page_size, n_pages, _ptr(k_cache), _ptr(v_cache), Hkv, D,
        _ptr(err_word), _stream(stream)), "kv_append")


def kv_append_prefill(k, v, batch_idx, input_pos, dev_table, n_slots, max_pages_per_seq,
                      page_size, n_pages, k_cache, v_cache, err_word=None, stream=None) -> None:
    """Scatter L packed prefill tokens; k and v are head-major [Hkv][L][D]."""
    _bf16(k, "k"), _bf16(v, "v"), _bf16(k_cache, "k_cache"), _bf16(v_cache, "v_cache")
    _i32(batch_idx, "batch_idx"), _i32(input_pos, "input_pos"), _i32(dev_table, "dev_table")
    Hkv, L, D = k.shape
    _check(load_library().kv_append_prefill(
        _ptr(k), _ptr(v), _ptr(batch_idx), _ptr(input_pos), L, _ptr(dev_table), n_slots,
        max_pages_per_seq, page_size, n_pages, _ptr(k_cache), _ptr(v_cache), Hkv, D,
        _ptr(err_word), _stream(stream)), "kv_append_prefill")


def _word(t) -> None:
    """Refuses an error word that is not one (None and addresses pass)."""
    if t is not None and type(t) is not int and (
            not isinstance(t, torch.Tensor) or t.dtype is not _I32 or t.numel() < 1):
        raise BadArgError("err_word must be an int32 tensor")


def _q8_cache(k_cache, v_cache, k_scale, v_scale, n_rows: int) -> tuple:
    """Checks an 8-bit cache's tensors; returns the kv heads, the head dim and the
    tokens that share a scale."""
    try:
        shape, v_shape, scales, v_scales = (k_cache.shape, v_cache.shape, k_scale.shape,
                                            v_scale.shape)
    except AttributeError:
        raise BadArgError("k_cache, v_cache, k_scale and v_scale must be tensors") from None
    for t, size, name in ((k_cache, shape, "k_cache"), (v_cache, v_shape, "v_cache")):
        if t.dtype is not _E4M3 or len(size) != 3 or not t.is_contiguous():
            raise BadArgError(f"{name} must be a contiguous float8_e4m3fn tensor "
                              "[Hkv][n_pages * page_size][D]")
    for t, size, name in ((k_scale, scales, "k_scale"), (v_scale, v_scales, "v_scale")):
        if t.dtype is not _F32 or len(size) != 2 or not t.is_contiguous():
            raise BadArgError(f"{name} must be a contiguous float32 tensor "
                              "[Hkv][n_pages * page_size / scale_block]")
    Hkv, rows, D = shape
    if v_shape != shape or rows != n_rows:
        raise BadArgError("k_cache and v_cache must both hold n_pages * page_size rows")
    heads, n = scales
    if v_scales != scales or heads != Hkv or n < 1 or n_rows % n:
        raise BadArgError("k_scale and v_scale must both be [Hkv][n_pages * page_size / "
                          "scale_block]")
    return Hkv, D, n_rows // n


def _append_q8(name, head_major, k, v, batch_idx, input_pos, dev_table, n_slots,
               max_pages_per_seq, page_size, n_pages, k_cache, v_cache, k_scale, v_scale,
               err_word, stream) -> None:
    _bf16(k, "k"), _bf16(v, "v")
    _i32(batch_idx, "batch_idx"), _i32(input_pos, "input_pos"), _i32(dev_table, "dev_table")
    if err_word is not None:
        _word(err_word)
    Hkv, D, block = _q8_cache(k_cache, v_cache, k_scale, v_scale, n_pages * page_size)
    try:
        shape = k.shape
        if len(shape) != 3 or v.shape != shape:
            raise BadArgError(f"{name}: k and v must have one shape of three dimensions")
        if head_major:
            heads, N, width = shape
        else:
            N, heads, width = shape
        if heads != Hkv or width != D:
            raise BadArgError(f"{name}: k, v and the caches differ in heads or head dim")
        if input_pos is None or input_pos.numel() < N or (
                batch_idx is not None and batch_idx.numel() < N):
            raise BadArgError(f"{name}: batch_idx and input_pos must hold a value for every "
                              "token")
        if dev_table is None or dev_table.numel() < n_slots * max_pages_per_seq:
            raise BadArgError(f"{name}: dev_table must be [n_slots][max_pages_per_seq]")
    except AttributeError:
        raise BadArgError(f"{name}: k, v, batch_idx, input_pos and dev_table must be tensors"
                          ) from None
    _on_device(k, v, batch_idx, input_pos, dev_table, k_cache, v_cache, k_scale, v_scale, err_word)
    lib = load_library()
    fn = lib.kv_append_prefill_q8 if head_major else lib.kv_append_q8
    _check(fn(k.data_ptr(), v.data_ptr(), _ptr(batch_idx), input_pos.data_ptr(), N,
              dev_table.data_ptr(), n_slots, max_pages_per_seq, page_size, n_pages, block,
              k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), Hkv,
              D, _ptr(err_word), _stream(stream)), name)


def kv_append_q8(k, v, batch_idx, input_pos, dev_table, n_slots, max_pages_per_seq, page_size,
                 n_pages, k_cache, v_cache, k_scale, v_scale, err_word=None,
                 stream=None) -> None:
    """kv_append into the 8-bit cache (float8_e4m3fn codes, fp32 scales
    [Hkv][n_pages * page_size / scale_block]); k and v are bf16 [B][Hkv][D]."""
    _append_q8("kv_append_q8", False, k, v, batch_idx, input_pos, dev_table, n_slots,
               max_pages_per_seq, page_size, n_pages, k_cache, v_cache, k_scale, v_scale,
               err_word, stream)


def kv_append_prefill_q8(k, v, batch_idx, input_pos, dev_table, n_slots, max_pages_per_seq,
                         page_size, n_pages, k_cache, v_cache, k_scale, v_scale, err_word=None,
                         stream=None) -> None:
    """kv_append_q8 of L packed prefill tokens; k and v are head-major
    [Hkv][L][D]."""
    _append_q8("kv_append_prefill_q8", True, k, v, batch_idx, input_pos, dev_table, n_slots,
               max_pages_per_seq, page_size, n_pages, k_cache, v_cache, k_scale, v_scale,
               err_word, stream)


def kv_copy_pages(caches, n_pages, pairs, stream=None) -> None:
    """Copies page pairs[i][0] to page pairs[i][1] of every head of every cache
    in `caches` (contiguous device tensors [heads][...], each head n_pages
    pages: K and V caches, scales, any number of layers). pairs: CPU int32
    [n][2], as pt_fork, pt_unshare and pt_compact return, or a sequence of
    (source, destination)."""
    if not isinstance(pairs, torch.Tensor):
        try:
            given = torch.tensor(list(pairs))
            pairs = given.to(torch.int32).reshape(-1, 2)
            if given.numel() and (given.dtype.is_floating_point or given.dtype.is_complex
                                  or given.dtype == torch.bool
                                  or (given.reshape(-1, 2) != pairs).any()):
                raise ValueError("not whole numbers of 32 bits")
        except (TypeError, ValueError, RuntimeError) as e:
            raise BadArgError(f"kv_copy_pages: pairs must be (source, destination)s: {e}") from None
    if (pairs.device.type != "cpu" or pairs.dtype != torch.int32 or pairs.dim() != 2
            or pairs.shape[1] != 2):
        raise BadArgError("kv_copy_pages: pairs must be a CPU int32 tensor [n][2]")
    pairs = pairs.contiguous()
    try:
        if isinstance(caches, torch.Tensor):
            raise TypeError
        n = len(caches)
        ptrs, heads, nbytes = (_c_p * n)(), (_c_int * n)(), (ctypes.c_int64 * n)()
        for i, c in enumerate(caches):
            if not c.is_contiguous() or c.dim() < 2:
                raise BadArgError("kv_copy_pages: caches must be contiguous tensors [heads][...]")
            size, h = c.nbytes, c.shape[0]
            each = size // max(h * n_pages, 1)
            if each * h * n_pages != size:
                raise BadArgError("kv_copy_pages: a head of a cache must be n_pages equal pages")
            ptrs[i], heads[i], nbytes[i] = c.data_ptr(), h, each
    except (AttributeError, TypeError):
        raise BadArgError("kv_copy_pages: caches must be a list of tensors") from None
    _on_device(*caches)
    _check(load_library().kv_copy_pages(ptrs, heads, nbytes, n, n_pages, pairs.data_ptr(),
                                        pairs.shape[0], _stream(stream)), "kv_copy_pages")


def qk_norm_rope(q, k, gamma_q, gamma_k, pos, theta: float, eps: float = 1e-6,
                 stream=None) -> None:
    _bf16(q, "q"), _bf16(k, "k"), _bf16(gamma_q, "gamma_q"), _bf16(gamma_k, "gamma_k")
    _i32(pos, "pos")
    B, Hq, D = q.shape
    Hkv = 0 if k is None else k.shape[1]
    _check(load_library().qk_norm_rope(
        _ptr(q), _ptr(k), _ptr(gamma_q), _ptr(gamma_k), _ptr(pos), float(theta), float(eps),
        B, Hq, Hkv, D, _stream(stream)), "qk_norm_rope")


def qkv_norm_rope(q, k, v, gamma_q, gamma_k, pos, theta: float, eps: float = 1e-6,
                  rotary_dims: int | None = None, stream=None) -> None:
    """qk_norm_rope with partial rotary (leading rotary_dims of D) and, when v
    is given, v normalised in place without a gain."""
    _bf16(q, "q"), _bf16(k, "k"), _bf16(v, "v"), _bf16(gamma_q, "gamma_q")
    _bf16(gamma_k, "gamma_k"), _i32(pos, "pos")
    B, Hq, D = q.shape
    Hkv = 0 if k is None else k.shape[1]
    rd = D if rotary_dims is None else int(rotary_dims)
    _check(load_library().qkv_norm_rope(
        _ptr(q), _ptr(k), _ptr(v), _ptr(gamma_q), _ptr(gamma_k), _ptr(pos), float(theta),
        float(eps), rd, B, Hq, Hkv, D, _stream(stream)), "qkv_norm_rope")


def qk_norm_rope_append(q, k, v, gamma_q, gamma_k, batch_idx, input_pos, theta: float,
                        eps, dev_table, n_slots, max_pages_per_seq, page_size, n_pages,
                        k_cache, v_cache, err_word=None, stream=None) -> None:
    _bf16(q, "q"), _bf16(k, "k"), _bf16(v, "v"), _bf16(gamma_q, "gamma_q")
    _bf16(gamma_k, "gamma_k"), _bf16(k_cache, "k_cache"), _bf16(v_cache, "v_cache")
    _i32(batch_idx, "batch_idx"), _i32(input_pos, "input_pos"), _i32(dev_table, "dev_table")
    B, Hq, D = q.shape
    Hkv = k.shape[1]
    _check(load_library().qk_norm_rope_append(
        _ptr(q), _ptr(k), _ptr(v), _ptr(gamma_q), _ptr(gamma_k), _ptr(batch_idx),
        _ptr(input_pos), float(theta), float(eps), B, Hq, Hkv, D, _ptr(dev_table), n_slots,
        max_pages_per_seq, page_size, n_pages, _ptr(k_cache), _ptr(v_cache), _ptr(err_word),
        _stream(stream)), "qk_norm_rope_append")


def paged_decode_attn_splits(B, Hkv, D, max_pages_per_seq, page_size, window=0) -> int:
    n = _c_int()
    _check(load_library().paged_decode_attn_splits(B, Hkv, D, max_pages_per_seq, page_size,
                                                   window, ctypes.byref(n)),
           "paged_decode_attn_splits")
    return n.value


def paged_decode_attn_workspace(B, Hq, D, num_splits) -> int:
    return int(load_library().paged_decode_attn_workspace(B, Hq, D, num_splits))


def paged_decode_attn(q, k_cache, v_cache, dev_table, n_slots, max_pages_per_seq, page_size,
                      n_pages, batch_idx, seq_lens, window, scale, num_splits, workspace,
                      out, err_word=None, stream=None) -> None:
    _bf16(q, "q"), _bf16(k_cache, "k_cache"), _bf16(v_cache, "v_cache"), _bf16(out, "out")
    _i32(dev_table, "dev_table"), _i32(batch_idx, "batch_idx"), _i32(seq_lens, "seq_lens")
    B, Hq, D = q.shape
    Hkv = k_cache.shape[0]
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load_library().paged_decode_attn(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(dev_table), n_slots, max_pages_per_seq,
        page_size, n_pages, _ptr(batch_idx), _ptr(seq_lens), int(window), float(scale), B, Hq,
        Hkv, D, int(num_splits), _ptr(workspace), ws_bytes, _ptr(out), _ptr(err_word),
        _stream(stream)), "paged_decode_attn")


def paged_decode_attn_q8_workspace(Hq, Hkv, D) -> int:
    return int(load_library().paged_decode_attn_q8_workspace(Hq, Hkv, D))


def paged_decode_attn_q8(q, k_cache, v_cache, k_scale, v_scale, dev_table, n_slots,
                         max_pages_per_seq, page_size, n_pages, batch_idx, seq_lens, window,
                         scale, workspace, out, err_word=None, stream=None) -> None:
    """paged_decode_attn over the 8-bit cache (see kv_append_q8). workspace: a
    zeroed byte tensor of paged_decode_attn_q8_workspace(Hq, Hkv, D)."""
    _bf16(q, "q"), _bf16(out, "out")
    _i32(dev_table, "dev_table"), _i32(batch_idx, "batch_idx"), _i32(seq_lens, "seq_lens")
    if err_word is not None:
        _word(err_word)
    Hkv, D, block = _q8_cache(k_cache, v_cache, k_scale, v_scale, n_pages * page_size)
    try:
        shape = q.shape
        if len(shape) != 3 or shape[2] != D or out.shape != shape:
            raise BadArgError("paged_decode_attn_q8: q, out and the caches differ in shape")
        B, Hq, _ = shape
        if seq_lens is None or seq_lens.numel() < B or (
                batch_idx is not None and batch_idx.numel() < B):
            raise BadArgError("paged_decode_attn_q8: batch_idx and seq_lens must hold a value "
                              "for every row")
        if dev_table is None or dev_table.numel() < n_slots * max_pages_per_seq:
            raise BadArgError("paged_decode_attn_q8: dev_table must be [n_slots]"
                              "[max_pages_per_seq]")
        if workspace is None:
            raise BadArgError("paged_decode_attn_q8: workspace is missing")
        if not workspace.is_contiguous():
            raise BadArgError("paged_decode_attn_q8: workspace must be a contiguous tensor")
    except AttributeError:
        raise BadArgError("paged_decode_attn_q8: q, out, batch_idx, seq_lens, dev_table and "
                          "workspace must be tensors") from None
    _on_device(q, k_cache, v_cache, k_scale, v_scale, dev_table, batch_idx, seq_lens, workspace,
               out, err_word)
    _check(load_library().paged_decode_attn_q8(
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(),
        v_scale.data_ptr(), dev_table.data_ptr(), n_slots, max_pages_per_seq, page_size, n_pages,
        block, _ptr(batch_idx), seq_lens.data_ptr(), window, scale, B, Hq, Hkv, D,
        workspace.data_ptr(), workspace.nbytes, out.data_ptr(), _ptr(err_word),
        _stream(stream)), "paged_decode_attn_q8")


def paged_decode_step(q, k, v, gamma_q, gamma_k, batch_idx, input_pos, theta, eps, dev_table,
                      n_slots, max_pages_per_seq, page_size, n_pages, k_cache, v_cache, window,
                      scale, num_splits, workspace, out, err_word=None, stream=None) -> None:
    """qk_norm_rope + kv_append + paged_decode_attn (seq_lens = input_pos + 1)
    in one pass; q, k and v are read only."""
    _bf16(q, "q"), _bf16(k, "k"), _bf16(v, "v"), _bf16(gamma_q, "gamma_q")
    _bf16(gamma_k, "gamma_k"), _bf16(k_cache, "k_cache"), _bf16(v_cache, "v_cache")
    _bf16(out, "out")
    _i32(dev_table, "dev_table"), _i32(batch_idx, "batch_idx"), _i32(input_pos, "input_pos")
    B, Hq, D = q.shape
    Hkv = k_cache.shape[0]
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load_library().paged_decode_step(
        _ptr(q), _ptr(k), _ptr(v), _ptr(gamma_q), _ptr(gamma_k), _ptr(batch_idx),
        _ptr(input_pos), float(theta), float(eps), _ptr(dev_table), n_slots, max_pages_per_seq,
        page_size, n_pages, _ptr(k_cache), _ptr(v_cache), int(window), float(scale), B, Hq, Hkv,
        D, int(num_splits), _ptr(workspace), ws_bytes, _ptr(out), _ptr(err_word),
        _stream(stream)), "paged_decode_step")


def paged_decode_step_ex(q, k, v, gamma_q, gamma_k, batch_idx, input_pos, theta, eps,
                         rotary_dims, v_norm, k_eq_v, dev_table, n_slots, max_pages_per_seq,
                         page_size, n_pages, k_cache, v_cache, window, scale, num_splits,
                         workspace, out, err_word=None, stream=None) -> None:
    """paged_decode_step with the Gemma-4 options: rotary on the leading
    rotary_dims (None: all of D), gain-free value norm, value = raw k."""
    _bf16(q, "q"), _bf16(k, "k"), _bf16(v, "v"), _bf16(gamma_q, "gamma_q")
    _bf16(gamma_k, "gamma_k"), _bf16(k_cache, "k_cache"), _bf16(v_cache, "v_cache")
    _bf16(out, "out")
    _i32(dev_table, "dev_table"), _i32(batch_idx, "batch_idx"), _i32(input_pos, "input_pos")
    B, Hq, D = q.shape
    Hkv = k_cache.shape[0]
    rd = D if rotary_dims is None else int(rotary_dims)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load_library().paged_decode_step_ex(
        _ptr(q), _ptr(k), _ptr(v), _ptr(gamma_q), _ptr(gamma_k), _ptr(batch_idx),
        _ptr(input_pos), float(theta), float(eps), rd, int(bool(v_norm)), int(bool(k_eq_v)),
        _ptr(dev_table), n_slots, max_pages_per_seq, page_size, n_pages, _ptr(k_cache),
        _ptr(v_cache), int(window), float(scale), B, Hq, Hkv, D, int(num_splits),
        _ptr(workspace), ws_bytes, _ptr(out), _ptr(err_word), _stream(stream)),
        "paged_decode_step_ex")


def paged_decode_attn_noalloc(q, k_cache, v_cache, dev_table, n_slots, max_pages_per_seq,
                              page_size, n_pages, batch_idx, seq_lens, window, scale, num_splits,
                              out, err_word=None, stream=None) -> None:
    """paged_decode_attn for callers that cannot allocate device memory: the
    split partials go to the library's fixed 32 MiB device scratch instead
    of a caller workspace. Calls share that scratch, so calls that overlap on
    the GPU must be serialized by the caller."""
    _bf16(q, "q"), _bf16(k_cache, "k_cache"), _bf16(v_cache, "v_cache"), _bf16(out, "out")
    _i32(dev_table, "dev_table"), _i32(batch_idx, "batch_idx"), _i32(seq_lens, "seq_lens")
    B, Hq, D = q.shape
    Hkv = k_cache.shape[0]
    _check(load_library().paged_decode_attn_noalloc(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(dev_table), n_slots, max_pages_per_seq,
        page_size, n_pages, _ptr(batch_idx), _ptr(seq_lens), int(window), float(scale), B, Hq,
        Hkv, D, int(num_splits), _ptr(out), _ptr(err_word), _stream(stream)),
        "paged_decode_attn_noalloc")


def convert_logical_block_mask(kv_indices, dev_table, n_slots, max_pages_per_seq,
                               batch_idx=None, n_cols=None, err_word=None, stream=None):
    """Logical -> physical key-block indices of a block mask (int32
    [B][H][rows][max_blocks], device) through the page table; returns int32
    [B][H][rows][n_cols] (n_cols defaults to max(max_blocks, max_pages_per_seq))."""
    _i32(kv_indices, "kv_indices"), _i32(dev_table, "dev_table"), _i32(batch_idx, "batch_idx")
    if kv_indices.dim() != 4:
        raise BadArgError("kv_indices must be [B][H][rows][max_blocks]")
    B, H, R, M = kv_indices.shape
    if n_cols is None:
        n_cols = max(M, max_pages_per_seq)
    out = torch.empty((B, H, R, n_cols), dtype=torch.int32, device=kv_indices.device)
    _check(load_library().convert_logical_block_mask(
        _ptr(dev_table), n_slots, max_pages_per_seq, _ptr(batch_idx), B, H, R, M,
        _ptr(kv_indices), n_cols, _ptr(out), _ptr(err_word), _stream(stream)),
        "convert_logical_block_mask")
    return out


PREFILL_BLOCK = 64


class PrefillBlockMask:
    """The block mask prefill_block_mask writes (int32 device tensors):
    kv_num_blocks [n], kv_indices [n][n] (partial blocks),
    full_kv_num_blocks [n], full_kv_indices [n][n], for n = ceil(L / 64),
    plus the docs and window it was built for."""

    __slots__ = ("kv_num_blocks", "kv_indices", "full_kv_num_blocks", "full_kv_indices",
                 "docs", "window")

    def __init__(self, kv_num_blocks, kv_indices, full_kv_num_blocks, full_kv_indices, docs,
                 window):
        self.kv_num_blocks = kv_num_blocks
        self.kv_indices = kv_indices
        self.full_kv_num_blocks = full_kv_num_blocks
        self.full_kv_indices = full_kv_indices
        self.docs = docs
        self.window = int(window)


def prefill_block_mask(docs, window: int = 0, stream=None) -> PrefillBlockMask:
    """Builds the document-causal (window > 0: sliding) block mask of the
    packed tokens' document ids docs (int32 [L], device)."""
    _i32(docs, "docs")
    L = docs.numel()
    n = -(-L // PREFILL_BLOCK)
    dev = docs.device
    bm = PrefillBlockMask(torch.empty(n, dtype=torch.int32, device=dev),
                          torch.empty((n, n), dtype=torch.int32, device=dev),
                          torch.empty(n, dtype=torch.int32, device=dev),
                          torch.empty((n, n), dtype=torch.int32, device=dev), docs, window)
    _check(load_library().prefill_block_mask(
        _ptr(docs), L, int(window), _ptr(bm.kv_num_blocks), _ptr(bm.kv_indices),
        _ptr(bm.full_kv_num_blocks), _ptr(bm.full_kv_indices), _stream(stream)),
        "prefill_block_mask")
    return bm


def prefill_attn(q, k, v, block_mask: PrefillBlockMask, scale, out, stream=None) -> None:
    """Document-causal attention over packed tokens: q [Hq][L][D], k/v
    [Hkv][L][D], out [Hq][L][D]; block_mask from prefill_block_mask (its docs
    and window are the mask's)."""
    _bf16(q, "q"), _bf16(k, "k"), _bf16(v, "v"), _bf16(out, "out")
    bm = block_mask
    for name in ("docs", "kv_num_blocks", "kv_indices", "full_kv_num_blocks",
                 "full_kv_indices"):
        _i32(getattr(bm, name), name)
    Hq, L, D = q.shape
    Hkv = k.shape[0]
    if bm.docs.numel() != L or bm.kv_num_blocks.numel() != -(-L // PREFILL_BLOCK):
        raise BadArgError("prefill_attn: block mask built for another length")
    _check(load_library().prefill_attn(
        _ptr(q), _ptr(k), _ptr(v), _ptr(bm.docs), _ptr(bm.kv_num_blocks), _ptr(bm.kv_indices),
        _ptr(bm.full_kv_num_blocks), _ptr(bm.full_kv_indices), L, Hq, Hkv, D, bm.window,
        float(scale), _ptr(out), _stream(stream)), "prefill_attn")


# --------------------------------------------------------------------------
# speculative steps: trees of drafted tokens
# --------------------------------------------------------------------------

TREE_MAX = 64

# Each call looks its tensors over in one go (_fits, _fits_i32: about 0.3 us a tensor) and only
# where something does not fit finds out what, and raises, in its _refuse_ function (with
# everything told apart first, the binding took 13.9 us for an append, 8.3 for an attention, 10.0
# for a verification, 41.2 for a move of 48 caches; so 6.4, 4.7, 4.8 and 20.3 with the call
# itself). The arguments go to the library in a record: one by one, ctypes took 2 us longer for
# the append's 31.

_RECORDS = {
    "tree_qkv_norm_rope_append": struct.Struct("@3P3q6P2f7iP4i5P"),
    "paged_tree_attn": struct.Struct("@4P4i4Pif5iPN3P"),
    "tree_verify": struct.Struct("@PqPq5P4i5P"),
    "kv_keep_path": struct.Struct("@3PiP4i4P2i2P"),
}
_pack_append, _pack_attn, _pack_verify, _pack_keep = (r.pack for r in _RECORDS.values())


# what a record does not hold, such as numbers beyond their type's range
_UNPACKABLE = (struct.error, OverflowError)


def _fits(t, dtype, shape, dev) -> bool:
    return (t.dtype is dtype and t.shape == shape and t.is_contiguous()
            and t.get_device() == dev)


def _fits_i32(t, n, dev) -> bool:
    return (t.dtype is _I32 and t.numel() >= n and t.is_contiguous()
            and t.get_device() == dev)


def _stream_on(stream, dev) -> int | None:
    """_stream of a call whose tensors are on the current device `dev`."""
    if stream is None and dev >= 0 and _raw_stream is not None:
        return _raw_stream(dev)
    return _stream(stream)


def _is_tensor(name, **tensors) -> None:
    """Refuses what is no tensor (missing ones too)."""
    for what, t in tensors.items():
        if not isinstance(t, torch.Tensor):
            raise BadArgError(f"{name}: {what} must be a tensor")


def _tree(name, N, row_start, parents) -> int:
    """Checks the packed trees of a call; returns the number of rows."""
    _at_least(name, "row_start", row_start, 1)
    _at_least(name, "parents", parents, N)
    return row_start.numel() - 1


def _tree_rows(name, B, batch_idx, ctx_lens) -> None:
    _at_least(name, "ctx_lens", ctx_lens, B)
    if batch_idx is not None:
        _at_least(name, "batch_idx", batch_idx, B)


def _at_least(name, what, t, n) -> None:
    _is_tensor(name, **{what: t})
    _i32(t, what)
    if t.numel() < n:
        raise BadArgError(f"{name}: {what} must hold {n} values")


def _tree_cache(name, k_cache, v_cache, dev_table, n_slots, max_pages_per_seq, page_size,
                n_pages) -> tuple:
    _is_tensor(name, k_cache=k_cache, v_cache=v_cache, dev_table=dev_table)
    _bf16(k_cache, "k_cache"), _bf16(v_cache, "v_cache"), _i32(dev_table, "dev_table")
    if k_cache.dim() != 3 or v_cache.shape != k_cache.shape or (
            k_cache.shape[1] != n_pages * page_size):
        raise BadArgError(f"{name}: k_cache and v_cache must both be [Hkv][n_pages * page_size]"
                          "[D]")
    if dev_table.numel() < n_slots * max_pages_per_seq:
        raise BadArgError(f"{name}: dev_table must be [n_slots][max_pages_per_seq]")
    return k_cache.shape[0], k_cache.shape[2]


def _tokens(name, what, t, heads, D) -> int:
    """Checks bf16 tokens [N][heads][D] whose rows may stand apart; returns their stride."""
    _is_tensor(name, **{what: t})
    if t.dtype is not _BF16 or t.dim() != 3 or t.shape[1] != heads or t.shape[2] != D:
        raise BadArgError(f"{name}: {what} must be a bfloat16 tensor [N][{heads}][{D}]")
    if t.shape[0] > 0 and (t.stride(2) != 1 or (heads > 1 and t.stride(1) != D)):
        raise BadArgError(f"{name}: {what}'s heads must be contiguous")
    return t.stride(0) if t.shape[0] > 1 else heads * D


def tree_qkv_norm_rope_append(q, k, v, gamma_q, gamma_k, batch_idx, ctx_lens, row_start, parents,
                              theta, eps, rotary_dims, v_norm, dev_table, n_slots,
                              max_pages_per_seq, page_size, n_pages, k_cache, v_cache, q_out,
                              err_word=None, stream=None) -> None:
    """Norm, rotation at ctx + depth and the paged append of every row's tree of
    drafted tokens (row_start int32 [B + 1], parents int32 [N]); q, k and v are
    bf16 [N][heads][D], rows of any stride, and only read; the rotated q goes to
    q_out. v None: the value is the raw k. rotary_dims None: all of D."""
    try:
        N, Hq, D = q.shape
        Hkv = k_cache.shape[0]
        rows = (Hkv, n_pages * page_size, D)
        dev = _raw_device() if q.is_cuda else None
        B = row_start.numel() - 1
        sq, hq, eq = q.stride()
        sk, hk, ek = k.stride()
        fits = (q.dtype is _BF16 and hq == D and eq == 1 and k.dtype is _BF16 and hk == D
                and ek == 1 and k.shape == (N, Hkv, D) and q.get_device() == dev
                and k.get_device() == dev and N > 1)
        sv = 0
        if v is not None:
            sv, hv, ev = v.stride()
            fits = (fits and v.dtype is _BF16 and hv == D and ev == 1 and v.shape == (N, Hkv, D)
                    and v.get_device() == dev)
        fits = (fits and _fits(k_cache, _BF16, rows, dev) and _fits(v_cache, _BF16, rows, dev)
                and _fits(q_out, _BF16, (N, Hq, D), dev)
                and (gamma_q is None or _fits(gamma_q, _BF16, (D,), dev))
                and (gamma_k is None or _fits(gamma_k, _BF16, (D,), dev))
                and (batch_idx is None or _fits_i32(batch_idx, B, dev))
                and _fits_i32(ctx_lens, B, dev) and _fits_i32(row_start, 1, dev)
                and _fits_i32(parents, N, dev)
                and _fits_i32(dev_table, n_slots * max_pages_per_seq, dev)
                and (err_word is None or _fits_i32(err_word, 1, dev)))
    except (AttributeError, TypeError, ValueError, IndexError):
        fits = False
    if not fits:
        B, N, Hq, Hkv, D, sq, sk, sv, dev = _refuse_append(
            q, k, v, gamma_q, gamma_k, batch_idx, ctx_lens, row_start, parents, dev_table, n_slots,
            max_pages_per_seq, page_size, n_pages, k_cache, v_cache, q_out, err_word)
    lib = _lib or load_library()
    try:
        status = lib.tree_qkv_norm_rope_append_args(_pack_append(
            q.data_ptr(), k.data_ptr(), 0 if v is None else v.data_ptr(), sq, sk, sv,
            0 if gamma_q is None else gamma_q.data_ptr(),
            0 if gamma_k is None else gamma_k.data_ptr(),
            0 if batch_idx is None else batch_idx.data_ptr(), ctx_lens.data_ptr(),
            row_start.data_ptr(), parents.data_ptr(), float(theta), float(eps),
            D if rotary_dims is None else int(rotary_dims), 1 if v_norm else 0, B, N, Hq, Hkv, D,
            dev_table.data_ptr(), n_slots, max_pages_per_seq, page_size, n_pages,
            k_cache.data_ptr(), v_cache.data_ptr(), q_out.data_ptr(),
            0 if err_word is None else err_word.data_ptr(), _stream_on(stream, dev) or 0))
    except _UNPACKABLE as e:
        raise BadArgError(f"tree_qkv_norm_rope_append: {e}") from None
    if status:
        _check(status, "tree_qkv_norm_rope_append")


def _refuse_append(q, k, v, gamma_q, gamma_k, batch_idx, ctx_lens, row_start, parents, dev_table,
                   n_slots, max_pages_per_seq, page_size, n_pages, k_cache, v_cache, q_out,
                   err_word):
    """What is wrong with an append's tensors; their sizes where nothing is."""
    name = "tree_qkv_norm_rope_append"
    Hkv, D = _tree_cache(name, k_cache, v_cache, dev_table, n_slots, max_pages_per_seq, page_size,
                         n_pages)
    _is_tensor(name, q=q, q_out=q_out)
    if q.dim() != 3:
        raise BadArgError(f"{name}: q must be [N][Hq][D]")
    N, Hq, _ = q.shape
    sq, sk = _tokens(name, "q", q, Hq, D), _tokens(name, "k", k, Hkv, D)
    sv = 0 if v is None else _tokens(name, "v", v, Hkv, D)
    _bf16(q_out, "q_out"), _bf16(gamma_q, "gamma_q"), _bf16(gamma_k, "gamma_k")
    if k.shape[0] != N or (v is not None and v.shape[0] != N) or q_out.shape != q.shape:
        raise BadArgError(f"{name}: q, k, v and q_out differ in tokens or heads")
    for g in (gamma_q, gamma_k):
        if g is not None and (not isinstance(g, torch.Tensor) or g.numel() != D):
            raise BadArgError(f"{name}: gains must be [D]")
    B = _tree(name, N, row_start, parents)
    _tree_rows(name, B, batch_idx, ctx_lens)
    _word(err_word)
    _on_device(q, k, v, gamma_q, gamma_k, batch_idx, ctx_lens, row_start, parents, dev_table,
               k_cache, v_cache, q_out, err_word)
    return B, N, Hq, Hkv, D, sq, sk, sv, q.get_device()


def paged_tree_attn_workspace(Hq, Hkv, D) -> int:
    return int(load_library().paged_tree_attn_workspace(Hq, Hkv, D))


def paged_tree_attn(q, k_cache, v_cache, dev_table, n_slots, max_pages_per_seq, page_size, n_pages,
                    batch_idx, ctx_lens, row_start, parents, window, scale, workspace, out,
                    err_word=None, stream=None) -> None:
    """Attention of every row's tree of drafted tokens (already appended) over the
    paged cache: a node sees the context and its own path. q, out: bf16
    [N][Hq][D]; workspace: a zeroed byte tensor of
    paged_tree_attn_workspace(Hq, Hkv, D)."""
    try:
        N, Hq, D = q.shape
        Hkv = k_cache.shape[0]
        rows = (Hkv, n_pages * page_size, D)
        dev = _raw_device() if q.is_cuda else None
        B = row_start.numel() - 1
        fits = (_fits(q, _BF16, (N, Hq, D), dev) and _fits(out, _BF16, (N, Hq, D), dev)
                and _fits(k_cache, _BF16, rows, dev) and _fits(v_cache, _BF16, rows, dev)
                and (batch_idx is None or _fits_i32(batch_idx, B, dev))
                and _fits_i32(ctx_lens, B, dev) and _fits_i32(row_start, 1, dev)
                and _fits_i32(parents, N, dev)
                and _fits_i32(dev_table, n_slots * max_pages_per_seq, dev)
                and workspace.is_contiguous() and workspace.get_device() == dev
                and (err_word is None or _fits_i32(err_word, 1, dev)))
    except (AttributeError, TypeError, ValueError):
        fits = False
    if not fits:
        B, N, Hq, Hkv, D, dev = _refuse_attn(
            q, k_cache, v_cache, dev_table, n_slots, max_pages_per_seq, page_size, n_pages,
            batch_idx, ctx_lens, row_start, parents, workspace, out, err_word)
    lib = _lib or load_library()
    try:
        status = lib.paged_tree_attn_args(_pack_attn(
            q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), dev_table.data_ptr(), n_slots,
            max_pages_per_seq, page_size, n_pages, 0 if batch_idx is None else batch_idx.data_ptr(),
            ctx_lens.data_ptr(), row_start.data_ptr(), parents.data_ptr(), int(window),
            float(scale), B, N, Hq, Hkv, D, workspace.data_ptr(), workspace.nbytes, out.data_ptr(),
            0 if err_word is None else err_word.data_ptr(), _stream_on(stream, dev) or 0))
    except _UNPACKABLE as e:
        raise BadArgError(f"paged_tree_attn: {e}") from None
    if status:
        _check(status, "paged_tree_attn")


def _refuse_attn(q, k_cache, v_cache, dev_table, n_slots, max_pages_per_seq, page_size, n_pages,
                 batch_idx, ctx_lens, row_start, parents, workspace, out, err_word):
    """What is wrong with an attention's tensors; their sizes where nothing is."""
    name = "paged_tree_attn"
    Hkv, D = _tree_cache(name, k_cache, v_cache, dev_table, n_slots, max_pages_per_seq, page_size,
                         n_pages)
    _is_tensor(name, q=q, out=out, workspace=workspace)
    _bf16(q, "q"), _bf16(out, "out")
    if q.dim() != 3 or q.shape[2] != D or out.shape != q.shape:
        raise BadArgError(f"{name}: q, out and the caches differ in shape")
    if not workspace.is_contiguous():
        raise BadArgError(f"{name}: workspace must be a contiguous tensor")
    N, Hq, _ = q.shape
    B = _tree(name, N, row_start, parents)
    _tree_rows(name, B, batch_idx, ctx_lens)
    _word(err_word)
    _on_device(q, k_cache, v_cache, dev_table, batch_idx, ctx_lens, row_start, parents, workspace,
               out, err_word)
    return B, N, Hq, Hkv, D, q.get_device()


def _probs(name, what, t, N, V=None) -> int:
    """Checks fp32 rows [N][V] that may stand apart; returns their stride."""
    _is_tensor(name, **{what: t})
    if t.dtype is not _F32 or t.dim() != 2 or t.shape[0] < N or (V is not None and t.shape[1] != V):
        raise BadArgError(f"{name}: {what} must be a float32 tensor [N][V]")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise BadArgError(f"{name}: {what}'s rows must be contiguous")
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def tree_verify(target_probs, draft_probs, tokens, row_start, parents, u_accept, u_pick, accepted,
                path, next_token, err_word=None, stream=None) -> None:
    """Which drafted tokens the target accepts, and the token behind them, from the
    given uniform numbers. target_probs, draft_probs: fp32 [N][V], the
    distribution after each node (draft_probs None: drafts chosen without
    chance); tokens int32 [N]; u_accept fp32 [N], u_pick fp32 [B]. Writes accepted
    int32 [B], path int32 [B][cols] (node 0 and the accepted drafts, then -1) and
    next_token int32 [B]."""
    try:
        N, B, V = tokens.numel(), row_start.numel() - 1, target_probs.shape[1]
        dev = _raw_device() if tokens.is_cuda else None
        sp, one = target_probs.stride()
        fits = (target_probs.dtype is _F32 and one == 1 and target_probs.shape[0] >= N > 1
                and target_probs.get_device() == dev
                and _fits_i32(tokens, N, dev) and _fits_i32(row_start, 1, dev)
                and _fits_i32(parents, N, dev) and _fits_i32(accepted, B, dev)
                and _fits_i32(next_token, B, dev)
                and u_accept.dtype is _F32 and u_accept.numel() >= N and u_accept.is_contiguous()
                and u_accept.get_device() == dev
                and u_pick.dtype is _F32 and u_pick.numel() >= B and u_pick.is_contiguous()
                and u_pick.get_device() == dev
                and (err_word is None or _fits_i32(err_word, 1, dev)))
        cols = path.shape[1]
        fits = fits and path.shape[0] >= B and cols > 0 and _fits_i32(path, 1, dev)
        sq = 0
        if draft_probs is not None:
            sq, one = draft_probs.stride()
            fits = (fits and draft_probs.dtype is _F32 and one == 1
                    and draft_probs.shape[0] >= N and draft_probs.shape[1] == V
                    and draft_probs.get_device() == dev)
    except (AttributeError, TypeError, ValueError, IndexError):
        fits = False
    if not fits:
        B, N, V, cols, sp, sq, dev = _refuse_verify(
            target_probs, draft_probs, tokens, row_start, parents, u_accept, u_pick, accepted, path,
            next_token, err_word)
    lib = _lib or load_library()
    try:
        status = lib.tree_verify_args(_pack_verify(
            target_probs.data_ptr(), sp, 0 if draft_probs is None else draft_probs.data_ptr(), sq,
            tokens.data_ptr(), row_start.data_ptr(), parents.data_ptr(), u_accept.data_ptr(),
            u_pick.data_ptr(), B, N, V, cols, accepted.data_ptr(), path.data_ptr(),
            next_token.data_ptr(), 0 if err_word is None else err_word.data_ptr(),
            _stream_on(stream, dev) or 0))
    except _UNPACKABLE as e:
        raise BadArgError(f"tree_verify: {e}") from None
    if status:
        _check(status, "tree_verify")


def _refuse_verify(target_probs, draft_probs, tokens, row_start, parents, u_accept, u_pick,
                   accepted, path, next_token, err_word):
    """What is wrong with a verification's tensors; their sizes where nothing is."""
    name = "tree_verify"
    _is_tensor(name, tokens=tokens)
    N = tokens.numel()
    _i32(tokens, "tokens")
    sp = _probs(name, "target_probs", target_probs, N)
    V = target_probs.shape[1]
    sq = 0 if draft_probs is None else _probs(name, "draft_probs", draft_probs, N, V)
    B = _tree(name, N, row_start, parents)
    for what, t, n in (("u_accept", u_accept, N), ("u_pick", u_pick, B)):
        _is_tensor(name, **{what: t})
        if t.dtype is not _F32 or not t.is_contiguous() or t.numel() < n:
            raise BadArgError(f"{name}: {what} must be a contiguous float32 tensor of {n} values")
    _at_least(name, "accepted", accepted, B)
    _at_least(name, "next_token", next_token, B)
    _is_tensor(name, path=path)
    _i32(path, "path")
    if path.dim() != 2 or path.shape[0] < B or path.shape[1] < 1:
        raise BadArgError(f"{name}: path must be [B][cols]")
    _word(err_word)
    _on_device(target_probs, draft_probs, tokens, row_start, parents, u_accept, u_pick, accepted,
               path, next_token, err_word)
    return B, N, V, path.shape[1], sp, sq, tokens.get_device()


def kv_keep_path(caches, dev_table, n_slots, max_pages_per_seq, page_size, n_pages, batch_idx,
                 ctx_lens, accepted, path, err_word=None, stream=None) -> None:
    """After tree_verify: the accepted nodes' tokens move to the positions behind the
    context, in every head of every cache in `caches` (contiguous device tensors
    [heads][n_pages * page_size][...], any element type, all the layers of a
    model; one that is named twice moves once). The rows are path's: of a path kept for more rows than tree_verify was
    given, pass those alone (path[:B]), for the others would move once more."""
    try:
        B, cols = path.shape
        dev = _raw_device() if path.is_cuda else None
        fits = (cols > 0 and _fits_i32(path, 1, dev) and _fits_i32(accepted, B, dev)
                and (batch_idx is None or _fits_i32(batch_idx, B, dev))
                and _fits_i32(ctx_lens, B, dev)
                and _fits_i32(dev_table, n_slots * max_pages_per_seq, dev)
                and (err_word is None or _fits_i32(err_word, 1, dev)))
        # the caches of a model are alike: each is told from the first by shape and type
        n, first = len(caches), caches[0]
        shape, rows = first.shape, n_pages * page_size
        fits = (fits and shape[1] == rows and shape[0] > 0
                and list(map(_T.size, caches)) == [shape] * n
                and list(map(_dtype_of, caches)) == [first.dtype] * n
                and all(map(_T.is_contiguous, caches))
                and list(map(_T.get_device, caches)) == [dev] * n
                and not isinstance(caches, _T))
    except (AttributeError, TypeError, ValueError, IndexError):
        fits = False
    if fits:
        ptrs = array.array("Q", map(_T.data_ptr, caches))
        heads = array.array("i", shape[:1]) * n
        nbytes = array.array("q", (first.nbytes // (shape[0] * rows),)) * n
    else:
        B, cols, n, ptrs, heads, nbytes, dev = _refuse_keep(
            caches, dev_table, n_slots, max_pages_per_seq, page_size, n_pages, batch_idx, ctx_lens,
            accepted, path, err_word)
    lib = _lib or load_library()
    try:
        status = lib.kv_keep_path_args(_pack_keep(
            ptrs.buffer_info()[0], heads.buffer_info()[0], nbytes.buffer_info()[0], n,
            dev_table.data_ptr(), n_slots, max_pages_per_seq, page_size, n_pages,
            0 if batch_idx is None else batch_idx.data_ptr(), ctx_lens.data_ptr(),
            accepted.data_ptr(), path.data_ptr(), cols, B,
            0 if err_word is None else err_word.data_ptr(), _stream_on(stream, dev) or 0))
    except _UNPACKABLE as e:
        raise BadArgError(f"kv_keep_path: {e}") from None
    if status:
        _check(status, "kv_keep_path")


_T = torch.Tensor
_dtype_of = operator.attrgetter("dtype")


def _refuse_keep(caches, dev_table, n_slots, max_pages_per_seq, page_size, n_pages, batch_idx,
                 ctx_lens, accepted, path, err_word):
    """What is wrong with a move's tensors; their sizes where nothing is."""
    name = "kv_keep_path"
    _is_tensor(name, dev_table=dev_table, path=path)
    _i32(dev_table, "dev_table"), _i32(path, "path")
    if path.dim() != 2 or path.shape[1] < 1:
        raise BadArgError(f"{name}: path must be [B][cols]")
    B = path.shape[0]
    _at_least(name, "accepted", accepted, B)
    _tree_rows(name, B, batch_idx, ctx_lens)
    if dev_table.numel() < n_slots * max_pages_per_seq:
        raise BadArgError(f"{name}: dev_table must be [n_slots][max_pages_per_seq]")
    rows = n_pages * page_size
    ptrs, heads, nbytes = array.array("Q"), array.array("i"), array.array("q")
    try:
        if isinstance(caches, torch.Tensor):
            raise TypeError
        for c in caches:
            if not c.is_contiguous() or c.dim() < 2 or c.shape[1] != rows:
                raise BadArgError(f"{name}: caches must be contiguous tensors [heads][n_pages * "
                                  "page_size][...]")
            h = c.shape[0]
            ptrs.append(c.data_ptr()), heads.append(h), nbytes.append(c.nbytes // max(h * rows, 1))
    except (AttributeError, TypeError):
        raise BadArgError(f"{name}: caches must be a list of tensors") from None
    _word(err_word)
    _on_device(dev_table, batch_idx, ctx_lens, accepted, path, err_word, *caches)
    return B, path.shape[1], len(ptrs), ptrs, heads, nbytes, path.get_device()


def pkv_read_error_word(err_word, stream=None) -> int:
    v = ctypes.c_int32()
    _check(load_library().pkv_read_error_word(_ptr(err_word), _stream(stream), ctypes.byref(v)),
           "pkv_read_error_word")
    return v.value


def pkv_last_error() -> str:
    return load_library().pkv_last_error().decode(errors="replace")
