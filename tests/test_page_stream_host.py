"""The stream of a page table's copies, as the library reports it (no GPU needed)."""
import ctypes

import pytest

pkv = pytest.importorskip("paged_kv_decode_pagetable_gb300")


def test_get_stream():
    lib = pkv.load_library()
    pt = pkv.PageTable(2, 4, 8, 3)
    assert pkv.pt_get_stream(pt.handle) == 0
    pkv.pt_set_stream(pt.handle, 0x7f0000000010)      # never used: the table is on the host
    assert pkv.pt_get_stream(pt.handle) == 0x7f0000000010
    s = ctypes.c_void_p()
    assert lib.pt_get_stream(None, ctypes.byref(s)) == pkv.PKV_E_BAD_ARG
    assert lib.pt_get_stream(pt.handle, None) == pkv.PKV_E_BAD_ARG
