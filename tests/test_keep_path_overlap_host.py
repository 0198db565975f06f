"""kv_keep_path moves in place, each cache by CTAs of its own: caches that overlap are refused by
the library before anything runs. No GPU: the addresses are never followed."""
import ctypes

import pytest

pkv = pytest.importorskip("paged_kv_decode_pagetable_gb300")

A, ROWS, TOKEN, HEADS = 1 << 20, 64, 128, 2
SIZE = HEADS * ROWS * TOKEN


def call(bases, heads=None, nbytes=None):
    n = len(bases)
    arrays = ((ctypes.c_void_p * n)(*bases), (ctypes.c_int * n)(*(heads or [HEADS] * n)),
              (ctypes.c_int64 * n)(*(nbytes or [TOKEN] * n)))
    lib = pkv.load_library()
    return lib.kv_keep_path(*arrays, n, A, 3, 2, 16, ROWS // 16, A, A, A, A, 4, 2, None,
                            None), lib.pkv_last_error().decode()


@pytest.mark.parametrize("bases,heads,nbytes", [
    ([A, A + 16], None, None),
    ([A, A + SIZE - 1], None, None),
    ([A + SIZE - 1, A], None, None),
    ([A, A], [2, 1], None),                              # a part of its heads
    ([A, A], None, [TOKEN, TOKEN // 2]),                 # other tokens
    ([A, A + SIZE // 2], [2, 1], None),                  # its second head
    ([A, A + 4 * SIZE, A + 2 * SIZE, A + 3 * SIZE - 16], None, None),
    ([A + i * SIZE for i in range(200)] + [A + 150 * SIZE + 8], None, None),
    ([A, A, A + 16], None, None)])
def test_overlaps_are_refused(bases, heads, nbytes):
    status, said = call(bases, heads, nbytes)
    assert status == pkv.PKV_E_BAD_ARG and "overlap" in said

