"""Lists of caches and of pairs that kv_copy_pages refuses as bad arguments (no GPU needed)."""
import numpy as np
import pytest
import torch

pkv = pytest.importorskip("paged_kv_decode_pagetable_gb300")
FP8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def lib():
    pkv.load_library()


@pytest.mark.parametrize("caches", [torch.zeros((2, 4, 8), dtype=FP8), None, [None], [1 << 20],
                                    [torch.zeros((2, 4, 8)), [1.0]], 5])
def test_caches(caches):
    """A single tensor is not a list of caches: its heads would be taken for caches, and
    their rows for heads."""
    with pytest.raises(pkv.BadArgError, match="caches"):
        pkv.kv_copy_pages(caches, 4, [(1, 2)])


@pytest.mark.parametrize("pairs", [None, 7, [(1, 2, 3)], [1, 2, 3], torch.zeros((1, 2)), [(1.5, 2)],
                                   [(1, 2 ** 40)], ["ab"]])
def test_pairs(pairs):
    with pytest.raises(pkv.BadArgError, match="pairs"):
        pkv.kv_copy_pages([], 4, pairs)


@pytest.mark.parametrize("pairs", [np.array([[1, 2], [3, 0]], np.int32), [(1, 2)], ((1, 2), (3, 0)),
                                   np.array([[1, 2]]), [np.array([1, 2], np.int16)], [],
                                   np.zeros((0, 2), np.int32), iter([(1, 2)]),
                                   torch.tensor([[1, 2]], dtype=torch.int32)])
def test_whole_numbers_of_any_kind_are_taken(pairs):
    pkv.kv_copy_pages([], 4, pairs)
