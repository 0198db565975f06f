"""Lists of caches and of pairs that kv_copy_pages refuses as bad arguments (no GPU needed)."""
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
