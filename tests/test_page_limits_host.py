"""Page tables at the ends of an int and of memory (no GPU needed): refused or right, never
an exception through the C entry, which would end the process."""
import subprocess
import sys

import pytest

pkv = pytest.importorskip("paged_kv_decode_pagetable_gb300")
MOST = (1 << 31) - 1


def test_tables_too_large_are_refused():
    """In a process of its own, which an exception would end."""
    code = ("import paged_kv_decode_pagetable_gb300 as pkv\n"
            "for a in ((1 << 30, 1, 100, 1 << 30), ((1 << 31) - 1, 1, 100, 1)):\n"
            "    try: pkv.pt_create(*a)\n"
            "    except pkv.BadArgError: print('refused')\n")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.split() == ["refused"] * 2, r.stderr[-500:]


def test_the_longest_sequences():
    pt = pkv.PageTable(4, 16, 100, 8)
    free = pt.free_page_list()
    assert not pt.can_reserve(MOST)
    with pytest.raises(pkv.BadArgError):
        pt.assign(MOST)
    assert pt.free_page_list() == free
    s = pt.assign(16)
    assert not pt.can_reserve(MOST, s)
    for n in (MOST, MOST - 15, MOST - 16):
        with pytest.raises(pkv.BadArgError):
            pt.reserve(s, n)
    assert pt.capacity(s) == 16 and len(pt.free_page_list()) == 98


def test_a_capacity_past_an_int_is_refused():
    """Pages of 2^30 tokens: one fits a sequence, two would hold 2^31."""
    pt = pkv.PageTable(2, 1 << 30, 8, 5)
    assert pt.can_reserve(1 << 30) and not pt.can_reserve((1 << 30) + 1)
    with pytest.raises(pkv.BadArgError):
        pt.assign((1 << 30) + 1)
    s = pt.assign(1 << 30)
    assert pt.capacity(s) == 1 << 30 and len(pt.pages(s)) == 1
    assert not pt.can_reserve(MOST, s)
    with pytest.raises(pkv.BadArgError):
        pt.reserve(s, MOST)
    (f,), pairs = pt.fork(s, (1 << 30) - 1)
    assert len(pairs) == 1 and pt.capacity(f) == 1 << 30
    pt.truncate(s, 0)
    pt.free(f)
    assert len(pt.free_page_list()) == 7
