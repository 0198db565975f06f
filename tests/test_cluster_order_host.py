"""Kernels whose CTAs write into one another's shared memory: they may do so only once all CTAs
of the cluster are known to run. A CTA that starts late shows on no ordinary run, so the order is
looked up in the source: a wait for the cluster stands before the first remote address."""
import pathlib
import re

import pytest

CSRC = pathlib.Path(__file__).resolve().parents[1] / "paged_kv_decode_pagetable_gb300" / "csrc"
REMOTE = r"map_shared_rank|\bmapa\b"
WAIT = r"cluster\.sync\(|cluster\.barrier_wait\(|barrier\.cluster\.wait"


def code(path):
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", path.read_text(), flags=re.S)


FILES = sorted(p.name for p in CSRC.glob("*.cu*") if re.search(REMOTE, code(p)))


def test_some_kernels_do():
    assert "tree_verify.cu" in FILES


@pytest.mark.parametrize("name", FILES)
def test_the_cluster_runs_before_its_shared_memory_is_used(name):
    text = code(CSRC / name)
    first = re.search(REMOTE, text).start()
    assert re.search(WAIT, text[:first]), f"{name}: no wait for the cluster before {text[first:][:60]}"
