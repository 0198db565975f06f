"""engine.accept_drafts on buffers kept for more rows than a step has: verification and move
handle the same rows. No GPU: the library's calls are recorded."""
import pytest
import torch

pkv = pytest.importorskip("paged_kv_decode_pagetable_gb300")
from paged_kv_decode_pagetable_gb300 import engine  # noqa: E402

I32 = torch.int32


class Recorder:
    def __init__(self):
        self.calls = {}

    def __getattr__(self, name):
        def call(record):
            self.calls[name] = pkv._RECORDS[name.removesuffix("_args")].unpack(record)
            return pkv.PKV_OK
        return call


@pytest.mark.parametrize("rows,kept", [(3, 8), (8, 8), (0, 8), (1, 2)])
def test_both_calls_have_the_steps_rows(rows, kept, monkeypatch):
    lib = Recorder()
    monkeypatch.setattr(pkv, "_lib", lib)
    monkeypatch.setattr(pkv, "_on_device", lambda *t: None)
    pt = type("Geometry", (), dict(dev_table=torch.zeros((9, 2), dtype=I32), n_slots=9,
                                   max_pages_per_seq=2, page_size=16, n_pages=4))
    i32 = lambda *s: torch.zeros(s, dtype=I32)  # noqa: E731
    path = i32(kept, 4)
    engine.accept_drafts(pt, [torch.zeros((2, 64, 64), dtype=torch.bfloat16)], torch.zeros(6, 9),
                         None, i32(6), i32(kept), i32(kept), i32(rows + 1), i32(6), torch.zeros(6),
                         torch.zeros(kept), i32(kept), path, i32(kept))
    verify, keep = lib.calls["tree_verify_args"], lib.calls["kv_keep_path_args"]
    assert verify[9] == keep[14] == rows           # their B
    assert verify[12] == keep[13] == 4             # the path's columns
    assert verify[14] == path.data_ptr()
    assert rows == 0 or keep[12] == path.data_ptr()
