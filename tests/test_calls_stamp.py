"""The compiled marshalling is built again for another Python or torch, not only for
newer sources."""
import os
import shutil

from bitlinear_b1_fwd_b200 import build


def test_stamp_decides(tmp_path, monkeypatch):
    build.build()
    assert not build.calls_stale()
    copy = tmp_path / "_calls.so"
    shutil.copy2(build.CALLS, copy)
    assert not build.calls_stale(str(copy))
    stamp = build.calls_stamp()
    for other in (stamp.replace("cpython-", "cpython-9"), stamp.replace("torch ", "torch 9."), stamp + "7"):
        assert other != stamp
        monkeypatch.setattr(build, "calls_stamp", lambda text=other: text)
        assert build.calls_stale(str(copy))
    monkeypatch.undo()
    os.utime(copy, (1, 1))
    assert build.calls_stale(str(copy))         # older than its sources
    assert build.calls_stale(str(tmp_path / "none.so"))


def test_module_says_what_it_was_built_for():
    from bitlinear_b1_fwd_b200 import binding
    build.build()
    assert binding._calls().built_for == build.calls_stamp()
