"""The paged-cache binding is rebuilt when what it is compiled against changes, not only its
sources."""
import os

import torch

from adaptive_sparse_attention_b200 import build


def test_binding_is_rebuilt_for_another_torch(monkeypatch):
    build.build()
    assert not build.binding_stale()
    before = os.path.getmtime(build.BINDING)
    assert build.build_binding() == build.BINDING and os.path.getmtime(build.BINDING) == before
    monkeypatch.setattr(torch, "__version__", "0.0.0")
    assert build.binding_stale()


def test_binding_is_rebuilt_without_a_record_of_its_build(monkeypatch, tmp_path):
    build.build()
    monkeypatch.setattr(build, "BINDING_STAMP", str(tmp_path / "none"))
    assert build.binding_stale()
