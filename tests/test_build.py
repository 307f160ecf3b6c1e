"""What the build leaves where a part of it cannot be made.  No GPU needed."""
import os
import types

import pytest
import torch

from free_block_sparse_predict_b200 import build, serving


def test_the_c_library_does_not_wait_for_the_binding(monkeypatch, tmp_path):
    """Without torch's headers or a host compiler the extension module fails; libsparge.so is there
    all the same, and the failure is still reported."""
    build.build()

    def fails():
        raise RuntimeError("g++ failed")

    monkeypatch.setattr(build, "_binding", fails)
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libsparge.so"))
    with pytest.raises(RuntimeError, match="g.. failed"):
        build.build()
    assert os.path.getsize(build.LIB) > 1 << 20


def test_the_binding_is_made_for_one_interpreter_and_one_torch(monkeypatch, tmp_path):
    src = os.path.join(build.CSRC, "serving_binding.cpp")
    build.build()
    assert build._binding_is_current(src)
    assert os.path.basename(build.BINDING).startswith("_serving.cpython-")
    for text in (None, "1.0"):
        monkeypatch.setattr(build, "STAMP", str(tmp_path / str(text)))
        if text is not None:
            (tmp_path / text).write_text(text)
        assert not build._binding_is_current(src)


def test_a_binding_for_another_torch_is_refused(monkeypatch):
    other = types.SimpleNamespace(torch_version="1.0", setup=lambda *a: None)
    monkeypatch.setattr(serving.importlib, "import_module", lambda *a: other)
    with pytest.raises(ImportError, match="built for torch 1.0"):
        serving._load()
    other.torch_version = str(torch.__version__)
    monkeypatch.setattr(serving, "_serving", None)
    assert serving._load() is other
