"""What the build leaves where a part of it cannot be made.  No GPU needed."""
import os

import pytest

from free_block_sparse_predict_b200 import build


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
