"""CPU checks of the build: which parts a machine gets."""
import os

import pytest

from tiled_top_sparse_gb300 import _build


@pytest.fixture()
def parts(monkeypatch, tmp_path):
    """The build with stand-ins for its outputs: the library counts as built."""
    monkeypatch.setattr(_build, "NATIVE", str(tmp_path / "_native.so"))
    monkeypatch.setattr(_build, "up_to_date", lambda: True)
    return tmp_path


def test_library_without_python_headers(parts, monkeypatch, capsys):
    """Without Python's C headers the library is built all the same; the binding is left out, which is
    said."""
    monkeypatch.setattr(_build.sysconfig, "get_paths", lambda: {"include": str(parts)})
    assert _build.build() == _build.LIB
    assert not os.path.exists(_build.NATIVE)
    assert "Python.h" in capsys.readouterr().err


def test_library_comes_first(parts, monkeypatch):
    """An error in the binding's build does not keep the library from being built, and is raised."""
    order = []
    monkeypatch.setattr(_build, "up_to_date", lambda: order.append("library") or True)
    monkeypatch.setenv("CC", "false")
    with pytest.raises(RuntimeError, match="false"):
        _build.build()
    assert order == ["library"]


def test_binding_is_built(parts):
    assert _build.build_native() == _build.NATIVE and os.path.exists(_build.NATIVE)


def test_a_missing_binding_is_an_error(monkeypatch):
    """The grouped-query calls of a tree without the binding raise."""
    import sys

    import torch

    import tiled_top_sparse_gb300 as tts
    monkeypatch.setattr(tts, "_nat", None)
    monkeypatch.setitem(sys.modules, "tiled_top_sparse_gb300._native", None)
    monkeypatch.delattr(tts, "_native", raising=False)
    x = torch.zeros(1, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ImportError, match="not built"):
        tts.rope_kv_append(x, x, x, x, x, x, x, 1)


def test_the_projection_with_axes_needs_no_binding(monkeypatch):
    """As the one without axes: what it refuses without the binding is the tensors, not the call."""
    import sys

    import torch

    import tiled_top_sparse_gb300 as tts
    monkeypatch.setattr(tts, "_nat", None)
    monkeypatch.setitem(sys.modules, "tiled_top_sparse_gb300._native", None)
    monkeypatch.delattr(tts, "_native", raising=False)
    x = torch.zeros(3, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="x must be a CUDA tensor"):
        tts.qkv_rope_axes(x, torch.zeros(3 * 64, 64, dtype=torch.bfloat16), None,
                          torch.zeros(2, 3, dtype=torch.int32), bytes(32), torch.zeros(9, 32, 2), 1)
