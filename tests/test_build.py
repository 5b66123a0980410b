"""What a build needs and when it is current, on a small source tree: libgdn.so from nvcc alone, the
layer operators' binding for the torch and the Python that are there."""
import os
import sys

import pytest

from linear_attention_prefill_gb300 import _build

GOOD = "#include <Python.h>\n#include <torch/version.h>\nextern \"C\" int layer_operators() { return 1; }\n"


@pytest.fixture
def tree(tmp_path, monkeypatch):
    csrc = tmp_path / "pkg" / "csrc"
    csrc.mkdir(parents=True)
    (tmp_path / "include").mkdir()
    (tmp_path / "include" / "gdn.h").write_text("")
    (csrc / "one.cu").write_text("extern \"C\" int one() { return 1; }\n")
    (csrc / "layer_binding.cpp").write_text(GOOD)
    pkg = str(tmp_path / "pkg")
    for name, value in dict(PKG=pkg, CSRC=str(csrc), BUILD=os.path.join(pkg, "_build"),
                            LIB=os.path.join(pkg, "libgdn.so"), BINDING=os.path.join(pkg, "_layer_native.so"),
                            BINDING_SRC=str(csrc / "layer_binding.cpp"),
                            BINDING_FOR=os.path.join(pkg, "_build", "_layer_native.txt")).items():
        monkeypatch.setattr(_build, name, value)
    return csrc


def test_library_without_torch(tree, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)  # import torch: ImportError
    assert _build.binding_key() is None
    assert _build.build() == _build.LIB and os.path.exists(_build.LIB)
    assert not os.path.exists(_build.BINDING) and _build.up_to_date()


def test_library_without_cuda_in_torch(tree, monkeypatch):
    import torch
    monkeypatch.setattr(torch.version, "cuda", None)
    _build.build()
    assert os.path.exists(_build.LIB) and not os.path.exists(_build.BINDING) and _build.up_to_date()


def test_library_beside_a_binding_that_does_not_compile(tree):
    (tree / "layer_binding.cpp").write_text("#error no\n")
    with pytest.raises(RuntimeError, match="layer_binding"):
        _build.build()
    assert os.path.exists(_build.LIB) and not os.path.exists(_build.BINDING)
    assert not _build.up_to_date()


def test_binding_is_current_for_one_torch_and_one_python(tree, monkeypatch):
    import sysconfig

    import torch
    _build.build()
    assert _build.up_to_date() and _build.binding_built_for() == _build.binding_key()
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "0.0.1+other")
        assert not _build.up_to_date()
    var = sysconfig.get_config_var
    with monkeypatch.context() as m:
        m.setattr(sysconfig, "get_config_var", lambda n: "cpython-399" if n == "SOABI" else var(n))
        assert not _build.up_to_date()
    assert _build.up_to_date()
    os.remove(_build.BINDING_FOR)
    assert not _build.up_to_date()
    _build.build()
    assert _build.up_to_date()
    os.utime(_build.LIB, (1, 1))
    assert not _build.up_to_date()


def test_a_binding_of_another_torch_is_not_loaded(monkeypatch):
    from linear_attention_prefill_gb300 import layer
    _build.build()
    monkeypatch.setattr(layer, "_native", None)
    monkeypatch.setattr(_build, "binding_built_for", lambda: "torch 0.0.1 cpython-399")
    with pytest.raises(RuntimeError, match="0.0.1"):
        layer._load()
