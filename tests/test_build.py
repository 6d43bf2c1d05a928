"""The build: the library does not depend on the Python entry's compiler and
headers, and an entry of another torch or Python is built again."""
import os
import shutil
import sys

import pytest

from attention_forward_14_gb300 import binding, build as B

pytestmark = pytest.mark.skipif(shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"),
                                reason="no nvcc")


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A library of one small source and an entry, in a folder of their own."""
    csrc = tmp_path / "csrc"
    csrc.mkdir()
    (csrc / "small.cu").write_text('extern "C" int small() { return 7; }\n')
    (csrc / "marshal.cpp").write_text('extern "C" int entry() { return 8; }\n')
    monkeypatch.setattr(B, "CSRC", str(csrc))
    monkeypatch.setattr(B, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(B, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(B, "LIB_CHECKED", str(tmp_path / "lib_checked.so"))
    monkeypatch.setattr(B, "MARSHAL", str(tmp_path / "entry.so"))
    monkeypatch.setattr(B, "SOURCES", ["small.cu"])
    monkeypatch.setattr(B, "CHECKED_SOURCES", ["small.cu"])
    return tmp_path


@pytest.mark.parametrize("lacks", ["compiler", "torch", "Python.h"])
def test_the_library_is_built_without_what_the_entry_needs(tree, monkeypatch, capfd, lacks):
    (tree / "entry.so").write_text("of an earlier build")
    if lacks == "compiler":
        monkeypatch.setenv("CXX", str(tree / "no-such-compiler"))
    elif lacks == "torch":
        monkeypatch.setattr(B, "_torch_dir", lambda: None)
    else:
        monkeypatch.setattr(B.sysconfig, "get_paths", lambda: {"include": str(tree)})
    assert B.build() == B.LIB and os.path.exists(B.LIB) and os.path.exists(B.LIB_CHECKED)
    assert not os.path.exists(B.MARSHAL) and "not built" in capfd.readouterr().err


def test_an_entry_that_does_not_compile_is_an_error_after_the_library_is_there(tree):
    (tree / "csrc" / "marshal.cpp").write_text("this is no C++\n")
    with pytest.raises(RuntimeError, match="marshal.cpp failed to compile"):
        B.build()
    assert os.path.exists(B.LIB) and not os.path.exists(B.MARSHAL)


def test_an_entry_for_another_torch_is_built_again(tree, monkeypatch):
    built = []
    link = B._link_marshal
    monkeypatch.setattr(B, "_link_marshal", lambda obj: (built.append(obj), link(obj)))
    B.build()
    B.build()
    assert len(built) == 1
    now = B._marshal_built_for()
    monkeypatch.setattr(B, "_marshal_built_for", lambda: now + " and more")
    B.build()
    B.build()
    assert len(built) == 2
    monkeypatch.setattr(B, "_marshal_built_for", lambda: now)
    os.remove(os.path.join(B.BUILD, B.MARSHAL_STAMP))
    B.build()
    assert len(built) == 3


def test_operators_say_that_the_entry_is_missing(monkeypatch):
    import attention_forward_14_gb300 as af
    monkeypatch.setattr(binding, "_lib", object())
    monkeypatch.setattr(binding, "_fast_lib", None)
    monkeypatch.delattr(af, "_marshal_ext", raising=False)
    monkeypatch.setitem(sys.modules, "attention_forward_14_gb300._marshal_ext", None)
    with pytest.raises(af.AttnError) as e:
        af.attn_qk_norm_rope(None, None)
    assert e.value.code == -8 and "_marshal_ext" in str(e.value)
