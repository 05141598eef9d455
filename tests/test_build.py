"""The build on a machine without a GPU: what is compiled when.  The compilers are replaced by a stand-in that writes the
file that they are asked for."""
import importlib.util
import os
import types

import pytest

from sparse_attention_indexer_e4m3_gb300 import build


@pytest.fixture
def place(tmp_path, monkeypatch):
    """The build's outputs under a temporary folder, and the names of what is compiled, in a list."""
    made = []

    def run(cmd, **kw):
        out = cmd[cmd.index("-o") + 1]
        made.append("link" if "-shared" in cmd and out.startswith(build.LIB_PATH) else os.path.basename(next(c for c in cmd if c.endswith((".cu", ".cpp")))))
        with open(out, "w") as f:
            f.write("x")
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(build.subprocess, "run", run)
    monkeypatch.setattr(build, "nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    for name, path in (("BUILD_DIR", "_build"), ("LIB_PATH", "libdsa_gb300.so"), ("MARSHAL_PATH", "_marshal.so"),
                       ("MARSHAL_STAMP", "_build/_marshal.txt")):
        monkeypatch.setattr(build, name, str(tmp_path / path), raising=False)
    return made


def without_torch(monkeypatch):
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))


def test_the_library_needs_no_torch(place, monkeypatch):
    without_torch(monkeypatch)
    assert build.build() == build.LIB_PATH
    assert sorted(place) == sorted(build.SOURCES + ["link"]) and os.path.exists(build.LIB_PATH)
    place.clear()
    assert build.up_to_date() and build.build() == build.LIB_PATH and place == []


def test_everything_once(place):
    build.build()
    assert sorted(place) == sorted(build.SOURCES + ["link", "marshal.cpp"])
    place.clear()
    build.build()
    assert place == []
    build.build(force=True)
    assert sorted(place) == sorted(build.SOURCES + ["link", "marshal.cpp"])


def test_each_part_for_itself(place):
    build.build()
    place.clear()
    os.remove(build.MARSHAL_PATH)
    build.build()
    assert place == ["marshal.cpp"]
    place.clear()
    os.remove(build.LIB_PATH)
    build.build()
    assert sorted(place) == sorted(build.SOURCES + ["link"])


def test_marshalling_is_built_again_for_another_torch(place):
    build.build()
    place.clear()
    with open(build.MARSHAL_STAMP) as f:
        ours = f.read()
    with open(build.MARSHAL_STAMP, "w") as f:
        f.write(ours.replace("__version__ = '", "__version__ = '1"))
    assert not build.up_to_date()
    build.build()
    assert place == ["marshal.cpp"] and build.up_to_date()
    with open(build.MARSHAL_STAMP) as f:
        assert f.read() == ours


def test_a_marshalling_that_does_not_load_says_how_to_build_it(monkeypatch):
    import sparse_attention_indexer_e4m3_gb300 as dsa

    build.build()
    monkeypatch.setattr(dsa, "_calls", None)

    def load(name, *a):
        raise ImportError("undefined symbol: _ZN3c10")

    monkeypatch.setattr(dsa.importlib, "import_module", load)
    with pytest.raises(RuntimeError, match=r"python -m sparse_attention_indexer_e4m3_gb300\.build"):
        dsa.fork_pages(None, None, None)
