"""Objects are reused only when they are what their sidecar file says (CPU, no compiler)."""
import os

import pytest

from gated_delta_rule_recurrent_b200 import build


@pytest.fixture
def units(tmp_path, monkeypatch):
    """A library of one source whose "compiler" writes the source into the object."""
    source = tmp_path / "unit.cu"
    source.write_text("first")
    lib = str(tmp_path / "lib.so")
    monkeypatch.setattr(build, "UNITS", {str(source): [str(source)]})
    monkeypatch.setattr(build, "DEPS", [str(source)])
    monkeypatch.setattr(build, "OBJ_DIR", str(tmp_path / "objects"))
    monkeypatch.setattr(build, "LIB_PATH", lib)
    state = dict(source=source, lib=lib, compiled=0, stop="")

    def run(cmd, verbose):
        with open(cmd[cmd.index("-o") + 1], "w") as out:
            if "-c" in cmd:
                out.write(source.read_text())
                state["compiled"] += 1
            else:
                out.write("".join(open(obj).read() for obj in cmd if obj.endswith(".o")))
        if state["stop"] == ("compile" if "-c" in cmd else "link"):
            raise KeyboardInterrupt

    monkeypatch.setattr(build, "_run", run)
    monkeypatch.setattr(build, "nvcc_path", lambda: "nvcc")
    return state


def test_an_unchanged_object_is_reused_and_a_changed_one_is_not(units):
    build.build(reuse=True)
    build.build(reuse=True)
    assert units["compiled"] == 1
    units["source"].write_text("second")
    build.build(reuse=True)
    assert units["compiled"] == 2 and open(units["lib"]).read() == "second"


def test_an_interrupted_compilation_leaves_no_object_to_reuse(units):
    """The object is the second source's, written just before the interruption; the sources
    then go back to the first."""
    build.build(reuse=True)
    units["source"].write_text("second")
    units["stop"] = "compile"
    with pytest.raises(KeyboardInterrupt):
        build.build(reuse=True)
    units["stop"] = ""
    units["source"].write_text("first")
    build.build(reuse=True)
    assert open(units["lib"]).read() == "first"
    assert os.path.exists(units["lib"] + ".srchash")


def test_an_interrupted_link_leaves_no_current_library(units):
    build.build()
    assert build.is_current()
    units["source"].write_text("second")
    units["stop"] = "link"
    with pytest.raises(KeyboardInterrupt):
        build.build()
    units["stop"] = ""
    units["source"].write_text("first")
    assert not build.is_current()
    build.ensure_built()
    assert open(units["lib"]).read() == "first"
