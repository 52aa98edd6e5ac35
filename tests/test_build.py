"""What a build needs and leaves, with the compilers stood in for: the library is made by hipcc
alone, the compiled binding where torch and g++ are at hand."""
import os

import pytest

from log_prob_amd import build as b


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """Outputs under tmp_path; every command is recorded and leaves its output file."""
    runs = []

    def run(cmd, check):
        assert check
        runs.append(cmd)
        if "broken" in tree_.state and any(tree_.state["broken"] in c for c in cmd):
            raise b.subprocess.CalledProcessError(1, cmd)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("new")

    class Tree:
        state = {}
        lib, binding = str(tmp_path / "libflce.so"), str(tmp_path / "_binding.so")

        def make(self):
            return b.build(out=self.lib)

        def left(self):
            return {f: open(tmp_path / f).read() for f in os.listdir(tmp_path)}

    tree_ = Tree()
    tree_.runs = runs
    monkeypatch.setattr(b, "LIB", tree_.lib)
    monkeypatch.setattr(b, "BINDING", tree_.binding)
    monkeypatch.setattr(b, "hipcc", lambda: "/opt/rocm/bin/hipcc")
    monkeypatch.setattr(b.subprocess, "run", run)
    for f in (tree_.lib, tree_.binding):
        with open(f, "w") as h:
            h.write("old")
    return tree_


def test_both(tree):
    assert tree.make() == tree.lib
    assert tree.left() == {"libflce.so": "new", "_binding.so": "new"}
    assert [c[0] for c in tree.runs].count("g++") == 2


@pytest.mark.parametrize("missing", ["torch", "g++"])
def test_library_without_torch_or_a_host_compiler(tree, monkeypatch, missing):
    """The binding that was there fitted another library: it goes."""
    if missing == "torch":
        monkeypatch.setattr(b.importlib.util, "find_spec", lambda name: None)
    else:
        which = b.shutil.which
        monkeypatch.setattr(b.shutil, "which", lambda name: None if name == "g++" else which(name))
    assert tree.make() == tree.lib
    assert tree.left() == {"libflce.so": "new"}
    assert all(c[0] == "/opt/rocm/bin/hipcc" for c in tree.runs)


@pytest.mark.parametrize("broken", ["ops_api.cpp", "binding.cpp", "-ltorch_python"])
def test_a_failed_build_leaves_what_was_there(tree, broken):
    tree.state = {"broken": broken}
    with pytest.raises(b.subprocess.CalledProcessError):
        tree.make()
    assert {f: v for f, v in tree.left().items() if not f.endswith(".tmp")} == {
        "libflce.so": "old", "_binding.so": "old"}


def test_another_library_leaves_the_binding_alone(tree, tmp_path):
    out = str(tmp_path / "other.so")
    assert b.build(out=out) == out
    assert tree.left() == {"libflce.so": "old", "_binding.so": "old", "other.so": "new"}
