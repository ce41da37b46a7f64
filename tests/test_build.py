"""The build's own logic, with stand-ins for the compilers in a folder of its own:
what is made again after a change, a failure, or under another torch."""
import importlib.util
import os
import time

import pytest
import torch

from memory_bound_transformer_gb300 import build as b

# writes what it was given to the file behind -o, fails while a file named like it lies beside the log
TOOL = """#!/bin/sh
echo "{name} $*" >> {log}
case "$*" in *" -c "*) step=compile;; *) step=link;; esac
test ! -e {fail}-{name}-$step || exit 1
out=; for a in "$@"; do test "$last" = -o && out=$a; last=$a; done
echo "{name} $*" > "$out"
for a in "$@"; do case "$a" in *.cu|*.cpp|*.o) test "$a" = "$out" || cat "$a" >> "$out";; esac; done
"""


class Tree:
    def __init__(self, root, monkeypatch):
        self.root, self.log, self.now = root, root / "log", time.time() - 10000
        pkg, tools = root / "pkg", root / "bin"
        for d in (pkg / "csrc", root / "include", tools):
            d.mkdir(parents=True)
        for name in ("nvcc", "g++"):
            (tools / name).write_text(TOOL.format(name=name, log=self.log, fail=root / "fail"))
            (tools / name).chmod(0o755)
        for f in ("a.cu", "b.cu", "binding.cpp", "common.cuh"):
            (pkg / "csrc" / f).write_text(f + " 1\n")
        (root / "include" / "ops.h").write_text("1\n")
        for k, v in dict(PKG=pkg, CSRC=pkg / "csrc", OBJ=pkg / "_build", LIB=pkg / "lib.so", BINDING=pkg / "ext.so").items():
            monkeypatch.setattr(b, k, str(v))
        monkeypatch.setattr(b, "SOURCES", ["a.cu", "b.cu"])
        monkeypatch.setenv("NVCC", str(tools / "nvcc"))
        monkeypatch.setenv("PATH", f"{tools}:{os.environ['PATH']}")
        self.lib, self.ext = pkg / "lib.so", pkg / "ext.so"

    def age(self):
        """Sources and what was made of them, in order, lie in the past."""
        made = sorted((self.root / "pkg" / "_build").iterdir()) + [self.lib, self.ext]
        for f in self.root.rglob("*"):
            if f.is_file() and f not in made:
                os.utime(f, (self.now, self.now))
        for i, f in enumerate(made):
            os.utime(f, (self.now + 100 + i, self.now + 100 + i))

    def change(self, *path):
        self.root.joinpath(*path).write_text("changed\n")

    def build(self):
        """The commands that one call of build() ran."""
        self.log.write_text("")
        b.build()
        return self.log.read_text().splitlines()

    def fails(self, tool, step):
        f = self.root / f"fail-{tool}-{step}"
        f.write_text("")
        self.log.write_text("")
        with pytest.raises(RuntimeError):
            b.build()
        f.unlink()


@pytest.fixture
def tree(tmp_path, monkeypatch):
    t = Tree(tmp_path, monkeypatch)
    assert len(t.build()) == 5 and t.lib.exists() and t.ext.exists()
    t.age()
    assert t.build() == []
    return t


def test_a_source(tree):
    tree.change("pkg", "csrc", "a.cu")
    got = tree.build()
    assert sum("a.cu" in c for c in got) == 1 and not any("b.cu" in c for c in got)
    assert any("lib.so" in c and "-shared" in c for c in got) and tree.ext.stat().st_mtime >= tree.lib.stat().st_mtime


@pytest.mark.parametrize("step", ["compile", "link"])
def test_a_header_while_the_library_fails(tree, step):
    """The extension is never left with the signatures of another library than the one beside it."""
    tree.change("include", "ops.h")
    tree.fails("nvcc", step)
    assert not tree.ext.exists()
    tree.build()
    assert tree.lib.exists() and tree.ext.exists()


@pytest.mark.parametrize("step", ["compile", "link"])
def test_the_extension_fails(tree, step):
    tree.change("pkg", "csrc", "binding.cpp")
    tree.fails("g++", step)
    assert tree.lib.exists() and not tree.ext.exists()
    tree.build()
    assert "changed" in tree.ext.read_text()


def test_another_torch(tree, monkeypatch):
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    got = tree.build()
    assert len(got) == 2 and all(c.startswith("g++") for c in got)
    assert tree.build() == []


def test_nothing_half_linked(tree):
    """A link that fails leaves no part behind."""
    tree.change("pkg", "csrc", "a.cu")
    tree.fails("nvcc", "link")
    assert sorted(f.name for f in (tree.root / "pkg").iterdir()) == ["_build", "csrc"]


def test_the_library_needs_nvcc_alone(tree, monkeypatch):
    """Without torch it is made, and no extension stays beside it."""
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    tree.change("include", "ops.h")
    got = tree.build()
    assert got and all(c.startswith("nvcc") for c in got) and tree.lib.exists() and not tree.ext.exists()


def test_the_library_asked_for_alone(tree):
    tree.change("pkg", "csrc", "common.cuh")
    tree.log.write_text("")
    b.build(library_only=True)
    assert all(c.startswith("nvcc") for c in tree.log.read_text().splitlines()) and tree.lib.exists() and not tree.ext.exists()
    assert all(c.startswith("g++") for c in tree.build()) and tree.ext.exists()


def test_a_broken_extension_leaves_the_library(tree):
    tree.lib.unlink(), tree.ext.unlink()
    tree.change("pkg", "csrc", "binding.cpp")
    tree.fails("g++", "compile")
    assert tree.lib.exists() and not tree.ext.exists()
