"""What the build makes where parts of the toolchain are missing: the C library needs nvcc alone. Compilers are scripts
that write their output files, so that nothing is compiled here."""
import os
import stat
import sys
import sysconfig

import pytest

from vision_transformer_encoder_gb300 import api, build


def script(path, body):
    path.write_text("#!/bin/sh\n" + body)
    path.chmod(path.stat().st_mode | stat.S_IXUSR)
    return str(path)


WRITE_OUTPUT = 'echo "$@" >> "$0.calls"\nwhile [ $# -gt 0 ]; do [ "$1" = -o ] && : > "$2"; shift; done\n'


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A tree with two kernels and a binding, an nvcc and a g++."""
    csrc = tmp_path / "csrc"
    csrc.mkdir()
    for name in ("a.cu", "b.cu", "binding.cpp"):
        (csrc / name).write_text("")
    monkeypatch.setattr(build, "HERE", str(tmp_path))
    monkeypatch.setattr(build, "CSRC", str(csrc))
    monkeypatch.setattr(build, "BUILD_DIR", str(tmp_path / "_build"))
    monkeypatch.setattr(build, "LIB_PATH", str(tmp_path / "libvit_block.so"))
    monkeypatch.setattr(build, "BINDING_SRC", str(csrc / "binding.cpp"))
    monkeypatch.setenv("NVCC", script(tmp_path / "nvcc", WRITE_OUTPUT))
    monkeypatch.setenv("CXX", script(tmp_path / "cxx", WRITE_OUTPUT))
    return tmp_path


def calls(tree, tool):
    p = tree / (tool + ".calls")
    return p.read_text().splitlines() if p.exists() else []


def bindings(tree):
    return [p.name for p in tree.glob("_serving*") if not p.name.endswith(".tmp")]


def test_both_are_built_once(tree):
    assert build.build() == build.LIB_PATH and os.path.exists(build.LIB_PATH)
    assert len(calls(tree, "nvcc")) == 3 and len(calls(tree, "cxx")) == 1 and len(bindings(tree)) == 1
    assert build.up_to_date()
    build.build()
    assert len(calls(tree, "nvcc")) == 3 and len(calls(tree, "cxx")) == 1
    assert not list(tree.glob("*.tmp"))


@pytest.mark.parametrize("missing", ["torch", "headers", "compiler"])
def test_without_the_bindings_needs_the_library_is_built(tree, monkeypatch, capsys, missing):
    if missing == "torch":
        monkeypatch.setitem(sys.modules, "torch", None)
    elif missing == "headers":   # a torch without CUDA's parts
        (tree / "site" / "torch" / "include").mkdir(parents=True)
        (tree / "site" / "torch" / "__init__.py").write_text("")
        monkeypatch.delitem(sys.modules, "torch", raising=False)
        monkeypatch.syspath_prepend(str(tree / "site"))
    else:
        monkeypatch.setenv("CXX", str(tree / "no such compiler"))
    assert build.build() == build.LIB_PATH and os.path.exists(build.LIB_PATH)
    assert not bindings(tree) and not calls(tree, "cxx")
    notice = capsys.readouterr().err
    assert notice.count("\n") == 1 and "left out" in notice
    # and there is nothing left to do
    assert build.up_to_date()
    build.build()
    assert len(calls(tree, "nvcc")) == 3


def test_a_binding_that_does_not_compile_is_an_error_and_leaves_the_library(tree, monkeypatch):
    monkeypatch.setenv("CXX", script(tree / "cxx", "echo no >&2; exit 1\n"))
    with pytest.raises(RuntimeError, match="binding.cpp"):
        build.build()
    assert os.path.exists(build.LIB_PATH) and not bindings(tree) and not build.up_to_date()


def fake_torch(site, version, git):
    torch = site / "torch"
    for part in ("include/torch/csrc/Dtype.h", "include/c10/cuda/CUDAGuard.h", "lib/libtorch_cuda.so", "__init__.py"):
        (torch / part).parent.mkdir(parents=True, exist_ok=True)
        (torch / part).write_text("")
    (torch / "version.py").write_text("from typing import Optional\n__version__ = '%s'\ncuda: Optional[str] = '13.0'\n"
                                      "git_version = '%s'\n" % (version, git))


def test_another_torch_gets_a_binding_of_its_own(tree, monkeypatch):
    monkeypatch.delitem(sys.modules, "torch", raising=False)
    monkeypatch.syspath_prepend(str(tree / "site"))
    made = []
    for i, (version, git) in enumerate((("2.9.1+cu130", "5811a8d"), ("2.11.0+cu130", "5811a8d"), ("2.11.0+cu130", "70d99e9"))):
        fake_torch(tree / "site", version, git)
        assert not build.up_to_date() and not os.path.exists(build.binding_path())
        build.build()
        made.append(build.binding_path())
        assert build.up_to_date() and os.path.exists(made[-1])
        assert len(calls(tree, "cxx")) == i + 1 and len(calls(tree, "nvcc")) == 3   # the library is not made again
    assert len(set(made)) == 3 and all(m.endswith(sysconfig.get_config_var("EXT_SUFFIX")) for m in made)
    # and back: what was built for it is still good
    fake_torch(tree / "site", "2.9.1+cu130", "5811a8d")
    assert build.up_to_date() and build.binding_path() == made[0]


def test_an_untagged_binding_is_not_taken(tree, monkeypatch):
    """A module without a tag in its name, as an earlier build left it, is neither up to date nor loaded."""
    (tree / "_serving.so").write_text("")
    assert not build.up_to_date()
    build.build()
    assert len(calls(tree, "cxx")) == 1
    monkeypatch.setattr(api, "_native", None)
    monkeypatch.setattr(api, "load_library", lambda: None)
    os.remove(build.binding_path())
    with pytest.raises(RuntimeError, match="is not built; run python -m vision_transformer_encoder_gb300.build$"):
        api.quantize(None)
    with open(build.binding_path(), "w"):   # no ELF file
        pass
    with pytest.raises(RuntimeError, match="cannot be loaded .*--force$"):
        api.quantize(None)
