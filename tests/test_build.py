"""The build, with compilers that only write their output: the library does
not depend on torch or on the Python module, and the module is made again when
torch changes."""
import os
import stat

import pytest
import torch

from rope_chain_gb300 import _build

COMPILER = """#!/bin/sh
echo "$0 $*" >> {log}
test {fails} = 0 || exit 1
while [ $# -gt 0 ]; do
    if [ "$1" = -o ]; then shift; echo made > "$1"; fi
    shift
done
"""


@pytest.fixture
def box(tmp_path, monkeypatch):
    class Box:
        def compiler(self, name, fails=0):
            path = tmp_path / name
            path.write_text(COMPILER.format(log=tmp_path / f"{name}.log", fails=fails))
            path.chmod(path.stat().st_mode | stat.S_IXUSR)
            return str(path)

        def ran(self, name):
            log = tmp_path / f"{name}.log"
            return len(log.read_text().splitlines()) if log.exists() else 0

        def cxx(self, fails=0):
            path = self.compiler("g++", fails)
            monkeypatch.setattr(_build.shutil, "which", lambda name: path if name == "g++" else None)

    b = Box()
    monkeypatch.setenv("NVCC", b.compiler("nvcc"))
    for name, at in (("BUILD", "build"), ("LIB", "librope_chain.so"), ("MODULE", "_draft.so"), ("MODULE_STAMP", "build/module.txt")):
        monkeypatch.setattr(_build, name, str(tmp_path / at), raising=False)
    b.cxx()
    return b


def test_library_is_built_where_the_module_cannot_be(box, monkeypatch):
    box.cxx(fails=1)
    with pytest.raises(RuntimeError):
        _build.build()
    assert os.path.exists(_build.LIB) and not os.path.exists(_build.MODULE)
    os.remove(_build.LIB)

    def no_torch():
        raise ImportError("no torch")
    monkeypatch.setattr(_build, "_torch_flags", no_torch)
    with pytest.raises(ImportError):
        _build.build()
    assert os.path.exists(_build.LIB)


def test_module_is_made_again_for_another_torch(box, monkeypatch):
    _build.build()
    assert os.path.exists(_build.LIB) and os.path.exists(_build.MODULE)
    library, module = box.ran("nvcc"), box.ran("g++")
    _build.build()
    assert (box.ran("nvcc"), box.ran("g++")) == (library, module)
    monkeypatch.setattr(torch, "__version__", "9.9.9")
    _build.build()
    assert box.ran("nvcc") == library and box.ran("g++") == 2 * module
