"""What build() makes in which order, with the compilers replaced: the C libraries need nothing of PyTorch."""
import os

import pytest

from moe_expert_layer_top_gb300 import build


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """An empty build tree; the commands that were run, in order."""
    home = tmp_path / "torch"
    home.mkdir()
    (home / "version.py").write_text("__version__ = '1'\n")
    for name in ("LIB_DIR", "DEBUG_DIR", "SYNTH_LIB_DIR"):
        monkeypatch.setattr(build, name, str(tmp_path / name))
    for name in ("LIB_PATH", "DEBUG_LIB_PATH", "SYNTH_LIB_PATH", "TORCH_LIB_PATH", "TORCH_STAMP_PATH"):
        monkeypatch.setattr(build, name, str(tmp_path / "LIB_DIR" / name))
    ran = []

    def run(cmd):
        out = cmd[cmd.index("-o") + 1]
        ran.append(os.path.basename(out))
        open(out, "w").close()
        return ""

    monkeypatch.setattr(build, "_run", run)
    monkeypatch.setattr(build, "nvcc", lambda: "/nvcc/bin/nvcc")
    monkeypatch.setattr(build, "_torch_home", lambda: str(home))
    return home, ran


def test_libraries_without_pytorch(tree, monkeypatch):
    home, ran = tree
    monkeypatch.setattr(build, "_torch_home", lambda: None)
    assert build.build() == build.LIB_PATH
    assert all(os.path.exists(p) for p in (build.LIB_PATH, build.DEBUG_LIB_PATH, build.SYNTH_LIB_PATH))
    assert not os.path.exists(build.TORCH_LIB_PATH)


def test_libraries_when_the_module_does_not_compile(tree, monkeypatch):
    home, ran = tree
    run = build._run

    def no_headers(cmd):
        if "-ltorch_python" in cmd:
            raise RuntimeError("Python.h: no such file")
        return run(cmd)

    monkeypatch.setattr(build, "_run", no_headers)
    with pytest.raises(RuntimeError, match="Python.h"):
        build.build()
    assert all(os.path.exists(p) for p in (build.LIB_PATH, build.DEBUG_LIB_PATH, build.SYNTH_LIB_PATH))


def test_module_follows_the_installed_pytorch(tree):
    home, ran = tree
    build.build()
    assert os.path.exists(build.TORCH_LIB_PATH)
    ran.clear()
    build.build()
    assert ran == []  # nothing to do
    (home / "version.py").write_text("__version__ = '2'\n")
    build.build()
    assert ran == ["TORCH_LIB_PATH.tmp"]
    os.remove(build.TORCH_STAMP_PATH)
    ran.clear()
    build.build()
    assert ran == ["TORCH_LIB_PATH.tmp"]


def test_pytorch_is_found_without_importing_it():
    import torch
    assert build._torch_home() == os.path.dirname(torch.__file__)
    assert torch.__version__.split("+")[0] in build._torch_stamp(build._torch_home())
