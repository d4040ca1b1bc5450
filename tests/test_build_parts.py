"""The library and its torch binding are built apart: what keeps the binding from
being built does not keep a program from the C ABI, and a binding of another
torch is not loaded.  The compilers here are stand-ins."""
import json
import os
import subprocess
import sys
import types

import pytest

from exact_tiled_attention_23_gb300 import _build


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """An empty lib/, and compilers that write their output file."""
    for name, path in (("LIB_DIR", tmp_path / "lib"), ("BUILD_DIR", tmp_path / "obj"), ("LIB_PATH", tmp_path / "lib" / "libfa.so"),
                       ("BINDING_PATH", tmp_path / "lib" / "fa_torch.so"), ("BINDING_STAMP", tmp_path / "lib" / "fa_torch.json")):
        monkeypatch.setattr(_build, name, str(path))
    monkeypatch.setattr(_build, "nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    state = types.SimpleNamespace(ran=[], gcc_fails=False, target=["9.9", "13.0", "abi"])
    monkeypatch.setattr(_build, "binding_target", lambda: state.target)
    fake = types.ModuleType("torch")
    fake._C = types.SimpleNamespace(_GLIBCXX_USE_CXX11_ABI=True)
    fake.__file__ = str(tmp_path / "torch" / "__init__.py")
    monkeypatch.setitem(sys.modules, "torch", fake)

    def run(cmd, **kw):
        state.ran.append(os.path.basename(cmd[0]))
        fails = cmd[0] == "g++" and state.gcc_fails
        if not fails:
            with open(cmd[cmd.index("-o") + 1], "w") as f:
                f.write("built")
        return subprocess.CompletedProcess(cmd, int(fails), "", "no headers" if fails else "")
    monkeypatch.setattr(_build.subprocess, "run", run)
    return state


def test_both_are_built_once(tree):
    assert _build.build() == _build.LIB_PATH and _build.up_to_date()
    assert os.path.exists(_build.BINDING_PATH) and tree.ran.count("g++") == 1
    done = len(tree.ran)
    _build.build()
    assert len(tree.ran) == done


def test_a_binding_that_fails_leaves_the_library(tree):
    tree.gcc_fails = True
    with pytest.warns(RuntimeWarning, match="no headers"):
        assert _build.build() == _build.LIB_PATH
    assert os.path.exists(_build.LIB_PATH) and _build.library_up_to_date()
    assert not os.path.exists(_build.BINDING_PATH) and not _build.up_to_date()
    # the next call tries the binding again, and the library not
    tree.gcc_fails, tree.ran = False, []
    _build.build()
    assert tree.ran == ["g++"] and _build.up_to_date()


def test_a_torch_that_does_not_import_leaves_the_library(tree, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)
    with pytest.warns(RuntimeWarning, match="torch"):
        _build.build()
    assert os.path.exists(_build.LIB_PATH) and not os.path.exists(_build.BINDING_PATH)


def test_no_torch_for_cuda_is_no_binding(tree):
    tree.target = None
    _build.build()
    assert _build.up_to_date() and "g++" not in tree.ran


def test_another_torch_builds_the_binding_again(tree):
    _build.build()
    tree.target = ["10.0"] + tree.target[1:]
    assert _build.library_up_to_date() and not _build.binding_up_to_date()
    tree.ran = []
    _build.build()
    assert tree.ran == ["g++"] and _build.up_to_date()
    with open(_build.BINDING_STAMP, "w") as f:
        f.write("{")
    assert not _build.binding_up_to_date()


def test_what_a_binding_is_built_for(tmp_path, monkeypatch):
    """torch's own version file, read without importing torch."""
    (tmp_path / "torch").mkdir()
    (tmp_path / "torch" / "__init__.py").write_text("raise ImportError('broken')\n")
    version = tmp_path / "torch" / "version.py"
    version.write_text("__version__ = '1.2+cu999'\ncuda = '99.9'\n")
    code = "import json; from exact_tiled_attention_23_gb300 import _build; print(json.dumps(_build.binding_target()))"
    root = os.path.dirname(_build.PKG)

    def target():
        env = dict(os.environ, PYTHONPATH=f"{tmp_path}:{root}")
        return json.loads(subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, env=env, check=True,
                                         cwd=tmp_path).stdout)
    got = target()
    assert got[:2] == ["1.2+cu999", "99.9"] and "cpython" in got[2]
    version.write_text("__version__ = '1.2'\ncuda = None\n")
    assert target() is None


def test_a_binding_of_another_torch_is_not_loaded(monkeypatch):
    import exact_tiled_attention_23_gb300 as fa
    fa.build()
    monkeypatch.setattr(fa, "_BINDING", None)
    monkeypatch.setattr(_build, "binding_target", lambda: ["0.0", "0.0", "abi"])
    with pytest.raises(RuntimeError, match="was built for"):
        fa._binding()


def test_a_copied_tree_is_loaded_whatever_its_files_dates(tmp_path):
    """A copy that dates the built files before the sources still runs."""
    import shutil

    import exact_tiled_attention_23_gb300 as fa
    fa.build()
    copy = tmp_path / "exact_tiled_attention_23_gb300"
    shutil.copytree(_build.PKG, copy, ignore=shutil.ignore_patterns("_build", "__pycache__"))
    shutil.copytree(_build.INCLUDE, tmp_path / "include")
    for f in (copy / "lib").iterdir():
        os.utime(f, (1, 1))
    code = "import exact_tiled_attention_23_gb300 as fa; print(fa.__file__); fa._binding()"
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=tmp_path,
                       env=dict(os.environ, PYTHONPATH=str(tmp_path)))
    assert r.returncode == 0 and str(copy) in r.stdout, r.stderr[-2000:]
