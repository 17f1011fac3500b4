"""The binding's native part is an addition: without it every operator still runs, through Python and the C ABI."""
import os
import shutil
import subprocess
import sys

import pytest

from sliding_window_attention_device_gb300 import build

PKG = os.path.dirname(build.__file__)


@pytest.fixture(scope="module")
def built():
    build.build()


def package_in(folder, leave_out=lambda name: name.startswith("_calls")):
    """The package's Python files and libraries in another folder, some left out."""
    to = folder / os.path.basename(PKG)
    to.mkdir()
    for name in os.listdir(PKG):
        if name.endswith((".py", ".so")) and not leave_out(name):
            (to / name).symlink_to(os.path.join(PKG, name))
    return folder


def python(folder, code):
    head = f"import sys; sys.path.insert(0, {str(folder)!r})\nfrom sliding_window_attention_device_gb300 import bdattn\n"
    env = {k: v for k, v in os.environ.items() if k != "PYTHONPATH"}
    return subprocess.run([sys.executable, "-c", head + code], capture_output=True, text=True, cwd=folder, env=env)


def test_without_the_native_calls(built, tmp_path):
    """A package that holds the library alone loads, answers, and says what is slower."""
    r = python(package_in(tmp_path), f"""
assert bdattn.__file__.startswith({str(tmp_path)!r})
lib = bdattn.load()
assert bdattn._calls is None
pg = bdattn.paged_geom(4, 8, 2, 128, 100, 16, 200)
assert bdattn.paged4_decode_workspace_bytes(pg) > 0 and bdattn.paged_decode_workspace_bytes(pg) > 0
g = bdattn.geom(1, 2, 1, 64, 256, 64, 0, 0, 256)
assert bdattn.seg_bytes(g) > 0
for call in (bdattn.bd_attn_paged4_decode, bdattn.bd_attn_paged_decode):
    try:
        call(*[None] * (6 if "4" in call.__name__ else 7))
    except ValueError as e:
        assert "CUDA tensor" in str(e)
    else:
        raise AssertionError
""")
    assert r.returncode == 0, r.stderr
    assert r.stderr.count("RuntimeWarning") == 1 and "_calls" in r.stderr


def test_with_them(built, tmp_path):
    r = python(package_in(tmp_path, lambda name: False), "bdattn.load()\nassert bdattn._calls is not None")
    assert r.returncode == 0 and "Warning" not in r.stderr, r.stderr


def test_the_module_is_of_one_torch_and_python(built, monkeypatch):
    """It inlines torch's and Python's structs, so another version of either has a module of its own to build."""
    import sysconfig

    import torch
    here = build.calls_path()
    assert os.path.exists(here) and not build.calls_stale()
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "9.9.9+cu990")
        assert build.calls_path() != here and build.calls_stale() and not build.library_stale()
    soabi = sysconfig.get_config_var("SOABI")
    with monkeypatch.context() as m:
        m.setattr(sysconfig, "get_config_var", lambda name: "cpython-399-other" if name == "SOABI" else None)
        assert soabi and build.calls_path() != here and build.calls_stale() and not build.library_stale()
    assert build.calls_path() == here and not build.calls_stale()


def test_a_module_of_another_torch_is_not_loaded(built, tmp_path):
    """All files are there, under another torch: its module is not."""
    r = python(package_in(tmp_path, lambda name: False), """
import torch
torch.__version__ = "9.9.9+cu990"
bdattn.load()
assert bdattn._calls is None
""")
    assert r.returncode == 0 and "RuntimeWarning" in r.stderr, r.stderr


@pytest.mark.parametrize("missing", ["torch", "torch_headers", "Python.h", "g++"])
def test_the_library_is_built_without_what_the_module_needs(built, monkeypatch, capsys, missing):
    """Of the C ABI's library nothing needs torch, Python's headers or g++: it is brought up to date, and the module
    that does is named as left out."""
    import importlib.util
    import sysconfig
    torch_dir = list(importlib.util.find_spec("torch").submodule_search_locations)[0]
    old = os.path.getmtime(build.LIB)
    ran = []

    def run(cmd, what):  # the compiler's and linker's calls, of the library only
        ran.append(what)
        assert "calls" not in what
        if "-shared" in cmd:
            shutil.copy2(build.LIB, cmd[cmd.index("-o") + 1])
        return ""

    monkeypatch.setattr(build, "_run", run)
    isfile, which, find = os.path.isfile, shutil.which, importlib.util.find_spec
    if missing == "torch":
        monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    elif missing == "torch_headers":
        monkeypatch.setattr(os.path, "isfile", lambda p: not str(p).startswith(torch_dir) and isfile(p))
    elif missing == "Python.h":
        inc = sysconfig.get_paths()["include"]
        monkeypatch.setattr(os.path, "isfile", lambda p: not str(p).startswith(inc) and isfile(p))
    else:
        monkeypatch.setattr(shutil, "which", lambda name, *a, **k: None if name == "g++" else which(name, *a, **k))
    assert build.build(force=True) == build.LIB
    assert "link of libbdattn.so" in ran and os.path.getmtime(build.LIB) == old
    assert "_calls is left out" in capsys.readouterr().err


def test_a_module_that_does_not_compile_is_an_error_behind_the_library(built, monkeypatch):
    """Where everything is there but g++ fails, the library is in place before that is raised."""
    ran = []

    def run(cmd, what):
        ran.append(what)
        if "calls" in what:
            raise RuntimeError(f"{what} failed")
        if "-shared" in cmd:
            shutil.copy2(build.LIB, cmd[cmd.index("-o") + 1])
        return ""

    monkeypatch.setattr(build, "_run", run)
    with pytest.raises(RuntimeError, match="calls"):
        build.build(force=True)
    assert "link of libbdattn.so" in ran


@pytest.mark.parametrize("gxx", [True, False])
def test_what_is_up_to_date_needs_no_compiler(built, monkeypatch, capsys, gxx):
    monkeypatch.setattr(build, "_nvcc", lambda: 1 / 0)
    if not gxx:
        monkeypatch.setattr(shutil, "which", lambda *a, **k: None)
    assert build.build() == build.LIB and capsys.readouterr().err == ""
