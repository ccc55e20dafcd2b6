"""What build.py builds, with what is installed (compiler and linker faked)."""
import os
import subprocess
import sys
import threading
import time

import pytest

from paged_kv_cache_108_gb300 import build as b


@pytest.fixture
def made(tmp_path, monkeypatch):
    """Outputs in a folder of their own; compiles and links are recorded."""
    log = []
    monkeypatch.setattr(b, "BUILD", str(tmp_path / "o"))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "libpa.so"))
    monkeypatch.setattr(b, "BINDING", str(tmp_path / "_binding.so"))
    monkeypatch.setattr(b, "BUILT_FOR", str(tmp_path / "_binding.built_for"), raising=False)

    def compile_(src, verbose):
        log.append(("compile", os.path.basename(src)))
        return src + ".o"

    def link(cmd, inputs, out):
        log.append(("link", os.path.basename(out)))
        open(out, "w").close()

    monkeypatch.setattr(b, "_compile", compile_)
    monkeypatch.setattr(b, "_link", link)
    return log


def _without_torch(monkeypatch):
    find = b.importlib.util.find_spec
    monkeypatch.setattr(b.importlib.util, "find_spec", lambda n, *a: None if n == "torch" else find(n, *a))


def test_the_library_is_built_without_torch(made, monkeypatch):
    _without_torch(monkeypatch)
    assert b.build() == b.LIB
    assert ("link", "libpa.so") in made and ("compile", "binding.cpp") not in made
    assert b.up_to_date()
    with pytest.raises(RuntimeError, match="torch not found"):
        b.build_binding()


def test_a_binding_that_does_not_compile_leaves_the_library(made, monkeypatch):
    compile_ = b._compile

    def fails(src, verbose):
        if src == b.BINDING_SRC:
            raise RuntimeError("compile failed: no Python.h")
        return compile_(src, verbose)

    monkeypatch.setattr(b, "_compile", fails)
    with pytest.raises(RuntimeError, match="Python.h"):
        b.build()
    assert os.path.exists(b.LIB) and not os.path.exists(b.BINDING)


def test_each_is_built_when_it_is_stale(made):
    b.build()
    assert made[-1] == ("link", "_binding.so") and ("link", "libpa.so") in made
    made.clear()
    b.build()
    assert not made
    os.remove(b.BINDING)
    b.build()
    assert made == [("compile", "binding.cpp"), ("link", "_binding.so")]
    made.clear()
    os.remove(b.LIB)
    b.build()
    assert ("link", "libpa.so") in made and ("link", "_binding.so") not in made


@pytest.mark.parametrize("what", ["torch", "python", "record"])
def test_a_binding_for_another_torch_or_python_is_built_again(made, monkeypatch, what):
    b.build()
    assert b.binding_up_to_date() and b.binding_fits()
    if what == "torch":
        with open(b.BUILT_FOR) as f:
            old = f.read()
        with open(b.BUILT_FOR, "w") as f:
            f.write(old.replace("torch ", "torch 1."))
    elif what == "python":
        monkeypatch.setattr(b.sysconfig, "get_config_var", lambda n: "cpython-399")
    else:
        os.remove(b.BUILT_FOR)
    assert not b.binding_fits() and not b.up_to_date()
    made.clear()
    b.build()
    assert made == [("compile", "binding.cpp"), ("link", "_binding.so")]
    assert b.binding_fits() and b.up_to_date()


def test_the_record_names_the_torch_that_is_imported():
    import torch

    assert f"torch {torch.__version__} " in b._built_for()


def test_the_loader_builds_a_binding_that_does_not_fit(monkeypatch):
    from paged_kv_cache_108_gb300 import _lib

    built = []
    monkeypatch.setattr(_lib, "_binding", None)
    monkeypatch.setattr(b, "binding_fits", lambda: bool(built))
    for f in ("build", "build_binding"):
        monkeypatch.setattr(b, f, lambda *a, **k: built.append(1))
    assert _lib.binding().__name__.endswith("_binding") and built == [1]


def _in_threads(n, f):
    got = []
    threads = [threading.Thread(target=lambda: got.append(f())) for _ in range(n)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    return got


def test_threads_whose_first_call_finds_no_binding_build_it_once(monkeypatch):
    from paged_kv_cache_108_gb300 import _lib

    built = []

    def build_binding():
        time.sleep(0.05)
        built.append("binding")

    monkeypatch.setattr(_lib, "_binding", None)
    monkeypatch.setattr(b, "binding_fits", lambda: bool(built))
    monkeypatch.setattr(b, "build_binding", build_binding)
    # the library, which is loaded, is not linked anew
    for f in ("build", "build_library"):
        monkeypatch.setattr(b, f, lambda *a, **k: built.append("library"))
    got = _in_threads(8, _lib.binding)
    assert len(set(got)) == 1 and len(got) == 8 and built == ["binding"]


@pytest.mark.parametrize("what", ["build", "build_binding"])
def test_builds_at_the_same_time_run_one_after_another(made, monkeypatch, what):
    if what == "build_binding":
        b.build_library()
        made.clear()
    compile_, running, most = b._compile, [], []

    def slow(src, verbose):
        if src == b.BINDING_SRC:
            running.append(1)
            most.append(len(running))
            time.sleep(0.02)
            running.pop()
        return compile_(src, verbose)

    monkeypatch.setattr(b, "_compile", slow)
    _in_threads(4, getattr(b, what))
    assert most == [1] and made.count(("link", "_binding.so")) == 1
    assert made.count(("link", "libpa.so")) == (what == "build")


def test_the_binding_and_the_loader_share_one_library():
    # what the binding's call fails with is what the loader reads
    from paged_kv_cache_108_gb300 import _lib

    code = """
from paged_kv_cache_108_gb300 import _lib
_lib.lib(), _lib.binding()
with open("/proc/self/maps") as f:
    print(sorted({l.split()[-1] for l in f if "libpa.so" in l}))
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=120,
                       cwd=b.ROOT)
    assert r.stdout.strip() == str([_lib.LIB_PATH]), r.stderr[-500:]


def test_nothing_is_written_where_nothing_is_stale(made, monkeypatch):
    b.build()
    made.clear()
    monkeypatch.setattr(b, "_alone", None)  # a tree that cannot be written to
    assert b.build() == b.LIB and b.build_library() == b.LIB and not made
