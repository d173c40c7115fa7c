"""The native packing of the per-layer calls (csrc/bind.cpp) is an addition: without it, or with a torch it was not built for, the
package builds, imports and works."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def run(code):
    return subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)


def test_import_with_a_torch_without_cuda():
    r = run("import torch; del torch._C._cuda_getCurrentRawStream\n"
            "from agent_kv_cache_lse_b200 import kvc; print(kvc.lib().kvc_version())")
    assert r.returncode == 0 and r.stdout.strip() == "1", r.stderr


@pytest.mark.skipif(not os.path.exists(os.path.join(ROOT, "agent_kv_cache_lse_b200", "_bind.so")), reason="_bind.so is not built")
def test_the_native_module_is_refused_by_another_torch():
    code = "import torch\n%sfrom agent_kv_cache_lse_b200 import kvc; print(kvc._bind is None, kvc.lib().kvc_version())"
    r = run(code % "")
    assert r.returncode == 0 and r.stdout.split() == ["False", "1"], r.stderr
    r = run(code % "torch.__version__ = '1.0.0'; ")
    assert r.returncode == 0 and r.stdout.split() == ["True", "1"], r.stderr


def test_the_build_looks_at_the_torch_it_was_made_for(monkeypatch, tmp_path):
    import torch

    from agent_kv_cache_lse_b200 import build
    for name in ("LIB", "BIND", "BIND_FOR"):
        path = tmp_path / name
        path.write_text(build._bind_target())
        os.utime(path, (4e9, 4e9))
        monkeypatch.setattr(build, name, str(path))
    assert build.up_to_date()
    monkeypatch.setattr(torch, "__version__", "1.0.0")
    assert not build.up_to_date()


@pytest.mark.parametrize("cxx", ["/nonexistent/g++", "false"])
def test_the_library_builds_without_a_host_compiler_for_the_native_module(monkeypatch, tmp_path, capfd, cxx):
    from agent_kv_cache_lse_b200 import build
    lib = tmp_path / "libkvc.so"
    lib.write_text("")
    os.utime(lib, (4e9, 4e9))
    (tmp_path / "_bind.so").write_text("older")
    for name, path in (("LIB", lib), ("BIND", tmp_path / "_bind.so"), ("BIND_FOR", tmp_path / "bind_for.txt")):
        monkeypatch.setattr(build, name, str(path))
    monkeypatch.setenv("CXX", cxx)
    assert build.build() == str(lib)
    assert "_bind.so was not built" in capfd.readouterr().err and not (tmp_path / "_bind.so").exists()
