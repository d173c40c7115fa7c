"""The native packing of the per-layer calls (csrc/bind.cpp) is an addition: without it, or with a torch it was not built for, the
package builds, imports and works."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def run(code):
    return subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)


def test_import_with_a_torch_without_cuda():
    r = run("import torch; del torch._C._cuda_getCurrentRawStream\n"
            "from agent_kv_cache_lse_b200 import kvc; print(kvc.lib().kvc_version())")
    assert r.returncode == 0 and r.stdout.strip() == "1", r.stderr
