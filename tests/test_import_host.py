"""The package without torch (not gpu): everything but the products loads, as the C ABI's
binding needs torch only when a call is made."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def run(code):
    return subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)


def test_star_import_without_torch():
    r = run("import sys; sys.modules['torch'] = None\n"
            "from exl3_trellis_weight_gb300 import *\n"
            "assert callable(quantize) and callable(rotate) and 'linear' not in globals()")
    assert r.returncode == 0, r.stderr


def test_star_import_with_torch():
    r = run("from exl3_trellis_weight_gb300 import *\n"
            "assert callable(linear) and callable(linear_backward) and callable(expert_linear) and callable(quantize)\n"
            "assert callable(linear_workspace_bytes)")
    assert r.returncode == 0, r.stderr


def test_import_leaves_torch_alone():
    r = run("import sys, exl3_trellis_weight_gb300\nassert 'torch' not in sys.modules")
    assert r.returncode == 0, r.stderr
