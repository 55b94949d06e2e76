"""The build of the C library does not depend on the Python module over it."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# builds one source into a folder of its own, beside a module of an earlier build
SCRIPT = r"""
import importlib.util, os, sys
build_py, out, case = sys.argv[1:]
if case == "no torch":
    sys.modules["torch"] = None
spec = importlib.util.spec_from_file_location("_build", build_py)
b = importlib.util.module_from_spec(spec)
spec.loader.exec_module(b)
b.OUT_DIR, b.SOURCES = out, ["flce_ops.cu"]
b.LIB, b.MODULE = os.path.join(out, "libflce.so"), os.path.join(out, "_flce_torch.so")
open(b.MODULE, "w").close()
if case == "broken module":
    def compile_module(obj):
        raise RuntimeError("no module today")
    b._compile_module = compile_module
try:
    assert b.build() == b.LIB
except RuntimeError as e:
    print("raised", e)
print("library", os.path.getsize(b.LIB) > 0, "module", os.path.exists(b.MODULE))
"""


@pytest.mark.parametrize("case", ["no torch", "broken module"])
def test_the_library_is_linked_without_the_module(case, tmp_path):
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("no nvcc")
    r = subprocess.run([sys.executable, "-c", SCRIPT,
                        os.path.join(ROOT, "lm_head_linear_flce_gb300", "_build.py"),
                        str(tmp_path), case], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    assert r.stdout.splitlines()[-1] == "library True module False"  # nor the earlier one
    if case == "no torch":
        assert "without the Python module" in r.stderr and "raised" not in r.stdout
    else:  # a module that should be there and is not is an error
        assert "raised no module today" in r.stdout
