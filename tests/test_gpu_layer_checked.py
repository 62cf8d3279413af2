"""The decoder layer's other operators in the bounds-checked build: their
suites run against it in a child process, and each test reads the device
error word after its calls, so that one access outside its buffer fails it."""
import subprocess
import sys

import pytest

from bit_weight_only_g128_gb300 import build as wbuild
from test_gpu_checked import ROOT, _child_env

pytestmark = pytest.mark.gpu

SUITES = ["tests/test_gpu_layer.py", "tests/test_gpu_layer_edges.py", "tests/test_gpu_layer_nonfinite.py",
          "tests/test_gpu_layer_workspace.py", "tests/test_gpu_run_layer_limits.py"]


def test_layer_suites_pass_in_the_checked_build():
    lib = wbuild.build(checked=True)
    res = subprocess.run([sys.executable, "-m", "pytest", *SUITES, "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider"],
                         cwd=ROOT, env=_child_env(lib), capture_output=True, text=True, timeout=1800)
    tail = "\n".join((res.stdout + res.stderr).splitlines()[-30:])
    assert res.returncode == 0, tail
    assert " passed" in tail and " failed" not in tail, tail
