"""The bounds, the ends of the types' ranges, unusual routings and graphs of the
products grouped by expert in the bounds-checked build (as
test_gpu_experts_checked.py)."""
import subprocess
import sys

import pytest

from bit_weight_only_g128_gb300 import build as wbuild
from test_gpu_checked import ROOT, _child_env

pytestmark = pytest.mark.gpu

SUITES = ["tests/test_gpu_experts_bounds.py", "tests/test_gpu_experts_range.py", "tests/test_gpu_experts_routing.py",
          "tests/test_gpu_experts_graphs.py"]


def test_experts_edge_suites_pass_in_the_checked_build():
    lib = wbuild.build(checked=True)
    res = subprocess.run([sys.executable, "-m", "pytest", *SUITES, "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider"],
                         cwd=ROOT, env=_child_env(lib), capture_output=True, text=True, timeout=1800)
    tail = "\n".join((res.stdout + res.stderr).splitlines()[-30:])
    assert res.returncode == 0, tail
    assert " passed" in tail and " failed" not in tail, tail
