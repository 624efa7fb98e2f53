"""The GEMV's rows in K chunks, the last of them smaller (copy length and
destination pitch differ), in the checked build (-DQK_DEBUG), where every bulk
copy is tested for alignment and shared-memory extent before it is issued."""
import os
import subprocess
import sys

import pytest

from tests import test_gpu_operators

pytestmark = pytest.mark.gpu

_CHILD = r"""
import os, sys
sys.path.insert(0, sys.argv[1])
import pytest

class Count:
    passed = 0
    def pytest_runtest_logreport(self, report):
        self.passed += report.when == "call" and report.passed

count = Count()
rc = pytest.main([os.path.join(sys.argv[1], "tests", "test_gpu_operators.py"), "-x", "-q", "-p", "no:cacheprovider",
                  "-k", "test_matmul_rows_in_unequal_chunks"], plugins=[count])
assert rc == 0, rc
import torch
import quantized_q4_matmul_gb300 as qk
torch.cuda.synchronize()
st = qk.lib().qk_get_device_status(None)
assert st == 0, qk.lib().qk_status_string(st).decode()
print("passed", count.passed)
"""


def test_unequal_chunks_in_the_checked_build(qk_lib, cuda, tmp_path):
    from quantized_q4_matmul_gb300 import build as qk_build
    cases = [m for m in test_gpu_operators.test_matmul_rows_in_unequal_chunks.pytestmark if m.name == "parametrize"]
    assert len(cases) == 1 and len(cases[0].args[1]) >= 4
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    lib = qk_build.build(extra_flags=["-DQK_DEBUG"], out_dir=str(tmp_path))
    env = dict(os.environ, QK_LIB=lib)
    r = subprocess.run([sys.executable, "-c", _CHILD, root], env=env, capture_output=True, text=True, timeout=900)
    said = r.stdout.strip().splitlines()[-1:]
    assert r.returncode == 0 and said == ["passed %d" % len(cases[0].args[1])], r.stdout[-3000:] + r.stderr[-3000:]
