"""The operators that copy in bulk (products from int8 x, windowed attention) and
a run of all of them in the checked build (-DQK_DEBUG), where every bulk and
tensor copy is tested for alignment and shared-memory extent before it is
issued: their tests pass there too and leave the device status clean."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

_CHILD = r"""
import os, sys
sys.path.insert(0, sys.argv[1])
import pytest
rc = pytest.main([os.path.join(sys.argv[1], "tests", "test_gpu_operators.py"), "-x", "-q", "-p", "no:cacheprovider",
                  "-k", "window or matmul_q8 or decoder_layer"])
assert rc == 0, rc
import torch
import quantized_q4_matmul_gb300 as qk
torch.cuda.synchronize()
st = qk.lib().qk_get_device_status(None)
assert st == 0, qk.lib().qk_status_string(st).decode()
print("ok")
"""


def test_operators_in_the_checked_build(qk_lib, cuda, tmp_path):
    from quantized_q4_matmul_gb300 import build as qk_build
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    lib = qk_build.build(extra_flags=["-DQK_DEBUG"], out_dir=str(tmp_path))
    env = dict(os.environ, QK_LIB=lib)
    r = subprocess.run([sys.executable, "-c", _CHILD, root], env=env, capture_output=True, text=True, timeout=900)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stdout[-3000:] + r.stderr[-3000:]
