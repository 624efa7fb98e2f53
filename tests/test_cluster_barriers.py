"""The cluster barriers are .aligned: all lanes of a warp execute them together.
Every call in the kernels follows a __syncwarp(), so that lanes which just left a
branch have met again."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "quantized_q4_matmul_gb300", "csrc")


def test_every_cluster_barrier_follows_a_syncwarp():
    calls, bare = 0, []
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        with open(path) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        assert "barrier.cluster" not in text, path  # the helpers of qk_device.cuh are the only ones
        statements = [s.strip() for s in re.split(r"[;{}]", text)]
        statements = [s for s in statements if s]
        for before, s in zip(statements, statements[1:]):
            if re.search(r"\bcluster_(sync_all|arrive|wait)\(\)$", s):
                calls += 1
                if before != "__syncwarp()":
                    bare.append((os.path.basename(path), before, s))
    assert calls >= 9 and not bare, bare
