"""qk_gqa_attention_window at the ends of its range: a long tail of tiny weights."""
import math

import numpy as np
import pytest

from tests.test_gpu_operators import D, _host

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,H,Hkv", [(900, 24, 8), (2, 24, 8), (1, 24, 8)])
def test_a_long_tail_of_small_weights(qk_lib, cuda, M, H, Hkv):
    """Position 0 has all but 2^-8 of the weight; 2^17 others have 2^-25.05 of its
    weight each, and the only values that are not 0.  With L positions the exact
    result is x / (1 + x), x = 2^-25.05 (L - 1).  Allowed: 2^-10 of max|v| = 1, the
    bound that the header states."""
    import torch
    L, gap = 2 ** 17, 25.05
    scale = float(np.float32(gap * math.log(2) / 25))
    q = torch.zeros(M, H, D, dtype=torch.float16, device=cuda)
    q[:, :, 0] = 1
    k = torch.zeros(Hkv, L, D, dtype=torch.float16, device=cuda)
    k[:, 0, 0] = 25
    v = torch.ones(Hkv, L, D, dtype=torch.float16, device=cuda)
    v[:, 0] = 0
    out = torch.full((M, H, D), math.nan, dtype=torch.float16, device=cuda)
    qk_lib.qk_gqa_attention_window(q, k, v, out, M, H, Hkv, D, L - M, L, scale, L, 0)
    qk_lib.qk_get_device_status()
    x = math.exp(-25 * scale) * np.arange(L - M, L, dtype=np.float64)
    ref = (x / (1 + x))[:, None, None]
    assert ref.min() > 2.0 ** -8.2
    err = np.abs(_host(out).astype(np.float64) - ref).max()
    assert err <= 2.0 ** -10, err
    del k, v
