"""qk_gqa_attention_window at the ends of its range: a long tail of tiny weights,
and averages at the largest fp16 value."""
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


@pytest.mark.parametrize("M,H,Hkv,pos0,window,sinks", [
    (1, 24, 8, 15, 16, 0), (1, 6, 2, 15, 100, 0), (300, 24, 8, 0, 300, 0), (40, 8, 8, 2000, 2100, 0),
    (300, 8, 8, 500, 200, 1)])
@pytest.mark.parametrize("sign", [1, -1])
def test_values_at_the_largest_half(qk_lib, cuda, M, H, Hkv, pos0, window, sinks, sign):
    """Every value is +-65504, so every average is.  Position 0 has weight 1 and
    each other one 0.5 + 2^-12 + 2e-6, which rounds up to 0.5 + 2^-11 in fp16: the
    rounded weights' sum is up to 2^-11 too large, past 65520, which would round to
    infinity.  A row that does not reach it may be 2^-10 off."""
    import torch
    L = pos0 + M
    scale = float(np.float32(-math.log(0.5 + 2.0 ** -12 + 2e-6)))
    q = torch.zeros(M, H, D, dtype=torch.float16, device=cuda)
    q[:, :, 0] = 1
    k = torch.zeros(Hkv, L, D, dtype=torch.float16, device=cuda)
    k[:, 1:, 0] = -1
    v = torch.full((Hkv, L, D), 65504.0 * sign, dtype=torch.float16, device=cuda)
    out = torch.full((M, H, D), math.nan, dtype=torch.float16, device=cuda)
    qk_lib.qk_gqa_attention_window(q, k, v, out, M, H, Hkv, D, pos0, L, scale, window, sinks)
    qk_lib.qk_get_device_status()
    got = _host(out).astype(np.float64) * sign
    assert np.isfinite(got).all() and (got >= 65504 * (1 - 2.0 ** -10)).all(), (np.isinf(got).sum(), got.min())
