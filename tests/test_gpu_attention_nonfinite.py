"""Keys that are not finite, alone in what one warp or one CTA sees of a row:
attention's parts without a largest score still hand a NaN on.

Finite outputs have the tolerance of the other attention tests (derived at
_attn_check and at test_gpu_attention.py's bar).
"""
import numpy as np
import pytest

from tests.test_gpu_operators import D, SCALE, _attn, _attn_check, _attn_inputs, _attn_reference, _dev, _host

pytestmark = pytest.mark.gpu


def _compare(got, ref, v, what):
    got = got.astype(np.float64)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), what
    fine = np.isfinite(ref)
    assert np.isfinite(got[fine]).all(), what
    if fine.any():
        _attn_check(got[fine], ref[fine], v, what)


# (pos0, window, sinks, positions whose key is not finite): the newest position alone
# in a warp's 16, one distant sink, a warp's first slices, a rank's edge
DECODE = [(16, 17, 0, [16]), (64, 65, 0, [64]), (16, 100, 0, [16]), (0, 1, 0, [0]), (500, 200, 1, [0]),
          (500, 17, 0, [500]), (500, 17, 2, [484]), (300, 301, 0, range(16)), (5000, 4096, 4, [905, 3]),
          (5000, 4096, 0, [5000]), (5000, 4097, 1, [0]), (700, 0, 1, [0]), (700, 0, 17, [16])]


@pytest.mark.parametrize("value", [np.nan, np.inf])
@pytest.mark.parametrize("pos0,window,sinks,at", DECODE)
def test_window_decode_keys(qk_lib, cuda, pos0, window, sinks, at, value):
    """One element of the keys is NaN, or infinite: a score of -inf has weight 0,
    one of +inf makes its row NaN.  The second key/value head stays finite."""
    H, Hkv = 6, 2
    q, k, v = _attn_inputs(230, 1, H, Hkv, pos0, pos0 + 3, window, sinks)
    k[0, list(at), 5] = value
    got = _attn(qk_lib, cuda, q, k, v, H, Hkv, pos0, window, sinks)
    with np.errstate(invalid="ignore"):
        ref = _attn_reference(q, k, v, H, Hkv, pos0, window, sinks)
    assert np.isfinite(ref[:, 3:]).all() and (np.isnan(ref[:, :3]).all() or value == np.inf)
    _compare(got, ref, v, "decode")


@pytest.mark.parametrize("pos0,at", [(16, [16]), (64, [64]), (0, [0]), (300, range(16)), (2047, [2047]), (2048, [2048]),
                                     (2303, range(1792, 1808))])
def test_causal_decode_keys(qk_lib, cuda, pos0, at):
    """The causal decode step shares the kernel."""
    import torch
    H, Hkv = 6, 2
    q, k, v = _attn_inputs(231, 1, H, Hkv, pos0, pos0 + 3, pos0 + 1, 0)
    k[0, list(at), 5] = np.nan
    out = torch.full(q.shape, 7.0, device=cuda)
    qk_lib.qk_gqa_attention(*(_dev(a.view(np.uint16), cuda) for a in (q, k, v)), out, 1, H, Hkv, D, pos0, k.shape[1],
                            SCALE)
    qk_lib.qk_get_device_status()
    with np.errstate(invalid="ignore"):
        ref = _attn_reference(q, k, v, H, Hkv, pos0, pos0 + 1, 0)
    assert np.isnan(ref[:, :3]).all() and np.isfinite(ref[:, 3:]).all()
    _compare(_host(out), ref, v, "causal decode")


# One key that is NaN, at the edges of what a query sees and of what a CTA of the
# cluster takes.  M = 256: 18 key tiles from position 5953, two or three for each of
# eight CTAs; the last query's window begins at 6208, the last row of the first two.
@pytest.mark.parametrize("M,H,Hkv,pos0,window,sinks,at", [
    (256, 8, 8, 8000, 2048, 0, [6208, 6207, 6209, 8000, 8127, 8128, 8255]),
    (256, 8, 8, 8000, 2048, 1, [0, 6208]), (2, 6, 2, 6000, 4096, 0, [1905, 1906, 6001, 4000]),
    (9, 4, 1, 4000, 0, 4000, [0, 3999]), (300, 8, 8, 100, 150, 100, [0, 99, 399]), (40, 24, 8, 3000, 2900, 7, [140, 6])])
def test_window_prefill_keys(qk_lib, cuda, M, H, Hkv, pos0, window, sinks, at):
    """The queries that see it are NaN, in the heads that have it; every other
    output keeps its bits."""
    q, k, v = _attn_inputs(232, M, H, Hkv, pos0, pos0 + M, window, sinks)
    k, v = np.nan_to_num(k, posinf=0, neginf=0), np.nan_to_num(v, posinf=0, neginf=0)
    clean = _attn(qk_lib, cuda, q, k, v, H, Hkv, pos0, window, sinks)
    assert np.isfinite(clean).all()
    p = pos0 + np.arange(M)
    for j in at:
        bad = k.copy()
        bad[Hkv - 1, j, 77] = np.nan
        got = _attn(qk_lib, cuda, q, bad, v, H, Hkv, pos0, window, sinks)
        sees = (j <= p) & ((j > p - window) | (j < sinks))
        hit = np.zeros(got.shape, bool)
        hit[sees, H - H // Hkv:] = True
        assert np.array_equal(np.isnan(got), hit), (j, np.isnan(got).any((1, 2)).sum(), sees.sum())
        assert np.array_equal(got[~hit], clean[~hit]), j
