"""Head norms with rotary positions and the cache append, the 4-bit cache and
attention over it, against plain numpy in 64 bits, through the binding.

Tolerances are sums of the roundings on the way: half a step of the output's
type (fp16 2^-11 relative, 2^-25 below the normal range) and the fp32
arithmetic's share, derived beside each test.
"""
import math

import numpy as np
import pytest

from tests import kv4_reference as ref4
from tests import synth

pytestmark = pytest.mark.gpu

EPS = 1e-6
D = 128
SCALE = 1 / math.sqrt(D)


def _dev(a, cuda):
    import torch
    a = np.ascontiguousarray(a)
    return torch.from_numpy(a.view(np.uint16)).to(cuda).view(torch.float16) if a.dtype == np.float16 else torch.from_numpy(
        a).to(cuda)


def _host(t):
    return t.cpu().numpy()


def _within(got, ref, tol, what):
    bad = ~(np.abs(got.astype(np.float64) - ref) <= tol)
    assert not bad.any(), "%s: %d of %d off, worst %.3e (allowed %.3e)" % (
        what, bad.sum(), bad.size, np.nanmax(np.abs(got - ref)), np.max(tol))


# ---------------------------------------------------------------------------
# Head norms, rotary positions, cache append
# ---------------------------------------------------------------------------
def _append_case(qk, cuda, M, H, Hkv, Dh, n_rot, pos0, L, half, qn, kn, mag=1.0, size=1.0, seed=401):
    """Both forms of one call, checked; returns the 4-bit cache."""
    import torch
    rng = synth.rng_for(seed, M * 7 + Dh + n_rot)
    q, k, v = (size * rng.standard_normal((M, h, Dh)).astype(np.float32) for h in (H, Hkv, Hkv))
    gq, gk = ((1 + 0.2 * rng.standard_normal(Dh)).astype(np.float16) if on else None for on in (qn, kn))
    f = 500000.0 ** (-np.arange(0, n_rot, 2, dtype=np.float64) / max(1, n_rot))
    angle = np.arange(pos0, pos0 + M, dtype=np.float64)[:, None] * f[None]
    layout = qk.QK_ROPE_HALF if half else qk.QK_ROPE_INTERLEAVED
    head = [_dev(a, cuda) if a is not None else None for a in (q, k, v, gq, gk)] + [EPS, _dev(f, cuda) if n_rot else None]
    sizes = (M, H, Hkv, Dh, n_rot, pos0, L)

    def exact(x, gamma):
        """(64-bit values, what fp32 may be off by), in steps of 2^-24: a lane adds 8 (D > 256:
        16) squares and shuffles 5 more, halved by the root; the mean and eps one half each;
        rsqrtf 4; two products 2.  Sine and cosine within 2^-21, two products and a sum of
        2^-24.  A rotated value has two such parts."""
        y = ref4.head_norm(x, gamma, EPS)
        most = np.abs(y).max(-1, keepdims=True) * 2 * max(1.0, abs(mag))
        return ref4.rotate(y, angle, n_rot, half, mag), most * (2.0 ** -20.5 + ((21 if Dh > 256 else 13) / 2 + 7) * 2.0 ** -24)

    eq, dq = exact(q, gq)
    ek, dk = exact(k, gk)
    qo = torch.full((M, H, Dh), math.nan, dtype=torch.float16, device=cuda)
    kc0, vc0 = (rng.standard_normal((Hkv, L, Dh)).astype(np.float16) for _ in range(2))
    kc, vc = _dev(kc0, cuda), _dev(vc0, cuda)
    qk.qk_norm_rope_kv_append(*head, qo, kc, vc, *sizes, layout=layout, magnitude=mag)
    new = slice(pos0, pos0 + M)
    _within(_host(qo), eq, np.abs(eq) * 2.0 ** -11 + dq + 2.0 ** -25, "q")
    _within(_host(kc)[:, new].transpose(1, 0, 2), ek, np.abs(ek) * 2.0 ** -11 + dk + 2.0 ** -25, "k")
    assert np.array_equal(_host(vc)[:, new].transpose(1, 0, 2), v.astype(np.float16))
    for got, was in ((_host(kc), kc0), (_host(vc), vc0)):  # the other rows are untouched
        assert np.array_equal(got[:, :pos0], was[:, :pos0]) and np.array_equal(got[:, pos0 + M:], was[:, pos0 + M:])
    if Dh % 32:
        return None
    k40, kd0 = ref4.random_cache(rng, Hkv, L, Dh)
    v40, vd0 = ref4.random_cache(rng, Hkv, L, Dh)
    k4, kd, v4, vd = (_dev(a, cuda) for a in (k40, kd0, v40, vd0))
    qo4 = torch.full_like(qo, math.nan)
    qk.qk_norm_rope_kv_append_q4(*head, qo4, k4, kd, v4, vd, *sizes, layout=layout, magnitude=mag)
    assert torch.equal(qo, qo4)
    for got, was in ((k4, k40), (kd, kd0), (v4, v40), (vd, vd0)):
        got = _host(got)
        assert np.array_equal(got[:, :pos0], was[:, :pos0]) and np.array_equal(got[:, pos0 + M:], was[:, pos0 + M:])
    # v comes from the inputs themselves: to the bit
    pq, pdm = ref4.pack(v.transpose(1, 0, 2))
    assert np.array_equal(_host(v4)[:, new], pq) and np.array_equal(_host(vd)[:, new].view(np.uint16), pdm.view(np.uint16))
    # k: m and d are the roundings of values within dk, each q is a level nearest to such a value
    lv, d, m = ref4.unpack(_host(k4)[:, new], _host(kd)[:, new])
    x = ek.transpose(1, 0, 2)
    off = np.broadcast_to(dk.transpose(1, 0, 2), x.shape).reshape(*d.shape, 32)[..., 0]
    b = x.reshape(*d.shape, 32)
    _within(m, b.min(-1), np.abs(b.min(-1)) * 2.0 ** -11 + 2.0 ** -25 + 1.001 * off, "m")
    _within(d, np.maximum(b.max(-1) - m, 0) / 15, d * 2.0 ** -10.99 + 2.0 ** -25 + off, "d")
    level = np.clip(lv.reshape(*d.shape, 32), 0, 15)
    dist = np.abs(d[..., None] * level + m[..., None] - b)
    best = np.abs(d[..., None, None] * np.arange(16) + m[..., None, None] - b[..., None]).min(-1)
    _within(dist, best, np.broadcast_to(2 * off[..., None] + d[..., None] * 2.0 ** -18, dist.shape), "k's levels")
    return k4, kd, v4, vd


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("Dh,n_rot", [(128, 128), (128, 64), (128, 96), (80, 46), (64, 2), (64, 0), (8, 8), (256, 256),
                                      (512, 512), (96, 30), (72, 72), (40, 4), (32, 32), (320, 100), (16, 6)])
@pytest.mark.parametrize("M", [1, 9])
def test_append_layouts(qk_lib, cuda, M, Dh, n_rot, half):
    _append_case(qk_lib, cuda, M, 6, 2, Dh, n_rot, 1000, 1000 + M + 3, half, True, True)


@pytest.mark.parametrize("qn,kn", [(True, False), (False, True), (False, False)])
@pytest.mark.parametrize("half", [False, True])
def test_append_with_some_norms(qk_lib, cuda, qn, kn, half):
    _append_case(qk_lib, cuda, 5, 8, 4, 96, 64, 3, 10, half, qn, kn, mag=1.25)


@pytest.mark.parametrize("M,H,Hkv,Dh,pos0", [(1, 24, 8, 128, 0), (2, 1, 1, 128, 5), (63, 8, 8, 64, 0), (65, 32, 4, 128, 100),
                                             (303, 24, 8, 128, 1), (700, 5, 3, 32, 31), (1, 1024, 1024, 64, 3),
                                             (400, 2, 1, 512, 0), (3, 7, 7, 256, 131071)])
def test_append_sizes(qk_lib, cuda, M, H, Hkv, Dh, pos0):
    _append_case(qk_lib, cuda, M, H, Hkv, Dh, Dh, pos0, pos0 + M, M % 2 == 0, True, True)


@pytest.mark.parametrize("size", [1e-6, 1e-3, 3000.0])
def test_append_small_and_large_values(qk_lib, cuda, size):
    """Groups whose d is subnormal or 0, and rows that the norm brings back to 1."""
    for qn in (True, False):
        _append_case(qk_lib, cuda, 4, 4, 2, 64, 64, 7, 20, True, qn, qn, size=size)


def test_append_constant_and_bad_groups(qk_lib, cuda):
    """A constant group has d = 0 or its rounding's remainder; zero rows are zero; a group
    with NaN, an infinity or more than fp16 holds is NaN, and no other."""
    import torch
    M, Hkv, Dh, L = 6, 2, 64, 8
    k = np.zeros((M, Hkv, Dh), np.float32)
    v = np.zeros((M, Hkv, Dh), np.float32)
    k[1], v[1] = 5.003, -5.003
    v[2, 0, 5], v[2, 1, 40] = np.nan, np.inf
    v[3, 0, 31], v[3, 1, :32] = -np.inf, np.nan
    v[4, 0, 0], v[4, 1, 63] = 1e6, -1e6
    v[5] = np.linspace(-65000, 65000, Dh, dtype=np.float32)[None]
    z = torch.zeros(M, 2, Dh, device=cuda)
    k4, v4 = (torch.full((Hkv, L, Dh // 2), 255, dtype=torch.uint8, device=cuda) for _ in range(2))
    kd, vd = (torch.zeros(Hkv, L, Dh // 32, 2, dtype=torch.float16, device=cuda) for _ in range(2))
    qo = torch.empty(M, 2, Dh, dtype=torch.float16, device=cuda)
    g = torch.ones(Dh, dtype=torch.float16, device=cuda)
    qk_lib.qk_norm_rope_kv_append_q4(z, _dev(k, cuda), _dev(v, cuda), g, None, EPS, None, qo, k4, kd, v4, vd, M, 2, Hkv, Dh,
                                     0, 1, L)
    assert (qo == 0).all()
    out = torch.empty(Hkv, M, Dh, dtype=torch.float16, device=cuda)
    for x, q4, dm in ((k, k4, kd), (v, v4, vd)):
        qk_lib.qk_dequant_kv_q4(q4, dm, out, Hkv, Dh, 1, M, L)
        got = _host(out).astype(np.float64)
        for i in range(M):
            for h in range(Hkv):
                for a in (0, 32):
                    b = x[i, h, a: a + 32]
                    if not (np.abs(b) <= 65504).all():
                        assert np.isnan(got[h, i, a: a + 32]).all(), (i, h, a)
                        continue
                    d = (float(b.max()) - float(b.min())) / 15
                    # half a step, and the roundings of m, 15 d and the value
                    _within(got[h, i, a: a + 32], b.astype(np.float64),
                            d / 2 + np.abs(b.astype(np.float64)).max() * 2.0 ** -9 + 2.0 ** -24, (i, h, a))
    assert (_host(out)[:, 0] == 0).all() and (_host(v4)[:, 0] == 255).all() and (_host(v4)[:, 1 + M:] == 255).all()


@pytest.mark.parametrize("Hkv,Dh,L,pos0,M", [(1, 32, 1, 0, 1), (3, 128, 700, 0, 700), (2, 96, 50, 17, 31), (8, 512, 40, 39, 1),
                                             (1, 256, 3000, 5, 2900)])
def test_dequant_rows(qk_lib, cuda, Hkv, Dh, L, pos0, M):
    """To the bit, with subnormal, huge and NaN scales among them; nothing past the rows is written."""
    import torch
    rng = synth.rng_for(402, L * Dh)
    q4 = rng.integers(0, 256, (Hkv, L, Dh // 2), dtype=np.uint8)
    dm = rng.integers(0, 65536, (Hkv, L, Dh // 32, 2), dtype=np.uint16).view(np.float16)
    out = torch.full((Hkv * M * Dh + 64,), 7.0, dtype=torch.float16, device=cuda)
    qk_lib.qk_dequant_kv_q4(_dev(q4, cuda), _dev(dm, cuda), out, Hkv, Dh, pos0, M, L)
    got, ref = _host(out)[:-64].reshape(Hkv, M, Dh), ref4.values(q4, dm)[:, pos0: pos0 + M]
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    fine = ~np.isnan(ref)
    assert np.array_equal(got[fine], ref[fine]) and (_host(out)[-64:] == 7).all()


# ---------------------------------------------------------------------------
# Attention over the 4-bit cache
# ---------------------------------------------------------------------------
def _attn_inputs(seed, M, H, Hkv, pos0, L, window, sinks):
    """Inputs whose rows that no query sees are NaN or infinite."""
    rng = synth.rng_for(seed, M * 1000 + pos0 + window % 100003)
    q = (1.5 * rng.standard_normal((M, H, D))).astype(np.float16)
    cache = ref4.random_cache(rng, Hkv, L) + ref4.random_cache(rng, Hkv, L)
    j = np.arange(L)
    unseen = (j >= pos0 + M) | ((j <= pos0 - window) & (j >= sinks)) | (window == 0) & (j >= sinks)
    for dm in cache[1::2]:
        dm[:, unseen] = np.where(j[unseen] % 2, np.nan, np.inf)[None, :, None, None]
    return q, cache


def _attn(qk, cuda, q, cache, H, Hkv, pos0, window, sinks, scratch=None):
    import torch
    M = q.shape[0]
    out = torch.full(q.shape, math.nan, dtype=torch.float16, device=cuda)
    need = qk.qk_gqa_attention_q4_scratch_bytes(M, H, Hkv, D, pos0, window, sinks)
    if scratch is None and need:
        scratch = torch.full((need + 64,), 0x7E, dtype=torch.uint8, device=cuda)  # NaN until it is written
    qk.qk_gqa_attention_q4(_dev(q, cuda), *(_dev(a, cuda) for a in cache), out, M, H, Hkv, D, pos0, cache[0].shape[1],
                           SCALE, window, sinks, scratch=scratch)
    qk.qk_get_device_status()
    if need:
        assert (scratch[need:] == 0x7E).all()
    return _host(out)


def _check(qk, cuda, seed, M, H, Hkv, pos0, window, sinks, slack=3, rows=None):
    """Weights rounded to fp16 2^-11 relative each, those below 2^-24 of the largest flushed
    (2^-25 each, 2^13 of them in a warp at most), scores in fp32 (2^-12 of a weight in
    all), the output's rounding 2^-11: against the largest |v|.  Few tokens have the
    exact values d q + m, whose d (q - 8) is rounded, 2^-11 of 8 d; chunks those of fp16."""
    q, cache = _attn_inputs(seed, M, H, Hkv, pos0, pos0 + M + slack, window, sinks)
    few = M * (H // Hkv) <= 32
    k, v = ((ref4.exact if few else ref4.values)(*c) for c in (cache[:2], cache[2:]))
    got = _attn(qk, cuda, q, cache, H, Hkv, pos0, window, sinks)
    assert np.isfinite(got).all()
    vmax = np.abs(v[np.isfinite(v)].astype(np.float64)).max()
    if rows is not None:
        got = got[rows]
    _within(got, ref4.attention(q, k, v, H, Hkv, pos0, window, sinks, SCALE, rows),
            vmax * (2.0 ** -10 + 2.0 ** -12 + 2.0 ** -12) + few * 8 * 0.35 * 2.0 ** -11, "attention")


NONE = 10 ** 9


@pytest.mark.parametrize("pos0,window,sinks", [
    (0, 1, 0), (0, 0, 1), (0, 5, 3), (15, 16, 0), (15, NONE, 0), (16, NONE, 0), (63, 64, 0), (64, 64, 1), (255, NONE, 0),
    (256, NONE, 0), (700, 1, 0), (700, 0, 2), (700, 0, 100), (700, 1, 64), (700, 65, 65), (700, 635, 66), (700, 634, 66),
    (700, 636, 66), (700, NONE, 0), (700, 3, 701), (700, 0, 10 ** 6), (5000, 4096, 4), (5000, 1000, 300), (4095, 4095, 0),
    (9000, 300, 1), (9000, NONE, 0)])
def test_attention_one_token(qk_lib, cuda, pos0, window, sinks):
    _check(qk_lib, cuda, 403, 1, 24, 8, pos0, window, sinks)


@pytest.mark.parametrize("H,Hkv", [(8, 8), (32, 4), (6, 2), (4, 1), (7, 1), (24, 8), (40, 40), (5, 5), (16, 2)])
def test_attention_group_sizes(qk_lib, cuda, H, Hkv):
    for M, pos0, window, sinks in ((1, 900, 333, 9), (1, 2077, NONE, 0), (2, 1500, NONE, 0), (3, 640, 257, 130),
                                   (40, 200, 90, 5)):
        _check(qk_lib, cuda, 404, M, H, Hkv, pos0, window, sinks)


@pytest.mark.parametrize("M,pos0,window,sinks,H,Hkv", [
    (2, 0, NONE, 0, 8, 8), (8, 0, NONE, 0, 8, 8), (8, 0, 3, 2, 8, 8), (9, 1000, NONE, 0, 8, 8), (16, 3000, NONE, 0, 8, 8),
    (17, 3000, 1000, 5, 8, 8), (32, 5000, NONE, 0, 4, 4), (32, 0, 7, 3, 4, 4), (5, 20000, 8192, 4, 24, 8), (10, 77, NONE, 0, 24, 8),
    (10, 9000, NONE, 0, 24, 8), (4, 4000, 0, 900, 16, 2), (4, 3, 0, 5, 16, 2), (8, 500, 1, 0, 12, 3),
    (31, 100, 50, 60, 2, 2), (2, 40, 20, 10 ** 7, 6, 2)])
def test_attention_few_tokens(qk_lib, cuda, M, pos0, window, sinks, H, Hkv):
    """Several tokens in one to four tiles of columns; each its own window."""
    _check(qk_lib, cuda, 405, M, H, Hkv, pos0, window, sinks)


@pytest.mark.parametrize("M,pos0,window,sinks", [
    (11, 0, NONE, 0), (100, 0, NONE, 0), (129, 0, 128, 0), (257, 0, 1, 1), (300, 0, 0, 200), (300, 37, 0, 5), (33, 777, 200, 4),
    (130, 1000, 129, 127), (130, 1000, 64, 300), (260, 500, 300, 600), (515, 300, 250, 17), (200, 3, 50, 10 ** 7),
    (40, 6000, 4096, 4), (64, 3000, 1, 1500)])
def test_attention_chunks(qk_lib, cuda, M, pos0, window, sinks):
    assert qk_lib.qk_gqa_attention_q4_scratch_bytes(M, 6, 2, D, pos0, window, sinks) > 0
    _check(qk_lib, cuda, 406, M, 6, 2, pos0, window, sinks)


def test_attention_large_chunk_sampled(qk_lib, cuda):
    M = 1023
    rows = np.unique(np.concatenate([[0, 1, 127, 128, M - 1], synth.rng_for(407, 0).choice(M, 30)]))
    _check(qk_lib, cuda, 408, M, 24, 8, 1701, NONE, 0, rows=rows)


def test_attention_long_cache(qk_lib, cuda):
    """100000 positions.  A warp's share of 391 rounds its small weights to fp16 one by one:
    2^-25 each of the largest, 2^-16 in all; the tolerance above holds."""
    _check(qk_lib, cuda, 409, 1, 4, 2, 99999, NONE, 0)


@pytest.mark.parametrize("M,pos0,H,Hkv", [(1, 500, 32, 8), (1, 40000, 8, 2), (1, 60000, 8, 8), (5, 3000, 24, 8), (10, 700, 24, 8),
                                          (4, 50000, 8, 4)])
def test_attention_few_tokens_precision(qk_lib, cuda, M, pos0, H, Hkv):
    """Three roundings to fp16 (weights, d (q - 8), outputs) of at most half a step, evenly
    spread: 2^-11 / sqrt(3) of a value each, at random.  Of random values, whose mean nearly
    vanishes, d (q - 8) is as large as d q + m: together 2^-11 in the 2-norm.  Scores are off by
    2^-21 of sums of 1024 |Q| d 32, 2^-11 / sqrt(3) less by far."""
    q, cache = _attn_inputs(419, M, H, Hkv, pos0, pos0 + M, NONE, 0)
    want = ref4.attention(q, ref4.exact(*cache[:2]), ref4.exact(*cache[2:]), H, Hkv, pos0, NONE, 0, SCALE)
    got = _attn(qk_lib, cuda, q, cache, H, Hkv, pos0, NONE, 0).astype(np.float64)
    assert np.linalg.norm(got - want) <= 2.0 ** -11 * np.linalg.norm(want)


@pytest.mark.parametrize("M,sizes", [(1, (1e-3, 1.0, 300.0, 2e-4)), (3, (1e-3, 1.0, 300.0, 2e-4)), (10, (1.0, 1e-3, 3.0, 0.1))])
def test_attention_heads_of_very_different_sizes(qk_lib, cuda, M, sizes):
    """Queries of one key/value head whose sizes lie far apart: each as exact as alone.  Of
    the largest, whose scores are beyond what fp32 holds to 2^-12, only that they are finite."""
    q, cache = _attn_inputs(420, M, 8, 2, 900, 900 + M, NONE, 0)
    size = np.array(sizes * 2)[None, :, None]
    q = (q * size).astype(np.float16)
    k, v = ref4.exact(*cache[:2]), ref4.exact(*cache[2:])
    want = ref4.attention(q, k, v, 8, 2, 900, NONE, 0, SCALE)
    got = _attn(qk_lib, cuda, q, cache, 8, 2, 900, NONE, 0)
    assert np.isfinite(got).all()
    fine = np.flatnonzero(size[0, :, 0] < 100)
    vmax = np.abs(v).max()
    _within(got[:, fine], want[:, fine], vmax * (2.0 ** -10 + 2.0 ** -11) + 8 * 0.35 * 2.0 ** -11, "heads")


def test_attention_sees_nothing(qk_lib, cuda):
    for M in (1, 3, 50):
        q, cache = _attn_inputs(410, M, 6, 2, 30, 90, 0, 0)
        assert qk_lib.qk_gqa_attention_q4_scratch_bytes(M, 6, 2, D, 30, 0, 0) == 0
        assert (_attn(qk_lib, cuda, q, cache, 6, 2, 30, 0, 0) == 0).all()


@pytest.mark.parametrize("M,H,Hkv", [(1, 6, 2), (2, 6, 2), (5, 6, 2), (10, 6, 2), (24, 6, 2)])
def test_attention_non_finite_rows(qk_lib, cuda, M, H, Hkv):
    """A NaN key makes its row's queries NaN; a NaN or infinite value group its 32 dimensions;
    queries that do not see the row are as without it.  Alone in a warp's share too."""
    pos0, window, sinks = 600, 100, 3
    need = M * (H // Hkv) > 32  # a chunk
    for key, row in ((False, pos0 + M - 1), (False, pos0 - 50), (False, 1), (True, pos0 + M - 1), (True, pos0 - 97),
                     (True, 2)):
        for bad in (np.nan, np.inf):
            if key and bad == np.inf:
                continue  # a score of infinity or NaN by q's sign: not pinned
            q, cache = _attn_inputs(411, M, H, Hkv, pos0, pos0 + M, window, sinks)
            clean = _attn(qk_lib, cuda, q, cache, H, Hkv, pos0, window, sinks)
            cache[1 if key else 3][1, row, 2] = bad
            got = _attn(qk_lib, cuda, q, cache, H, Hkv, pos0, window, sinks)
            hit = np.zeros(got.shape, bool)
            for i in range(M):
                if row in ref4.seen(pos0 + i, window, sinks):
                    hit[i, H // Hkv:, slice(None) if key else slice(64, 96)] = True
            assert np.array_equal(~np.isfinite(got), hit), (key, row, bad)
            # In a chunk the value row meets the weight 0 of the tile's queries that do not see
            # it, and rows that are not finite then are done again, in another order: each of
            # the two results is within _check's bound of the exact one, so they are within
            # twice that of each other.  Few tokens have the same bits.
            assert need or np.array_equal(got[~hit], clean[~hit])
            vmax = 15 * 0.35 + 1.5 + 7.5 * 0.35  # of random_cache: |m| at most 7.5 d + 5 x 0.3
            _within(got[~hit], clean[~hit].astype(np.float64), 2 * vmax * (2.0 ** -10 + 2.0 ** -11), "finite parts")


@pytest.mark.parametrize("M", [1, 4, 10, 60])
def test_attention_is_deterministic_and_leaves_the_cache(qk_lib, cuda, M):
    import torch
    q, cache = _attn_inputs(412, M, 24, 8, 5000, 5000 + M, 3000, 4)
    dev = [_dev(a, cuda) for a in cache]
    was = [t.clone() for t in dev]
    need = qk_lib.qk_gqa_attention_q4_scratch_bytes(M, 24, 8, D, 5000, 3000, 4)
    outs = []
    for _ in range(3):
        out = torch.empty(M, 24, D, dtype=torch.float16, device=cuda)
        qk_lib.qk_gqa_attention_q4(_dev(q, cuda), *dev, out, M, 24, 8, D, 5000, 5000 + M, SCALE, 3000, 4,
                                   scratch=torch.empty(need, dtype=torch.uint8, device=cuda) if need else None)
        outs.append(out)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(dev, was))


def test_attention_large_values(qk_lib, cuda):
    """Averages of values near fp16's largest stay finite."""
    import torch
    rng = synth.rng_for(413, 0)
    for M in (1, 3, 40):
        L = 300 + M
        q = (rng.standard_normal((M, 4, D))).astype(np.float16)
        k4, kd = ref4.random_cache(rng, 2, L)
        v4 = np.full((2, L, D // 2), 0xFF, np.uint8)
        vd = np.zeros((2, L, 4, 2), np.float16)
        vd[..., 0], vd[..., 1] = 4000.0, 5504.0  # 65504
        got = _attn(qk_lib, cuda, q, (k4, kd, v4, vd), 4, 2, 300, NONE, 0)
        _within(got, 65504.0, 65504 * 2.0 ** -10, "largest")


def test_scale_zero_and_negative(qk_lib, cuda):
    import torch
    for M in (1, 4, 40):
        q, cache = _attn_inputs(414, M, 6, 2, 500, 500 + M, 200, 3)
        k, v = ref4.values(*cache[:2]), ref4.values(*cache[2:])
        need = qk_lib.qk_gqa_attention_q4_scratch_bytes(M, 6, 2, D, 500, 200, 3)
        vmax = np.abs(v[np.isfinite(v)].astype(np.float64)).max()
        for scale in (0.0, -SCALE):
            out = torch.empty(M, 6, D, dtype=torch.float16, device=cuda)
            qk_lib.qk_gqa_attention_q4(_dev(q, cuda), *(_dev(a, cuda) for a in cache), out, M, 6, 2, D, 500, 500 + M, scale,
                                       200, 3, scratch=torch.empty(need, dtype=torch.uint8, device=cuda) if need else None)
            _within(_host(out), ref4.attention(q, k, v, 6, 2, 500, 200, 3, scale), vmax * 2.0 ** -9.4, scale)


# ---------------------------------------------------------------------------
# Calls that are refused, other streams, graphs
# ---------------------------------------------------------------------------
def test_overlapping_buffers_are_refused(qk_lib, cuda):
    import torch
    M, L = 40, 64
    q, cache = _attn_inputs(415, M, 6, 2, 0, L, NONE, 0)
    qd = _dev(q, cuda)
    dev = [_dev(a, cuda) for a in cache]
    out = torch.empty(M, 6, D, dtype=torch.float16, device=cuda)
    need = qk_lib.qk_gqa_attention_q4_scratch_bytes(M, 6, 2, D, 0, NONE, 0)
    scratch = torch.empty(need + 65536, dtype=torch.uint8, device=cuda)

    def call(q=qd, dev=dev, out=out, scratch=scratch):
        qk_lib.qk_gqa_attention_q4(q, *dev, out, M, 6, 2, D, 0, L, SCALE, NONE, 0, scratch=scratch)

    call()
    with pytest.raises(ValueError):
        call(scratch=scratch[: need - 16])
    with pytest.raises(ValueError):
        call(dev=[dev[0].view(torch.int8)] + dev[1:])
    for bad in (dict(out=qd), dict(scratch=None), dict(out=scratch.view(torch.float16)[:M * 6 * D].view(M, 6, D)),
                dict(q=scratch[4096:].view(torch.float16)[: M * 6 * D].view(M, 6, D))):
        with pytest.raises(qk_lib.QKError) as e:
            call(**bad)
        assert e.value.status == (-1 if "scratch" in bad else -7)
    k = torch.zeros(2, 2, 64, device=cuda)
    k4 = torch.zeros(2, 8, 32, dtype=torch.uint8, device=cuda)
    dm = torch.zeros(2, 8, 2, 2, dtype=torch.float16, device=cuda)
    qo = torch.zeros(2, 2, 64, dtype=torch.float16, device=cuda)
    with pytest.raises(qk_lib.QKError) as e:
        qk_lib.qk_norm_rope_kv_append_q4(k, k, k, None, None, EPS, None, qo, k4, dm, k4, dm.clone(), 2, 2, 2, 64, 0, 0, 8)
    assert e.value.status == -7
    with pytest.raises(qk_lib.QKError) as e:
        qk_lib.qk_dequant_kv_q4(k4, dm, k4.view(torch.float16), 2, 64, 0, 1, 8)
    assert e.value.status == -7


def test_offsets_beyond_32_bits(qk_lib, cuda):
    """A cache whose tensors pass 4 GB: rows at its end are read and written as in a short
    one, to the bit."""
    import torch
    Hkv, H, far, n = 2, 6, 40_000_000, 150
    rng = synth.rng_for(421, 0)
    small = [_dev(a, cuda) for a in ref4.random_cache(rng, Hkv, n) + ref4.random_cache(rng, Hkv, n)]
    big = [torch.empty(Hkv, far + n, *t.shape[2:], dtype=t.dtype, device=cuda) for t in small]
    assert big[0].numel() > 1 << 32
    for b, t in zip(big, small):
        b[:, far:] = t
    for M, pos0 in ((1, n - 1), (5, n - 5), (40, n - 40)):
        q = _dev((1.5 * rng.standard_normal((M, H, D))).astype(np.float16), cuda)
        outs = []
        for cache, at, L in ((small, pos0, n), (big, far + pos0, far + n)):
            need = qk_lib.qk_gqa_attention_q4_scratch_bytes(M, H, Hkv, D, at, 64, 0)
            out = torch.empty_like(q)
            qk_lib.qk_gqa_attention_q4(q, *cache, out, M, H, Hkv, D, at, L, SCALE, 64, 0,
                                       scratch=torch.empty(need, dtype=torch.uint8, device=cuda) if need else None)
            outs.append(out)
        assert torch.equal(*outs), M
    rows = [torch.empty(Hkv, n, D, dtype=torch.float16, device=cuda) for _ in range(2)]
    qk_lib.qk_dequant_kv_q4(*small[:2], rows[0], Hkv, D, 0, n, n)
    qk_lib.qk_dequant_kv_q4(*big[:2], rows[1], Hkv, D, far, n, far + n)
    assert torch.equal(*rows)
    x = [_dev(rng.standard_normal((3, h, D)).astype(np.float32), cuda) for h in (H, Hkv, Hkv)]
    q16 = torch.empty(3, H, D, dtype=torch.float16, device=cuda)
    for cache, at, L in ((small, 70, n), (big, far + 70, far + n)):
        qk_lib.qk_norm_rope_kv_append_q4(*x, None, None, EPS, None, q16, *cache, 3, H, Hkv, D, 0, at, L)
    for b, t in zip(big, small):
        assert torch.equal(b[:, far:].contiguous().view(torch.uint8), t.view(torch.uint8))
    del big, b
    far //= 2  # fp16 rows are longer
    wide = [torch.empty(Hkv, far, D, dtype=torch.float16, device=cuda) for _ in range(2)]
    want = [torch.empty(Hkv, n, D, dtype=torch.float16, device=cuda) for _ in range(2)]
    qk_lib.qk_norm_rope_kv_append(*x, None, None, EPS, None, q16, *wide, 3, H, Hkv, D, 0, far - 3, far)
    qk_lib.qk_norm_rope_kv_append(*x, None, None, EPS, None, q16, *want, 3, H, Hkv, D, 0, n - 3, n)
    for w, t in zip(wide, want):
        assert torch.equal(w[:, far - 3:], t[:, n - 3:])
    del wide, w
    torch.cuda.empty_cache()


def test_step_on_a_side_stream_and_in_a_graph(qk_lib, cuda):
    """Append, attention and append again as a decode loop makes them, on a stream of its
    own and replayed from a graph: the same bits as call by call."""
    import torch
    rng = synth.rng_for(416, 0)
    H, Hkv, L, M = 24, 8, 400, 50
    q, k, v = (_dev(rng.standard_normal((M, h, D)).astype(np.float32), cuda) for h in (H, Hkv, Hkv))
    gq, gk = (_dev((1 + 0.2 * rng.standard_normal(D)).astype(np.float16), cuda) for _ in range(2))
    f = _dev(500000.0 ** (-np.arange(0, D, 2) / D), cuda)
    need = qk_lib.qk_gqa_attention_q4_scratch_bytes(M, H, Hkv, D, 100, NONE, 0)

    def buffers():
        c = [torch.zeros(Hkv, L, D // 2, dtype=torch.uint8, device=cuda), torch.zeros(Hkv, L, 4, 2, dtype=torch.float16, device=cuda)]
        return dict(cache=c + [t.clone() for t in c], q=torch.zeros(M, H, D, dtype=torch.float16, device=cuda),
                    many=torch.zeros(M, H, D, dtype=torch.float16, device=cuda),
                    one=torch.zeros(1, H, D, dtype=torch.float16, device=cuda),
                    scratch=torch.zeros(need, dtype=torch.uint8, device=cuda))

    def step(b, stream=None):
        for pos0, n in ((0, M), (50, M), (100, M)):
            qk_lib.qk_norm_rope_kv_append_q4(q, k, v, gq, gk, EPS, f, b["q"], *b["cache"], n, H, Hkv, D, D, pos0, L,
                                             layout=qk_lib.QK_ROPE_HALF, stream=stream)
        qk_lib.qk_gqa_attention_q4(b["q"], *b["cache"], b["many"], M, H, Hkv, D, 100, L, SCALE, NONE, 0, scratch=b["scratch"],
                                   stream=stream)
        qk_lib.qk_norm_rope_kv_append_q4(q[:1], k[:1], v[:1], gq, gk, EPS, f, b["q"][:1], *b["cache"], 1, H, Hkv, D, D, 150, L,
                                         layout=qk_lib.QK_ROPE_HALF, stream=stream)
        qk_lib.qk_gqa_attention_q4(b["q"][:1], *b["cache"], b["one"], 1, H, Hkv, D, 150, L, SCALE, 128, 4, stream=stream)

    want, side, replay = buffers(), buffers(), buffers()
    step(want)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    step(side, stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        step(replay)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for got in (side, replay):
        for n in ("q", "many", "one"):
            assert torch.equal(got[n], want[n]), n
        for a, b in zip(got["cache"], want["cache"]):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
