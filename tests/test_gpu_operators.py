"""The operators around the linears (residual + RMSNorm, products from int8 x,
rotary positions with the cache append, windowed attention, log probabilities)
against plain numpy in 64 bits, through the binding.

Tolerances are sums of the roundings on the way: half a step of the output's
type (fp16 2^-11 relative, 2^-25 below the normal range) and the fp32
arithmetic's share, derived beside each test.
"""
import math

import numpy as np
import pytest

import oracle
from tests import synth

pytestmark = pytest.mark.gpu

EPS = 1e-5
QT = {"q4k": oracle.Q4K, "q6k": oracle.Q6K}


def _dev(a, cuda):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).to(cuda)


def _host(t):
    return t.cpu().numpy()


def _within(got, ref, tol, what):
    bad = ~(np.abs(got.astype(np.float64) - ref) <= tol)
    assert not bad.any(), "%s: %d of %d off, worst %.3e (allowed %.3e)" % (
        what, bad.sum(), bad.size, np.nanmax(np.abs(got - ref)), np.max(tol))


# ---------------------------------------------------------------------------
# Residual addition + RMSNorm
# ---------------------------------------------------------------------------
def _norm_inputs(seed, M, K, f32):
    rng = synth.rng_for(seed, M * 100003 + K)
    res = rng.standard_normal((M, K)) * np.where(rng.random(K) < 0.02, 20.0, 1.0)
    res = res.astype(np.float32 if f32 else np.float16)
    delta = (0.3 * rng.standard_normal((M, K))).astype(np.float32)
    gamma = (1 + 0.1 * rng.standard_normal(K)).astype(np.float16)
    return res, delta, gamma


def _norm_reference(res, delta, gamma):
    """(fp32 h, 64-bit xhat): h is one fp32 addition, exact to the bit."""
    h = res.astype(np.float32) + (delta if delta is not None else np.float32(0))
    hd = h.astype(np.float64)
    return h, hd / np.sqrt((hd ** 2).mean(1, keepdims=True) + EPS) * gamma.astype(np.float64)


NORM_SHAPES = [(1, 8), (1, 4096), (3, 248), (2, 264), (7, 2560), (300, 1024), (5, 8192), (2, 8200), (3, 16416),
               (1, 32768), (1, 70000)]


@pytest.mark.parametrize("M,K", NORM_SHAPES)
@pytest.mark.parametrize("f32", [False, True])
def test_add_rmsnorm(qk_lib, cuda, M, K, f32):
    """xhat: the fp16 rounding, plus fp32 arithmetic: a thread adds at most
    K / 256 + 8 squares one by one and the tree 13 more, each 2^-24, halved by
    the root; its reciprocal and two products 4 x 2^-24."""
    import torch
    res, delta, gamma = _norm_inputs(201, M, K, f32)
    g = _dev(gamma.view(np.uint16), cuda).view(torch.float16)
    for with_delta in (True, False):
        h, ref = _norm_reference(res, delta if with_delta else None, gamma)
        tol = np.abs(ref) * (2.0 ** -11 + (K / 512 + 15) * 2.0 ** -24) + 2.0 ** -25
        r = _dev(res, cuda)
        out, x = torch.full_like(r, math.nan), torch.full((M, K), math.nan, dtype=torch.float16, device=cuda)
        d = _dev(delta, cuda) if with_delta else None
        qk_lib.qk_add_rmsnorm(r, d, g, EPS, out, x, M, K)
        assert np.array_equal(_host(out), h.astype(res.dtype))
        assert np.array_equal(_host(r), res)
        _within(_host(x), ref, tol, "xhat")
        # without the residual's output, and in place: the same bits
        y = torch.full_like(x, math.nan)
        qk_lib.qk_add_rmsnorm(r, d, g, EPS, None, y, M, K)
        assert torch.equal(x, y)
        y.fill_(math.nan)
        qk_lib.qk_add_rmsnorm(r, d, g, EPS, r, y, M, K)
        assert torch.equal(x, y) and torch.equal(r, out)


@pytest.mark.parametrize("M,K", [(1, 32), (1, 4096), (5, 2592), (333, 2560), (2, 8224), (3, 16416), (1, 70400)])
@pytest.mark.parametrize("f32", [False, True])
def test_add_rmsnorm_q8(qk_lib, cuda, M, K, f32):
    """int8 out: to the bit the quantization of qk_add_rmsnorm's fp16 output."""
    import torch
    res, delta, gamma = _norm_inputs(202, M, K, f32)
    delta[0, :32] = -res[0, :32].astype(np.float32)  # a block of zeros: d = 0, q = 0
    r, d, g = _dev(res, cuda), _dev(delta, cuda), _dev(gamma.view(np.uint16), cuda).view(torch.float16)
    out, x = torch.empty_like(r), torch.empty(M, K, dtype=torch.float16, device=cuda)
    qk_lib.qk_add_rmsnorm(r, d, g, EPS, out, x, M, K)
    xq = torch.full((M, K), 99, dtype=torch.int8, device=cuda)
    xd = torch.full((M, K // 32), math.nan, device=cuda)
    qk_lib.qk_add_rmsnorm_q8(r, d, g, EPS, r, xq, xd, M, K)
    q, s = oracle.quantize_q8(_host(x))
    assert np.array_equal(_host(xd), s.reshape(M, -1)) and np.array_equal(_host(xq), q.reshape(M, K))
    assert torch.equal(r, out)
    if M * K > 32:
        assert s.reshape(-1)[0] == 0 and np.abs(q).max() == 127


def test_add_rmsnorm_zero_rows_and_alias(qk_lib, cuda):
    """A row of zeros has xhat 0 (eps > 0); overlapping buffers are refused."""
    import torch
    z = torch.zeros(4, 64, device=cuda)
    g = torch.ones(64, dtype=torch.float16, device=cuda)
    x = torch.full((4, 64), math.nan, dtype=torch.float16, device=cuda)
    qk_lib.qk_add_rmsnorm(z, None, g, EPS, None, x, 4, 64)
    assert (x == 0).all()
    buf = torch.zeros(8, 64, device=cuda)
    for bad in (dict(res=buf[:4], out=buf[1:5], d=None), dict(res=buf[:4], out=buf[:4], d=buf[2:6]),
                dict(res=buf[:4], out=buf[4:], d=buf[4:])):
        with pytest.raises(qk_lib.QKError) as e:
            qk_lib.qk_add_rmsnorm(bad["res"], bad["d"], g, EPS, bad["out"], x, 4, 64)
        assert e.value.status == -7
    with pytest.raises(qk_lib.QKError) as e:
        qk_lib.qk_add_rmsnorm(buf[:4], None, g, EPS, None, buf.view(torch.float16).view(-1)[:256], 4, 64)
    assert e.value.status == -7
    # the residual as its own second addend is no overlap problem: nothing is written over it
    qk_lib.qk_add_rmsnorm(z, z, g, EPS, None, x, 4, 64)
    assert (x == 0).all()


# ---------------------------------------------------------------------------
# Products from int8 x
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("qtype", ["q4k", "q6k"])
@pytest.mark.parametrize("N,K", [(200, 2560), (64, 8192), (1, 256), (33, 2304), (130, 1024), (4096, 4096)])
def test_matmul_q8(qk_lib, cuda, qtype, N, K):
    """To the bit qk_matmul_q8x_* on the fp16 x that the values come from, and
    within that path's fp32 margin of the 64-bit product (test_gpu_q8.py)."""
    import torch
    rng = synth.rng_for(203, N * K)
    W, x = synth.weights(rng, qtype, N, K), synth.activations(rng, 1, K)
    q, s = oracle.quantize_q8(x)
    y0, y1 = (torch.full((1, N), math.nan, device=cuda) for _ in range(2))
    w = _dev(W, cuda)
    (qk_lib.qk_matmul_q8x_q4k if qtype == "q4k" else qk_lib.qk_matmul_q8x_q6k)(w, _dev(x.view(np.uint16), cuda), y0, 1,
                                                                             N, K)
    qk_lib.qk_matmul_batch_q8([dict(qtype=qtype, blocks=w, x_q8=_dev(q.reshape(1, K), cuda),
                                    x_d=_dev(s.reshape(1, -1), cuda), y=y1, M=1, N=N, K=K)])
    qk_lib.qk_get_device_status()
    assert torch.equal(y0, y1)
    ref = oracle.q8_matmul(QT[qtype], W, x, N, K)
    assert np.abs(_host(y1) - ref).max() <= 2e-3 * np.sqrt((ref ** 2).mean())


@pytest.mark.parametrize("qtype,N,K", [("q4k", 40, 11008), ("q4k", 2500, 9472), ("q4k", 17, 12032), ("q6k", 40, 14336),
                                       ("q6k", 2500, 10240), ("q6k", 33, 22528)])
def test_matmul_rows_in_unequal_chunks(qk_lib, cuda, qtype, N, K):
    """Rows that go out in chunks of which the last is smaller: int8 x as above, and
    fp16 x of one token and of four within the fp16 path's bar."""
    test_matmul_q8(qk_lib, cuda, qtype, N, K)
    import torch
    rng = synth.rng_for(226, N * K)
    W, x = synth.weights(rng, qtype, N, K), synth.activations(rng, 4, K)
    ref = oracle.matmul(QT[qtype], W, x, N, K)
    w, f = _dev(W, cuda), qk_lib.qk_matmul_q4k if qtype == "q4k" else qk_lib.qk_matmul_q6k
    for M in (1, 4):
        y = torch.full((M, N), math.nan, device=cuda)
        f(w, _dev(x[:M].view(np.uint16), cuda), y, M, N, K)
        qk_lib.qk_get_device_status()
        assert np.abs(_host(y) - ref[:M]).max() <= 1e-2 * np.sqrt((ref[:M] ** 2).mean())
    if qtype == "q4k":
        y = torch.full((1, N), math.nan, dtype=torch.float16, device=cuda)
        qk_lib.qk_gateup_swiglu_q4k(w, w, _dev(x[:1].view(np.uint16), cuda), y, 1, N, K)
        ref = oracle.gateup_swiglu(W, W, x[:1], N, K)
        assert np.abs(_host(y).astype(np.float64) - ref).max() <= 1e-2 * np.sqrt((ref ** 2).mean())


def test_matmul_q8_extreme_values(qk_lib, cuda):
    """Any int8, -128 among them, and any finite scale."""
    import torch
    rng = synth.rng_for(204, 0)
    N, K = 48, 512
    for qtype in ("q4k", "q6k"):
        W = synth.weights(rng, qtype, N, K)
        q = rng.choice(np.array([-128, -127, 127, 0], np.int8), size=(1, K))
        s = np.exp(rng.uniform(-20, 20, (1, K // 32))).astype(np.float32)
        y = torch.full((1, N), math.nan, device=cuda)
        qk_lib.qk_matmul_batch_q8([dict(qtype=qtype, blocks=_dev(W, cuda), x_q8=_dev(q, cuda), x_d=_dev(s, cuda), y=y,
                                        M=1, N=N, K=K)])
        w = oracle.dequant(QT[qtype], W).astype(np.float64).reshape(N, K)
        xv = q.astype(np.float64) * np.repeat(s.astype(np.float64), 32, 1)
        # every product and sum of the at most K / 16 scaled sums in fp32
        _within(_host(y), xv @ w.T, (np.abs(xv) @ np.abs(w).T) * (K / 16 + 8) * 2.0 ** -24, qtype)


def test_matmul_q8_batch_and_gateup(qk_lib, cuda):
    """Ten problems (more than a launch holds), fused gate/up among them, one
    empty: the same bits as one by one; overlaps are refused."""
    import torch
    rng = synth.rng_for(205, 0)
    K = 768
    x = synth.activations(rng, 1, K)
    q, s = oracle.quantize_q8(x)
    xq, xd, xf = _dev(q.reshape(1, K), cuda), _dev(s.reshape(1, -1), cuda), _dev(x.view(np.uint16), cuda)
    ps, rs = [], []
    for i in range(10):
        qt, N = ("q4k", "q6k")[i % 2 if i != 8 else 0], 16 * i + 3 if i != 5 else 0
        up = _dev(synth.q4k_weights(rng, N, K), cuda) if i == 8 else None
        w = _dev(synth.weights(rng, qt, max(N, 1), K), cuda)
        y = [torch.full((1, max(N, 1)), -7.0, device=cuda, dtype=torch.float16 if up is not None else torch.float32)
             for _ in range(2)]
        ps.append(dict(qtype=qt, blocks=w, up_blocks=up, x_q8=xq, x_d=xd, y=y[0], M=1, N=N, K=K))
        rs.append(dict(qtype=qt, blocks=w, up_blocks=up, x_f16=xf, y=y[1], M=1, N=N, K=K))
    qk_lib.qk_matmul_batch_q8(ps)
    for r in rs:
        qk_lib.qk_matmul_batch_q8x([r])
    qk_lib.qk_get_device_status()
    for p, r in zip(ps, rs):
        assert torch.equal(p["y"], r["y"])
    shared = torch.zeros(64, device=cuda)
    for bad in (dict(y=xd.view(-1)[:3]), dict(x_d=shared[:24], y=shared[8:11]), dict(y=xq.view(torch.float32)[:, :3])):
        with pytest.raises((qk_lib.QKError, ValueError)) as e:
            qk_lib.qk_matmul_batch_q8([dict(ps[0], **bad)])
        assert isinstance(e.value, qk_lib.QKError) and e.value.status == -7
    K = 2048 * 256  # more than the decode GEMV can stage
    with pytest.raises(qk_lib.QKError) as e:
        qk_lib.qk_matmul_batch_q8([dict(qtype="q4k", blocks=torch.zeros(2048 * 144, dtype=torch.uint8, device=cuda),
                                        x_q8=torch.zeros(1, K, dtype=torch.int8, device=cuda),
                                        x_d=torch.zeros(1, K // 32, device=cuda), y=torch.zeros(1, 1, device=cuda),
                                        M=1, N=1, K=K)])
    assert e.value.status == -3


# ---------------------------------------------------------------------------
# Rotary positions and the cache append
# ---------------------------------------------------------------------------
def _rotate(x, angle, n_rot, half, mag):
    """64-bit rotation of x [M][heads][D] by angle [M][n_rot / 2]."""
    y = x.astype(np.float64).copy()
    a = y[..., : n_rot // 2] if half else y[..., 0:n_rot:2]
    b = y[..., n_rot // 2: n_rot] if half else y[..., 1:n_rot:2]
    c, s = mag * np.cos(angle)[:, None], mag * np.sin(angle)[:, None]
    ra, rb = a * c - b * s, b * c + a * s
    if half:
        y[..., : n_rot // 2], y[..., n_rot // 2: n_rot] = ra, rb
    else:
        y[..., 0:n_rot:2], y[..., 1:n_rot:2] = ra, rb
    return y


def _rope_case(qk, cuda, M, H, Hkv, D, n_rot, pos0, L, half, mag, seed=206):
    import torch
    rng = synth.rng_for(seed, M * 7 + D + n_rot)
    q, k, v = (rng.standard_normal((M, h, D)).astype(np.float32) for h in (H, Hkv, Hkv))
    f = np.array(qk.qk_rope_inv_freq(n_rot, 5e5, qk.QK_ROPE_SCALE_BANDED, 8.0), np.float64)
    kc0, vc0 = (rng.standard_normal((Hkv, L, D)).astype(np.float16) for _ in range(2))
    kc, vc = _dev(kc0, cuda), _dev(vc0, cuda)
    qo = torch.full((M, H, D), math.nan, dtype=torch.float16, device=cuda)
    qk.qk_rope_kv_append(_dev(q, cuda), _dev(k, cuda), _dev(v, cuda), _dev(f, cuda) if n_rot else None, qo, kc, vc, M, H,
                         Hkv, D, n_rot, pos0, L, layout=qk.QK_ROPE_HALF if half else qk.QK_ROPE_INTERLEAVED,
                         magnitude=mag)
    angle = np.arange(pos0, pos0 + M, dtype=np.float64)[:, None] * f[None]
    kc1, vc1 = _host(kc), _host(vc)

    def check(got, x, what):
        # sine and cosine within 2^-21 (the fraction of a turn in fp32 2^-25 of a turn, the functions
        # 2^-23), two products and a sum of 2^-24 each, then fp16
        ref = _rotate(x, angle, n_rot, half, mag)
        size = np.abs(x).max(-1, keepdims=True) * 2 * max(1.0, abs(mag))
        _within(got, ref, np.abs(ref) * 2.0 ** -11 + size * 2.0 ** -20.5 + 2.0 ** -25, what)
    check(_host(qo), q, "q")
    check(kc1[:, pos0: pos0 + M].transpose(1, 0, 2), k, "k")
    assert np.array_equal(vc1[:, pos0: pos0 + M].transpose(1, 0, 2), v.astype(np.float16))
    if n_rot < D:
        assert np.array_equal(_host(qo)[..., n_rot:], q[..., n_rot:].astype(np.float16))
    for got, was in ((kc1, kc0), (vc1, vc0)):  # the other rows are untouched
        assert np.array_equal(got[:, :pos0], was[:, :pos0]) and np.array_equal(got[:, pos0 + M:], was[:, pos0 + M:])


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("D,n_rot", [(128, 128), (128, 64), (80, 46), (64, 2), (64, 0), (8, 8), (256, 256), (512, 512),
                                     (96, 30), (72, 72), (40, 4)])
@pytest.mark.parametrize("M", [1, 9])
def test_rope_layouts(qk_lib, cuda, M, D, n_rot, half):
    _rope_case(qk_lib, cuda, M, 6, 2, D, n_rot, 1000, 1000 + M + 3, half, 1.0)


@pytest.mark.parametrize("M,H,Hkv,pos0", [(1, 24, 8, 0), (2, 1, 1, 5), (63, 8, 8, 0), (64, 24, 8, 1), (65, 32, 4, 100),
                                          (200, 24, 8, 31), (1, 1024, 1024, 3), (3, 5, 3, 0)])
def test_rope_sizes(qk_lib, cuda, M, H, Hkv, pos0):
    D = 128 if H < 1000 else 64
    _rope_case(qk_lib, cuda, M, H, Hkv, D, D, pos0, pos0 + M, M % 2 == 0, 1.1)


@pytest.mark.parametrize("pos0", [131071, 2 ** 21 + 12345])
def test_rope_far_positions(qk_lib, cuda, pos0):
    """Angles of 10^5 and 10^6 radians keep their fraction of a turn."""
    _rope_case(qk_lib, cuda, 2, 3, 1, 16, 16, pos0, pos0 + 2, False, 1.0)


# ---------------------------------------------------------------------------
# Attention with a window and sinks
# ---------------------------------------------------------------------------
D = 128
SCALE = 1 / math.sqrt(D)


def _attn_inputs(seed, M, H, Hkv, pos0, L, window, sinks):
    """Inputs whose rows that no query sees are NaN or infinite."""
    rng = synth.rng_for(seed, M * 1000 + pos0 + window)
    q = (1.5 * rng.standard_normal((M, H, D))).astype(np.float16)
    k, v = (rng.standard_normal((Hkv, L, D)).astype(np.float16) for _ in range(2))
    j = np.arange(L)
    unseen = (j >= pos0 + M) | ((j <= pos0 - window) & (j >= sinks)) | (window == 0) & (j >= sinks)
    k[:, unseen] = np.where(j[unseen] % 2, np.nan, np.inf)[None, :, None]
    v[:, unseen] = np.where(j[unseen] % 3, np.nan, -np.inf)[None, :, None]
    return q, k, v


def _attn_reference(q, k, v, H, Hkv, pos0, window, sinks, rows=None):
    M = q.shape[0]
    rows = np.arange(M) if rows is None else rows
    out = np.zeros((len(rows), H, D))
    for n, i in enumerate(rows):
        p = pos0 + i
        j = np.arange(p + 1)
        j = j[(j > p - window) | (j < sinks)]
        if not len(j):
            continue
        for g in range(Hkv):
            G = H // Hkv
            z = q[i, g * G:(g + 1) * G].astype(np.float64) @ k[g, j].astype(np.float64).T * SCALE
            e = np.exp(z - z.max(1, keepdims=True))
            out[n, g * G:(g + 1) * G] = e / e.sum(1, keepdims=True) @ v[g, j].astype(np.float64)
    return out


def _attn(qk, cuda, q, k, v, H, Hkv, pos0, window, sinks):
    import torch
    out = torch.full(q.shape, math.nan, dtype=torch.float16, device=cuda)
    dq, dk, dv = (_dev(a.view(np.uint16), cuda) for a in (q, k, v))
    qk.qk_gqa_attention_window(dq, dk, dv, out, q.shape[0], H, Hkv, D, pos0, k.shape[1], SCALE, window, sinks)
    qk.qk_get_device_status()
    return _host(out)


def _attn_check(got, ref, v, what):
    """fp16 weights 2^-11 relative each (below 2^-24 of the largest they flush:
    2^-25 each, 2^13 positions at most), the output's rounding 2^-11, scores in
    fp32 (2^-12 of a weight in all): against the largest finite |v|."""
    vmax = np.abs(v[np.isfinite(v)].astype(np.float64)).max()
    _within(got, ref, vmax * (2.0 ** -10 + 2.0 ** -12 + 2.0 ** -12), what)


@pytest.mark.parametrize("pos0,window,sinks", [
    (0, 1, 0), (0, 0, 1), (0, 5, 3), (63, 64, 0), (64, 64, 0), (64, 64, 1), (700, 1, 0), (700, 0, 2), (700, 0, 100),
    (700, 1, 64), (700, 65, 65), (700, 635, 66), (700, 634, 66), (700, 636, 66), (700, 10 ** 9, 0), (700, 3, 701),
    (5000, 4096, 4), (5000, 1000, 300), (4095, 4095, 0), (9000, 300, 1)])
def test_window_decode(qk_lib, cuda, pos0, window, sinks):
    q, k, v = _attn_inputs(207, 1, 24, 8, pos0, pos0 + 5, window, sinks)
    got = _attn(qk_lib, cuda, q, k, v, 24, 8, pos0, window, sinks)
    _attn_check(got, _attn_reference(q, k, v, 24, 8, pos0, window, sinks), v, "decode")


@pytest.mark.parametrize("H,Hkv", [(8, 8), (32, 4), (6, 2), (4, 1), (7, 1), (24, 8)])
def test_window_group_sizes(qk_lib, cuda, H, Hkv):
    for M, pos0, window, sinks in ((1, 900, 333, 9), (1, 77, 500, 0), (130, 200, 90, 5), (3, 640, 257, 130)):
        q, k, v = _attn_inputs(208, M, H, Hkv, pos0, pos0 + M, window, sinks)
        got = _attn(qk_lib, cuda, q, k, v, H, Hkv, pos0, window, sinks)
        _attn_check(got, _attn_reference(q, k, v, H, Hkv, pos0, window, sinks), v, "H%d/%d M%d" % (H, Hkv, M))


@pytest.mark.parametrize("M,pos0,window,sinks", [
    (2, 0, 1, 0), (2, 0, 1, 1), (2, 50, 0, 1), (17, 0, 4, 2), (100, 0, 10 ** 6, 0), (128, 0, 64, 0), (129, 0, 128, 0),
    (257, 0, 1, 0), (257, 0, 1, 1), (300, 0, 127, 128), (300, 0, 128, 129), (300, 0, 0, 200), (300, 37, 0, 5),
    (33, 777, 200, 4), (130, 1000, 129, 127), (130, 1000, 64, 300), (260, 500, 300, 600), (515, 300, 250, 17),
    (200, 3, 50, 10 ** 7)])
def test_window_prefill(qk_lib, cuda, M, pos0, window, sinks):
    H, Hkv = 6, 2
    q, k, v = _attn_inputs(209, M, H, Hkv, pos0, pos0 + M + 3, window, sinks)
    got = _attn(qk_lib, cuda, q, k, v, H, Hkv, pos0, window, sinks)
    _attn_check(got, _attn_reference(q, k, v, H, Hkv, pos0, window, sinks), v, "prefill")


@pytest.mark.parametrize("M,pos0,window,sinks,H,Hkv", [
    (2, 6000, 4096, 4, 24, 8), (5, 3000, 10 ** 6, 0, 8, 8), (43, 2500, 2048, 300, 6, 2), (85, 1500, 1200, 16, 24, 8),
    (9, 4000, 0, 4000, 4, 1), (130, 3000, 2900, 7, 7, 1), (16, 2000, 1, 1500, 32, 4), (300, 100, 150, 100, 8, 8),
    (257, 0, 10 ** 6, 0, 2, 2), (24, 1023, 1024, 1, 16, 2)])
def test_window_short_chunks(qk_lib, cuda, M, pos0, window, sinks, H, Hkv):
    """Few queries after a long context: a cluster shares their key tiles.  The
    joining is fp32, a few steps of 2^-24: the same tolerance."""
    q, k, v = _attn_inputs(220, M, H, Hkv, pos0, pos0 + M + 1, window, sinks)
    got = _attn(qk_lib, cuda, q, k, v, H, Hkv, pos0, window, sinks)
    _attn_check(got, _attn_reference(q, k, v, H, Hkv, pos0, window, sinks), v, "short chunk")


def test_window_is_deterministic(qk_lib, cuda):
    for M, pos0, window, sinks in ((1, 5000, 3000, 4), (7, 5000, 3000, 4), (300, 50, 100, 4), (1300, 0, 700, 0)):
        q, k, v = _attn_inputs(221, M, 24, 8, pos0, pos0 + M, window, sinks)
        a, b = (_attn(qk_lib, cuda, q, k, v, 24, 8, pos0, window, sinks) for _ in range(2))
        assert np.array_equal(a, b)


@pytest.mark.parametrize("M,pos0,window,sinks,H,Hkv", [
    (900, 30, 60, 3, 40, 40), (1150, 0, 33, 0, 40, 40), (150, 7, 50, 4, 40, 20), (300, 400, 20, 200, 8, 8)])
def test_window_pairs_and_single_tiles(qk_lib, cuda, M, pos0, window, sinks, H, Hkv):
    """More query tiles than SMs take, few more, or an odd number of them."""
    q, k, v = _attn_inputs(224, M, H, Hkv, pos0, pos0 + M, window, sinks)
    rows = np.unique(np.concatenate([[0, 63, 64, 127, 128, M - 1], synth.rng_for(225, M).choice(M, 60)]))
    got = _attn(qk_lib, cuda, q, k, v, H, Hkv, pos0, window, sinks)
    assert np.isfinite(got).all()
    _attn_check(got[rows], _attn_reference(q, k, v, H, Hkv, pos0, window, sinks, rows), v, "pairs and tiles")


def test_window_large_prefill_sampled(qk_lib, cuda):
    H, Hkv, M, pos0, window, sinks = 24, 8, 1500, 700, 512, 4
    q, k, v = _attn_inputs(210, M, H, Hkv, pos0, pos0 + M, window, sinks)
    rows = np.unique(np.concatenate([[0, 1, 127, 128, 255, 256, M - 1], synth.rng_for(211, 0).choice(M, 40)]))
    got = _attn(qk_lib, cuda, q, k, v, H, Hkv, pos0, window, sinks)
    assert np.isfinite(got).all()
    _attn_check(got[rows], _attn_reference(q, k, v, H, Hkv, pos0, window, sinks, rows), v, "large prefill")


def test_window_full_equals_causal(qk_lib, cuda):
    """A window over everything is qk_gqa_attention, rounded to fp16 (within the
    two kernels' tolerance), decode and prefill."""
    import torch
    for M, pos0 in ((1, 1500), (200, 31)):
        q, k, v = _attn_inputs(212, M, 24, 8, pos0, pos0 + M, 10 ** 6, 0)
        got = _attn(qk_lib, cuda, q, k, v, 24, 8, pos0, pos0 + M, 0)
        out = torch.empty(q.shape, device=cuda)
        qk_lib.qk_gqa_attention(*(_dev(a.view(np.uint16), cuda) for a in (q, k, v)), out, M, 24, 8, D, pos0,
                                k.shape[1], SCALE)
        _attn_check(got, _host(out).astype(np.float64), v, "causal")


def test_window_empty_rows_are_zero(qk_lib, cuda):
    for M in (1, 40):
        q, k, v = _attn_inputs(213, M, 6, 2, 50, 50 + M, 0, 0)
        assert (_attn(qk_lib, cuda, q, k, v, 6, 2, 50, 0, 0) == 0).all()


@pytest.mark.parametrize("M,pos0,window,sinks,H,Hkv", [
    (130, 0, 60, 0, 6, 2), (130, 200, 90, 5, 24, 8), (300, 400, 150, 0, 4, 4), (9, 3000, 2500, 4, 8, 2),
    (40, 5, 10 ** 6, 0, 7, 1), (70, 10, 0, 40, 6, 2), (1, 500, 200, 3, 6, 2)])
def test_window_values_reach_only_who_sees_them(qk_lib, cuda, M, pos0, window, sinks, H, Hkv):
    """Non-finite keys and values at positions that some queries of a tile see and
    others do not: the others' outputs are what they would be without them."""
    q, k, v = _attn_inputs(227, M, H, Hkv, pos0, pos0 + M, window, sinks)
    p1 = pos0 + M - 1
    for n, (j, what, dims) in enumerate([(p1, np.nan, slice(None)), (pos0 + M // 2, np.inf, slice(0, 5)),
                                         (max(0, pos0 - window + 1), -np.inf, slice(60, None)),
                                         (pos0 + M // 3, np.nan, slice(7, 8))]):
        v[:, j, dims] = what
        if n == 0:
            k[:, j, 3] = np.nan
    got = _attn(qk_lib, cuda, q, k, v, H, Hkv, pos0, window, sinks).astype(np.float64)
    with np.errstate(invalid="ignore", over="ignore"):
        ref = _attn_reference(q, k, v, H, Hkv, pos0, window, sinks)
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    inf = np.isinf(ref)
    assert np.array_equal(got[inf], ref[inf]) and not np.isinf(got[~inf]).any()
    fine = np.isfinite(ref)
    assert fine.any() or M == 1
    _attn_check(got[fine], ref[fine], v, "beside non-finite values")


@pytest.mark.parametrize("scale_sign", [1.0, -1.0])
def test_window_large_scores(qk_lib, cuda, scale_sign):
    """Scores of hundreds (one position takes all the weight), either sign of scale."""
    import torch
    for M, pos0, window, sinks in ((1, 600, 200, 3), (140, 300, 100, 3)):
        q, k, v = _attn_inputs(214, M, 6, 2, pos0, pos0 + M, window, sinks)
        q = (q * np.float16(20)).astype(np.float16)
        out = torch.full(q.shape, math.nan, dtype=torch.float16, device=cuda)
        qk_lib.qk_gqa_attention_window(*(_dev(a.view(np.uint16), cuda) for a in (q, k, v)), out, M, 6, 2, D, pos0,
                                       k.shape[1], SCALE * scale_sign, window, sinks)
        ref = _attn_reference((q * np.float16(scale_sign)).astype(np.float16), k, v, 6, 2, pos0, window, sinks)
        # scores s reach 500: fp32 sums leave 2^-24 * 128 * |q||k| scale < 2^-9 of a score unit
        vmax = np.abs(v[np.isfinite(v)].astype(np.float64)).max()
        _within(_host(out), ref, vmax * 2.0 ** -8, "large scores")


def test_long_cache_offsets(qk_lib, cuda):
    """Caches of more than 2^32 bytes and 2^31 elements: the append writes and the
    attention reads the last head's far rows."""
    import torch
    Hkv, H, L = 3, 6, 6_000_000
    kc = torch.full((Hkv, L, D), math.nan, dtype=torch.float16, device=cuda)
    vc = torch.full((Hkv, L, D), math.nan, dtype=torch.float16, device=cuda)
    rng = synth.rng_for(215, 0)
    n, pos0, window, sinks = 150, L - 150, 100, 5
    k, v = (rng.standard_normal((n, Hkv, D)).astype(np.float32) for _ in range(2))
    f = _dev(np.zeros(D // 2), cuda)  # no turn: the rows are the rounded inputs
    q32 = _dev(rng.standard_normal((n, H, D)).astype(np.float32), cuda)
    q16 = torch.empty(n, H, D, dtype=torch.float16, device=cuda)
    for p in (0, pos0):
        qk_lib.qk_rope_kv_append(q32, _dev(k, cuda), _dev(v, cuda), f, q16, kc, vc, n, H, Hkv, D, D, p, L)
    assert torch.isnan(kc[:, n:pos0]).all() and not torch.isnan(kc[:, pos0:]).any()
    k16, v16 = k.astype(np.float16).transpose(1, 0, 2), v.astype(np.float16).transpose(1, 0, 2)
    # the same attention in a short cache: sinks, then the last rows, window alike
    short_k, short_v = (np.concatenate([a[:, :sinks], a], 1) for a in (k16, v16))
    for M in (1, 50):
        out = torch.full((M, H, D), math.nan, dtype=torch.float16, device=cuda)
        qk_lib.qk_gqa_attention_window(q16[n - M:].contiguous(), kc, vc, out, M, H, Hkv, D, L - M, L, SCALE, window,
                                       sinks)
        qk_lib.qk_get_device_status()
        q = _host(q16)[n - M:]
        ref = _attn_reference(q, short_k, short_v, H, Hkv, sinks + n - M, window, sinks)
        _attn_check(_host(out), ref, v16, "long cache M=%d" % M)
    del kc, vc
    torch.cuda.empty_cache()


# ---------------------------------------------------------------------------
# Log probabilities
# ---------------------------------------------------------------------------
def _logprob_reference(x, n):
    xd = x.astype(np.float64)
    with np.errstate(all="ignore"):
        m = xd.max(1, keepdims=True)
        e = np.exp(xd - m)
        S = e.sum(1, keepdims=True)
        lp = (xd - m) - np.log(S)  # relative to m: m + log S would lose log S beside a large m
        z = np.where(e > 0, xd - m, 0.0)
        ent = np.log(S[:, 0]) - (e * z).sum(1) / S[:, 0]
    # larger first, NaN below -inf, equal ones in token order
    rank = np.lexsort((np.broadcast_to(np.arange(x.shape[1]), x.shape), np.where(np.isnan(x), 0, -xd),
                       np.isnan(x).astype(int)), axis=1)
    return lp, ent, rank[:, :n]


def _logprobs(qk, cuda, x, tok, n):
    import torch
    M, V = x.shape
    lp, ent = (torch.full((M,), 7.0, device=cuda) for _ in range(2))
    ids = torch.full((M, max(n, 1)), -5, dtype=torch.int32, device=cuda)
    tl = torch.full((M, max(n, 1)), 7.0, device=cuda)
    qk.qk_logprobs(_dev(x, cuda), _dev(tok.astype(np.int32), cuda), lp, ent, n, ids if n else None, tl if n else None, M,
                   V)
    return _host(lp), _host(ent), _host(ids)[:, :n], _host(tl)[:, :n]


def _logprob_check(qk, cuda, x, tok, n, what):
    """log S: 2^-21 for the exponentials, (V / 512 + 32) 2^-24 for the sums; the
    entropy's T / S the same, times its size (at most log V); z 2^-23 of itself."""
    M, V = x.shape
    lp, ent, ids, tl = _logprobs(qk, cuda, x, tok, n)
    ref, rent, rids = _logprob_reference(x, n)
    tol = 2.0 ** -21 + (V / 512 + 32) * 2.0 ** -24
    r = ref[np.arange(M), tok]

    def near(got, want, t):
        same = (got == want) | (np.isnan(got) & np.isnan(want))
        with np.errstate(invalid="ignore"):
            ok = same | (np.abs(got - want) <= t)
        assert ok.all(), (what, got[~ok][:4], want[~ok][:4])
    near(lp, r, tol + 2.0 ** -22 * np.abs(np.where(np.isfinite(r), r, 0)))
    near(ent, rent, tol * (2 + 2 * math.log(V)))
    assert np.array_equal(ids, rids), what
    t = np.take_along_axis(ref, rids, 1)
    near(tl, t, tol + 2.0 ** -22 * np.abs(np.where(np.isfinite(t), t, 0)))


@pytest.mark.parametrize("M,V", [(1, 1), (3, 5), (2, 37), (4, 511), (4, 513), (1, 128256), (5, 50257), (300, 1003),
                                 (64, 32000), (2, 262147), (700, 33)])
@pytest.mark.parametrize("n", [0, 1, 5, 32])
def test_logprobs(qk_lib, cuda, M, V, n):
    rng = synth.rng_for(216, M * V + n)
    n = min(n, V)
    x = (3 * rng.standard_normal((M, V))).astype(np.float32)
    x[np.arange(M), rng.integers(0, V, M)] += rng.uniform(0, 30, M).astype(np.float32)
    tok = rng.integers(0, V, M)
    _logprob_check(qk_lib, cuda, x, tok, n, "random")
    x = np.round(x)  # many equal logits
    _logprob_check(qk_lib, cuda, x, tok, n, "ties")
    x[rng.random((M, V)) < 0.3] = -np.inf
    x[:, 0] = 1.0
    _logprob_check(qk_lib, cuda, x, tok, n, "banned")


@pytest.mark.parametrize("V", [64, 5000, 40003])
def test_logprobs_special_rows(qk_lib, cuda, V):
    rng = synth.rng_for(217, V)
    low = np.float32(-np.finfo(np.float32).max)
    x = (2 * rng.standard_normal((14, V))).astype(np.float32)
    x[1] = 0.0                                   # all equal: the first tokens
    x[2] = -np.inf                               # nothing left
    x[3, 1:] = -np.inf                           # one left, the first
    x[4, :-1] = -np.inf                          # one left, the last
    x[5] = low                                   # all the lowest value: uniform
    x[6] = np.where(rng.random(V) < 0.9, low, x[6])
    x[7, V // 2] = np.nan
    x[8, V // 3] = np.inf
    x[9] += np.float32(1e6)                      # far from zero
    x[10] = np.sort(x[10])                       # ascending: every logit is the new maximum
    x[11] = np.sort(x[11])[::-1]
    x[12, 7] = 90.0                              # sure
    x[13] = np.where(np.arange(V) % 2, np.float32(0.0), np.float32(-0.0))
    tok = rng.integers(0, V, 14)
    tok[3] = 0
    for n in (1, 20, 32):
        _logprob_check(qk_lib, cuda, x, tok, n, "special")


def test_logprobs_optional_outputs_and_padding(qk_lib, cuda):
    import torch
    rng = synth.rng_for(218, 0)
    x = rng.standard_normal((4, 999)).astype(np.float32)
    tok = np.array([5, -1, 999, -2 ** 31], np.int64)
    lp, ent, ids, tl = _logprobs(qk_lib, cuda, x, tok, 3)
    assert np.isfinite(lp[0]) and np.isnan(lp[1:]).all() and np.isfinite(ent).all()
    dx = _dev(x, cuda)
    e2 = torch.empty(4, device=cuda)
    qk_lib.qk_logprobs(dx, None, None, e2, 0, None, None, 4, 999)
    i2, t2 = torch.empty(4, 3, dtype=torch.int32, device=cuda), torch.empty(4, 3, device=cuda)
    qk_lib.qk_logprobs(dx, None, None, None, 3, i2, t2, 4, 999)
    qk_lib.qk_logprobs(dx, None, None, None, 0, None, None, 4, 999)
    assert np.array_equal(_host(e2), ent) and np.array_equal(_host(i2), ids) and np.array_equal(_host(t2), tl)
    with pytest.raises(qk_lib.QKError) as e:
        qk_lib.qk_logprobs(dx, None, None, dx.view(-1)[:4], 0, None, None, 4, 999)
    assert e.value.status == -7


# ---------------------------------------------------------------------------
# A run of them: one decoder layer and the head, prompt then token
# ---------------------------------------------------------------------------
class _Layer:
    """A small decoder: hidden 1024, 8 / 2 heads of 128, FFN 1536, vocabulary 2000."""
    K, H, Hkv, FF, V, L = 1024, 8, 2, 1536, 2000, 400
    window, sinks, top = 64, 4, 8

    def __init__(self, qk, cuda):
        import torch
        self.qk, self.cuda, self.torch = qk, cuda, torch
        rng = synth.rng_for(219, 0)
        K, H, Hkv, FF, V = self.K, self.H, self.Hkv, self.FF, self.V
        self.shapes = dict(q=("q4k", H * D, K), k=("q4k", Hkv * D, K), v=("q6k", Hkv * D, K), o=("q4k", K, H * D),
                           gate=("q4k", FF, K), up=("q4k", FF, K), down=("q6k", K, FF), head=("q6k", V, K))
        self.packed = {n: synth.weights(rng, *s) for n, s in self.shapes.items()}
        self.w = {n: _dev(a, cuda) for n, a in self.packed.items()}
        self.wd = {n: oracle.dequant(QT[s[0]], self.packed[n]).astype(np.float64).reshape(s[1], s[2])
                   for n, s in self.shapes.items()}
        self.gamma = [(1 + 0.1 * rng.standard_normal(K)).astype(np.float16) for _ in range(3)]
        self.g = [_dev(a, cuda) for a in self.gamma]
        self.freq = qk.qk_rope_inv_freq(D, 5e5)
        self.f = _dev(np.array(self.freq), cuda)
        self.rng = rng
        self.kc, self.vc = (torch.full((Hkv, self.L, D), math.nan, dtype=torch.float16, device=cuda) for _ in range(2))

    def buffers(self, M):
        t = self.torch
        e16 = lambda *s: t.empty(*s, dtype=t.float16, device=self.cuda)  # noqa: E731
        e32 = lambda *s: t.empty(*s, device=self.cuda)  # noqa: E731
        K, H, Hkv, FF, V = self.K, self.H, self.Hkv, self.FF, self.V
        return dict(res=e32(M, K), x=e16(M, K), xq=t.empty(M, K, dtype=t.int8, device=self.cuda), xd=e32(M, K // 32),
                    q=e32(M, H * D), k=e32(M, Hkv * D), v=e32(M, Hkv * D), q16=e16(M, H, D), a=e16(M, H, D), o=e32(M, K),
                    ff=e16(M, FF), down=e32(M, K), logits=e32(M, V), tok=t.zeros(M, dtype=t.int32, device=self.cuda),
                    lp=e32(M), ent=e32(M), ids=t.empty(M, self.top, dtype=t.int32, device=self.cuda),
                    tl=e32(M, self.top))

    def step(self, b, M, pos0, int8, stream=None):
        """b["res"] holds the embeddings; enqueues the layer and the head."""
        qk, w, K, H, Hkv, FF, V = self.qk, self.w, self.K, self.H, self.Hkv, self.FF, self.V

        def mm(names, x, key, kk):
            qk.qk_matmul_batch([dict(qtype=self.shapes[n][0], blocks=w[n], x_f16=x, y=b[key.get(n, n)], M=M,
                                     N=self.shapes[n][1], K=kk) for n in names], stream=stream)
        if int8:
            qk.qk_add_rmsnorm_q8(b["res"], None, self.g[0], EPS, None, b["xq"], b["xd"], M, K, stream=stream)
            qk.qk_matmul_batch_q8([dict(qtype=self.shapes[n][0], blocks=w[n], x_q8=b["xq"], x_d=b["xd"], y=b[n], M=M,
                                        N=self.shapes[n][1], K=K) for n in "qkv"], stream=stream)
        else:
            qk.qk_add_rmsnorm(b["res"], None, self.g[0], EPS, None, b["x"], M, K, stream=stream)
            mm("qkv", b["x"], {}, K)
        qk.qk_rope_kv_append(b["q"], b["k"], b["v"], self.f, b["q16"], self.kc, self.vc, M, H, Hkv, D, D, pos0, self.L,
                             stream=stream)
        qk.qk_gqa_attention_window(b["q16"], self.kc, self.vc, b["a"], M, H, Hkv, D, pos0, self.L, SCALE, self.window,
                                   self.sinks, stream=stream)
        mm(["o"], b["a"], {}, H * D)
        if int8:
            qk.qk_add_rmsnorm_q8(b["res"], b["o"], self.g[1], EPS, b["res"], b["xq"], b["xd"], M, K, stream=stream)
            qk.qk_matmul_batch_q8([dict(qtype="q4k", blocks=w["gate"], up_blocks=w["up"], x_q8=b["xq"], x_d=b["xd"],
                                        y=b["ff"], M=M, N=FF, K=K)], stream=stream)
        else:
            qk.qk_add_rmsnorm(b["res"], b["o"], self.g[1], EPS, b["res"], b["x"], M, K, stream=stream)
            qk.qk_gateup_swiglu_q4k(w["gate"], w["up"], b["x"], b["ff"], M, FF, K, stream=stream)
        mm(["down"], b["ff"], {}, FF)
        qk.qk_add_rmsnorm(b["res"], b["down"], self.g[2], EPS, b["res"], b["x"], M, K, stream=stream)
        mm(["head"], b["x"], {"head": "logits"}, K)
        qk.qk_logprobs(b["logits"], b["tok"], b["lp"], b["ent"], self.top, b["ids"], b["tl"], M, V, stream=stream)

    def reference(self, emb, act=lambda x: x, quant=None):
        """The whole sequence in 64 bits: residual, logits [n][V].  act is applied to
        what the library holds in fp16, quant (default act) to the normalized
        activations that may be int8."""
        quant = quant or act
        n = emb.shape[0]
        wd, H, Hkv = self.wd, self.H, self.Hkv
        h = emb.astype(np.float64)
        norm = lambda a, g: a / np.sqrt((a ** 2).mean(1, keepdims=True) + EPS) * g.astype(np.float64)  # noqa: E731
        x = quant(norm(h, self.gamma[0]))
        q, k, v = ((x @ wd[m].T).reshape(n, -1, D) for m in "qkv")
        angle = np.arange(n)[:, None] * np.array(self.freq)[None]
        q, k, v = act(_rotate(q, angle, D, False, 1.0)), act(_rotate(k, angle, D, False, 1.0)), act(v)
        a = np.zeros((n, H, D))
        for i in range(n):
            j = np.arange(i + 1)
            j = j[(j > i - self.window) | (j < self.sinks)]
            for hh in range(H):
                z = k[j, hh * Hkv // H] @ q[i, hh] * SCALE
                e = np.exp(z - z.max())
                a[i, hh] = e / e.sum() @ v[j, hh * Hkv // H]
        h = h + act(a.reshape(n, -1)) @ wd["o"].T
        x = quant(norm(h, self.gamma[1]))
        g, u = x @ wd["gate"].T, x @ wd["up"].T
        h = h + act(g / (1 + np.exp(-g)) * u) @ wd["down"].T
        return h, act(norm(h, self.gamma[2])) @ wd["head"].T


@pytest.mark.parametrize("int8", [False, True])
def test_decoder_layer_prompt_and_tokens(qk_lib, cuda, int8):
    """A prompt of 150 tokens, then three tokens one by one (with int8 activations
    in the second run), against the layer in 64 bits.

    Bar, in the 2-norm of the residual's change and of the logits: what the
    roundings of the activations to fp16 (int8) alone do to the 64-bit layer
    (2e-3 of the logits; single logits move by 7e-2 of their rms, so the norm is
    compared), times 2 for the weights' and the softmax weights' roundings, which
    are of the same size, and times 4 for the three tokens, whose few rows vary."""
    layer = _Layer(qk_lib, cuda)
    n, M = 153, 150
    emb = layer.rng.standard_normal((n, layer.K)).astype(np.float32)

    def half(x):
        return x.astype(np.float16).astype(np.float64)

    def by_int8(x):
        q, d = oracle.quantize_q8(x.astype(np.float16))
        return (q.reshape(n, -1, 32) * d.reshape(n, -1, 1).astype(np.float64)).reshape(n, -1)
    ref = layer.reference(emb)
    rounded = {False: layer.reference(emb, half), True: layer.reference(emb, half, by_int8)}
    got = [[], []]
    for pos0, m in ((0, M), (M, 1), (M + 1, 1), (M + 2, 1)):
        b = layer.buffers(m)
        b["res"].copy_(_dev(emb[pos0:pos0 + m], cuda))
        layer.step(b, m, pos0, int8 and m == 1)
        qk_lib.qk_get_device_status()
        got[0].append(_host(b["res"]).astype(np.float64))
        got[1].append(_host(b["logits"]).astype(np.float64))
        lp, ent, ids = _logprob_reference(_host(b["logits"]), layer.top)
        assert np.array_equal(_host(b["ids"]), ids)
        assert np.abs(_host(b["ent"]) - ent).max() <= 1e-4
        assert np.abs(_host(b["lp"]) - lp[:, 0]).max() <= 1e-4
    for rows, times, q in ((slice(0, M), 2, False), (slice(M, n), 4, int8)):
        for what in (0, 1):
            base = emb[rows] if what == 0 else 0.0
            size = np.linalg.norm(ref[what][rows] - base)
            bar = times * np.linalg.norm(rounded[q][what] - ref[what]) / np.linalg.norm(
                ref[what] - (emb if what == 0 else 0.0))
            err = np.linalg.norm(np.concatenate(got[what])[rows] - ref[what][rows]) / size
            assert err <= bar, (what, rows, err, bar)
    assert layer.torch.isnan(layer.kc[:, n:]).all() and not layer.torch.isnan(layer.kc[:, :n]).any()


@pytest.mark.parametrize("int8", [False, True])
def test_decoder_step_in_a_graph_and_on_two_streams(qk_lib, cuda, int8):
    """A captured decode step, replayed on new inputs, and two steps on two
    streams at once give the bits of the same steps called one by one."""
    import torch
    layer = _Layer(qk_lib, cuda)
    M = 40
    b = layer.buffers(M)
    b["res"].copy_(_dev(layer.rng.standard_normal((M, layer.K)).astype(np.float32), cuda))
    layer.step(b, M, 0, False)
    embs = [_dev(layer.rng.standard_normal((1, layer.K)).astype(np.float32), cuda) for _ in range(3)]
    keys = ("res", "logits", "lp", "ent", "ids", "tl", "a")
    want = []
    for e in embs:
        b = layer.buffers(1)
        b["res"].copy_(e)
        layer.step(b, 1, M, int8)
        want.append({k: b[k].clone() for k in keys})
    b = layer.buffers(1)
    src = torch.empty_like(b["res"])
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        b["res"].copy_(src)
        layer.step(b, 1, M, int8)
    for e, w in zip(embs, want):
        src.copy_(e)
        graph.replay()
        torch.cuda.synchronize()
        for k in keys:
            assert torch.equal(b[k], w[k]), k
    # two streams, each with its own buffers and cache
    layers = [layer, _Layer(qk_lib, cuda)]
    layers[1].kc, layers[1].vc = layer.kc.clone(), layer.vc.clone()
    streams = [torch.cuda.Stream() for _ in range(2)]
    bs = [layer.buffers(1) for _ in range(2)]
    torch.cuda.synchronize()
    for rep in range(10):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                bs[i]["res"].copy_(embs[i])
                layers[i].step(bs[i], 1, M, int8)
    torch.cuda.synchronize()
    qk_lib.qk_get_device_status()
    for i in range(2):
        for k in keys:
            assert torch.equal(bs[i][k], want[i][k]), k
