"""The operators around the linears, as far as the host decides: refusals before
any pointer is looked at, the binding's buffer checks, and the rotation
frequencies (no GPU needed)."""
import math

import numpy as np
import pytest

A16, A8 = 0x10000, 0x10008  # fake, never-dereferenced addresses
B16, C16, D16, E16 = 0x20000000, 0x30000000, 0x40000000, 0x50000000
NO_DEVICE = (-4, -6, -8)  # past the host checks: CUDA error, unsupported device, inaccessible pointer
NULL, ALIGN, SHAPE = -1, -2, -3


def test_add_rmsnorm_refusals(qk_lib):
    f = qk_lib.lib().qk_add_rmsnorm
    assert f(A16, 2, B16, C16, 1e-5, None, D16, 4, 64, None) == SHAPE             # unknown residual type
    assert f(A16, 0, B16, C16, 1e-5, None, D16, 4, 60, None) == SHAPE             # K % 8
    assert f(A16, 0, B16, C16, 1e-5, None, D16, 4, 0, None) == SHAPE
    assert f(A16, 0, B16, C16, 1e-5, None, D16, -1, 64, None) == SHAPE
    assert f(A16, 0, B16, C16, 1e-5, None, D16, 1 << 31, 64, None) == SHAPE
    assert f(A16, 0, B16, C16, 1e-5, None, D16, (1 << 31) - 1, (1 << 31) - 8, None) == SHAPE  # byte extent
    assert f(A16, 0, B16, C16, -1e-5, None, D16, 4, 64, None) == SHAPE
    assert f(A16, 0, B16, C16, float("nan"), None, D16, 4, 64, None) == SHAPE
    assert f(None, 0, B16, C16, 1e-5, None, D16, 4, 64, None) == NULL
    assert f(A16, 0, B16, None, 1e-5, None, D16, 4, 64, None) == NULL
    assert f(A16, 0, B16, C16, 1e-5, None, None, 4, 64, None) == NULL
    assert f(A16, 0, B16 + 8, C16, 1e-5, None, D16, 4, 64, None) == ALIGN
    assert f(A16, 0, B16, C16, 1e-5, A8, D16, 4, 64, None) == ALIGN
    assert f(None, 0, None, None, 1e-5, None, None, 0, 64, None) == 0
    assert f(A16, 0, None, C16, 1e-5, None, D16, 4, 64, None) in NO_DEVICE        # delta and residual_out are optional
    q = qk_lib.lib().qk_add_rmsnorm_q8
    assert q(A16, 1, B16, C16, 1e-5, None, D16, E16, 4, 40, None) == SHAPE        # K % 32
    assert q(A16, 1, B16, C16, 1e-5, None, D16, None, 4, 64, None) == NULL
    assert q(A16, 1, B16, C16, 1e-5, None, None, E16, 4, 64, None) == NULL
    assert q(A16, 1, B16, C16, 1e-5, None, D16, E16 + 4, 4, 64, None) == ALIGN
    assert q(A16, 1, B16, C16, 1e-5, A16, D16, E16, 4, 64, None) in NO_DEVICE


def test_matmul_batch_q8_refusals(qk_lib):
    L = qk_lib.lib()
    D = qk_lib.qk_matmul_q8_desc
    f = L.qk_matmul_batch_q8

    def one(*a):
        return f((D * 1)(D(*a)), 1, None)
    assert f(None, 0, None) == 0 and f(None, 1, None) == NULL and f(None, -1, None) == SHAPE
    assert one(0, A16, None, B16, C16, D16, 2, 8, 256) == SHAPE     # several tokens
    assert one(0, A16, None, B16, C16, D16, 1, 8, 300) == SHAPE
    assert one(7, A16, None, B16, C16, D16, 1, 8, 256) == SHAPE
    assert one(1, A16, A16, B16, C16, D16, 1, 8, 256) == SHAPE      # gate/up is Q4_K
    assert one(0, A16, None, B16, None, D16, 1, 8, 256) == NULL
    assert one(0, A16, None, None, C16, D16, 1, 8, 256) == NULL
    assert one(0, A16, None, B16, C16 + 4, D16, 1, 8, 256) == ALIGN
    assert one(0, A16, None, B16 + 4, C16, D16, 1, 8, 256) == ALIGN
    assert one(0, None, None, None, None, None, 0, 8, 256) == 0
    assert one(0, A16, None, B16, C16, D16, 1, 8, 256) in NO_DEVICE


def test_rope_refusals(qk_lib):
    f = qk_lib.lib().qk_rope_kv_append

    def call(q=A16, k=B16, v=C16, fr=D16, qo=E16, kc=E16 + (1 << 26), vc=E16 + (2 << 26), M=2, H=4, Hkv=2, D=64, n=64,
             p=0, L=16, layout=0, mag=1.0):
        return f(q, k, v, fr, qo, kc, vc, M, H, Hkv, D, n, p, L, layout, mag, None)
    for bad in (dict(M=-1), dict(H=0), dict(Hkv=0), dict(H=1025), dict(D=60), dict(D=520), dict(D=0), dict(n=66),
                dict(n=-2), dict(n=3), dict(p=-1), dict(p=15), dict(L=0), dict(L=1 << 31), dict(layout=2),
                dict(mag=math.inf), dict(mag=math.nan)):
        assert call(**bad) == SHAPE, bad
    for name in ("q", "k", "v", "fr", "qo", "kc", "vc"):
        assert call(**{name: None}) == NULL, name
        assert call(**{name: A8}) == ALIGN, name
    assert call(M=0, q=None) == 0
    assert call(p=14) in NO_DEVICE
    assert call(n=0, fr=None) in NO_DEVICE


def test_attention_window_refusals(qk_lib):
    f = qk_lib.lib().qk_gqa_attention_window

    def call(q=A16, k=B16, v=C16, o=D16, M=2, H=8, Hkv=2, D=128, p=0, L=16, w=4, s=1):
        return f(q, k, v, o, M, H, Hkv, D, p, L, 0.1, w, s, None)
    for bad in (dict(M=-1), dict(H=7), dict(H=32), dict(D=64), dict(p=-1), dict(p=15), dict(L=1 << 31), dict(w=-1),
                dict(s=-1), dict(H=2048, Hkv=1024)):
        assert call(**bad) == SHAPE, bad
    for name in ("q", "k", "v", "o"):
        assert call(**{name: None}) == NULL, name
        assert call(**{name: A8}) == ALIGN, name
    assert call(M=0, q=None) == 0
    assert call(w=0, s=0) in NO_DEVICE
    assert call(w=1 << 62, s=1 << 62) in NO_DEVICE


def test_logprobs_refusals(qk_lib):
    f = qk_lib.lib().qk_logprobs

    def call(x=A16, t=B16, lp=C16, e=D16, n=2, ids=E16, tl=E16 + (1 << 26), M=3, V=10):
        return f(x, t, lp, e, n, ids, tl, M, V, None)
    for bad in (dict(M=-1), dict(V=0), dict(V=-4), dict(n=-1), dict(n=33, V=100), dict(n=11), dict(V=1 << 31),
                dict(M=1 << 31), dict(M=(1 << 31) - 1, V=(1 << 31) - 1)):
        assert call(**bad) == SHAPE, bad
    for name in ("x", "t", "lp", "ids", "tl"):
        assert call(**{name: None}) == NULL, name
        assert call(**{name: A8}) == ALIGN, name
    assert call(M=0, x=None) == 0
    assert call(e=None) in NO_DEVICE and call(t=None, lp=None) in NO_DEVICE
    assert call(n=0, ids=None, tl=None) in NO_DEVICE


def test_binding_checks_tensor_buffers(qk_lib):
    torch = pytest.importorskip("torch")
    M, K = 3, 64
    r16, r32 = torch.zeros(M, K, dtype=torch.float16), torch.zeros(M, K)
    g, x = torch.zeros(K, dtype=torch.float16), torch.zeros(M, K, dtype=torch.float16)
    xq, xd = torch.zeros(M, K, dtype=torch.int8), torch.zeros(M, K // 32)
    q, c = torch.zeros(M, 4, 128), torch.zeros(2, 16, 128, dtype=torch.float16)
    kv, fr, qo = torch.zeros(M, 2, 128), torch.zeros(64, dtype=torch.float64), torch.zeros(M, 4, 128, dtype=torch.float16)
    lg, tok, lp = torch.zeros(M, 10), torch.zeros(M, dtype=torch.int32), torch.zeros(M)
    ids, tl = torch.zeros(M, 2, dtype=torch.int32), torch.zeros(M, 2)

    def rope(q=q, k=kv, v=kv, fr=fr, qo=qo, kc=c, vc=c):
        qk_lib.qk_rope_kv_append(q, k, v, fr, qo, kc, vc, M, 4, 2, 128, 128, 0, 16, stream=0)

    def logp(lg=lg, tok=tok, lp=lp, ids=ids, tl=tl):
        qk_lib.qk_logprobs(lg, tok, lp, lp.clone(), 2, ids, tl, M, 10, stream=0)
    bad = [
        lambda: qk_lib.qk_add_rmsnorm(r16, r16, g, 1e-5, None, x, M, K, stream=0),           # delta not fp32
        lambda: qk_lib.qk_add_rmsnorm(r16, r32, g, 1e-5, r32, x, M, K, stream=0),            # another residual type
        lambda: qk_lib.qk_add_rmsnorm(r32, r32, g[:60], 1e-5, None, x, M, K, stream=0),
        lambda: qk_lib.qk_add_rmsnorm(A16, B16, C16, 1e-5, None, D16, M, K, stream=0),       # type of a raw address
        lambda: qk_lib.qk_add_rmsnorm(r32.t(), r32, g, 1e-5, None, x, M, K, stream=0),       # not contiguous
        lambda: qk_lib.qk_add_rmsnorm_q8(r32, r32, g, 1e-5, None, x, xd, M, K, stream=0),    # xq not int8
        lambda: qk_lib.qk_add_rmsnorm_q8(r32, r32, g, 1e-5, None, xq, xd[:2], M, K, stream=0),
        lambda: rope(fr=fr.float()), lambda: rope(fr=fr[:63]), lambda: rope(q=q.half()), lambda: rope(kc=c[:, :15]),
        lambda: logp(tok=tok.long()), lambda: logp(ids=ids[:2]), lambda: logp(lg=lg.half()), lambda: logp(lp=lp[1:]),
        lambda: qk_lib.qk_gqa_attention_window(qo, c, c, q, M, 4, 2, 128, 0, 16, 0.1, 4, stream=0),  # out not fp16
        lambda: qk_lib.qk_matmul_batch_q8([dict(qtype="q4k", blocks=torch.zeros(8 * 144, dtype=torch.uint8), x_q8=xq,
                                                x_d=xd, y=torch.zeros(1, 8), M=1, N=8, K=256)], stream=0),
        lambda: qk_lib.qk_rope_inv_freq(8, 1e4, freq_factors=[1.0, 2.0]),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
    for call in (rope, logp, lambda: qk_lib.qk_add_rmsnorm(r16, r32, g, 1e-5, r16, x, M, K, stream=0)):
        with pytest.raises(qk_lib.QKError) as e:  # host tensors pass the binding; the library refuses them
            call()
        assert e.value.status in NO_DEVICE


@pytest.mark.parametrize("n_rot", [2, 46, 128, 512])
def test_inv_freq(qk_lib, n_rot):
    """Against the formulas in numpy, within a few steps of fp64 (pow is not
    correctly rounded: 2^-50 relative)."""
    i = np.arange(n_rot // 2)
    base = 500000.0 ** (-2.0 * i / n_rot)
    tol = dict(rtol=2.0 ** -50, atol=0)
    f = qk_lib.qk_rope_inv_freq
    np.testing.assert_allclose(f(n_rot, 5e5), base, **tol)
    np.testing.assert_allclose(f(n_rot, 5e5, qk_lib.QK_ROPE_SCALE_LINEAR, 4.0), base / 4, **tol)
    ff = 1 + i.astype(np.float32) / 7
    np.testing.assert_allclose(f(n_rot, 5e5, freq_factors=ff), base / ff.astype(np.float64), **tol)
    for low, high, L in ((1.0, 4.0, 8192), (1.0, 32.0, 4096)):
        g = np.clip((L * base / (2 * np.pi) - low) / (high - low), 0, 1)
        got = np.array(f(n_rot, 5e5, qk_lib.QK_ROPE_SCALE_BANDED, 32.0, low, high, L))
        np.testing.assert_allclose(got, (1 - g) * base / 32 + g * base, rtol=2.0 ** -44, atol=0)
        assert got[0] == base[0]  # many turns: kept
        if n_rot >= 46:
            np.testing.assert_allclose(got[-1], base[-1] / 32, **tol)  # few: slowed


def test_inv_freq_refusals(qk_lib):
    f = qk_lib.qk_rope_inv_freq
    B = qk_lib.QK_ROPE_SCALE_BANDED
    for a in ((3, 1e4), (-2, 1e4), (514, 1e4), (8, 0.0), (8, math.inf), (8, 1e4, 5), (8, 1e4, 1, 0.0),
              (8, 1e4, B, 8.0, 4.0, 4.0), (8, 1e4, B, 8.0, -1.0, 4.0), (8, 1e4, B, 8.0, 1.0, 4.0, 0)):
        with pytest.raises(qk_lib.QKError) as e:
            f(*a)
        assert e.value.status == SHAPE, a
    with pytest.raises(qk_lib.QKError):
        f(4, 1e4, freq_factors=[1.0, 0.0])
    assert f(0, 1e4) == []
