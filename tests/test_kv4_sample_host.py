"""Head norms with the append, the 4-bit cache, attention over it and sampling, as
far as the host decides: refusals before any pointer is looked at, scratch sizes
and the binding's buffer checks (no GPU needed)."""
import math

import pytest

A16, A8 = 0x10000, 0x10008  # fake, never-dereferenced addresses
AT = [0x20000000 + (i << 26) for i in range(12)]
NO_DEVICE = (-4, -6, -8)  # past the host checks: CUDA error, unsupported device, inaccessible pointer
NULL, ALIGN, SHAPE = -1, -2, -3


@pytest.mark.parametrize("q4", [False, True])
def test_append_refusals(qk_lib, q4):
    f = qk_lib.lib().qk_norm_rope_kv_append_q4 if q4 else qk_lib.lib().qk_norm_rope_kv_append
    caches = ("k4", "kd", "v4", "vd") if q4 else ("kc", "vc")
    names = ("q", "k", "v", "gq", "gk", "fr", "qo") + caches
    at = dict(zip(names, AT))

    def call(M=2, H=4, Hkv=2, D=64, n=64, p=0, L=16, layout=0, mag=1.0, eps=1e-6, **ptr):
        b = dict(at, **ptr)
        return f(b["q"], b["k"], b["v"], b["gq"], b["gk"], eps, b["fr"], b["qo"], *(b[c] for c in caches), M, H, Hkv, D, n, p,
                 L, layout, mag, None)
    for bad in (dict(M=-1), dict(M=1 << 31), dict(H=0), dict(Hkv=0), dict(H=1025), dict(Hkv=1025), dict(D=60), dict(D=520),
                dict(D=544), dict(D=0), dict(n=66), dict(n=-2), dict(n=3), dict(p=-1), dict(p=15), dict(p=(1 << 63) - 1),
                dict(L=0), dict(L=1 << 31), dict(layout=2), dict(mag=math.inf), dict(mag=math.nan), dict(eps=-1e-6),
                dict(eps=math.inf), dict(eps=math.nan)):
        assert call(**bad) == SHAPE, bad
    assert (call(D=40, n=40) == SHAPE) == q4
    for name in names:
        if name not in ("gq", "gk"):
            assert call(**{name: None}) == NULL, name
        assert call(**{name: A8}) == ALIGN, name
    assert call(M=0, q=None) == 0
    assert call(p=14) in NO_DEVICE and call(gq=None, gk=None) in NO_DEVICE and call(n=0, fr=None) in NO_DEVICE
    assert call(eps=0.0, D=512) in NO_DEVICE


def test_dequant_kv_refusals(qk_lib):
    f = qk_lib.lib().qk_dequant_kv_q4

    def call(q=AT[0], d=AT[1], o=AT[2], Hkv=2, D=64, p=0, M=4, L=16):
        return f(q, d, o, Hkv, D, p, M, L, None)
    for bad in (dict(M=-1), dict(Hkv=0), dict(Hkv=1025), dict(D=48), dict(D=0), dict(D=544), dict(p=-1), dict(p=13), dict(L=0),
                dict(L=1 << 31), dict(p=(1 << 63) - 1)):
        assert call(**bad) == SHAPE, bad
    for name in ("q", "d", "o"):
        assert call(**{name: None}) == NULL and call(**{name: A8}) == ALIGN, name
    assert call(M=0, q=None) == 0 and call(p=12) in NO_DEVICE and call(D=512) in NO_DEVICE


def test_attention_q4_refusals(qk_lib):
    f = qk_lib.lib().qk_gqa_attention_q4
    at = dict(zip(("q", "k4", "kd", "v4", "vd", "o", "s"), AT))

    def call(M=2, H=8, Hkv=2, D=128, p=0, L=64, scale=0.1, w=4, sinks=1, **ptr):
        b = dict(at, **ptr)
        return f(b["q"], b["k4"], b["kd"], b["v4"], b["vd"], b["o"], M, H, Hkv, D, p, L, scale, w, sinks, b["s"], None)
    for bad in (dict(M=-1), dict(H=7), dict(H=32), dict(H=0), dict(Hkv=0), dict(D=64), dict(p=-1), dict(p=63), dict(L=1 << 31),
                dict(w=-1), dict(sinks=-1), dict(H=2048, Hkv=1024), dict(p=(1 << 30) - 2, L=(1 << 31) - 1),
                dict(p=(1 << 63) - 1), dict(scale=math.inf), dict(scale=math.nan)):
        assert call(**bad) == SHAPE, bad
    for name in ("q", "k4", "kd", "v4", "vd", "o"):
        assert call(**{name: None}) == NULL and call(**{name: A8}) == ALIGN, name
    assert call(s=None) in NO_DEVICE and call(s=A8) in NO_DEVICE  # few tokens of a short cache use no scratch
    assert call(M=40, s=None) == NULL and call(M=40, s=A8) == ALIGN
    assert call(M=1, p=65535, L=65536, w=65536, s=None) == NULL
    assert call(M=0, q=None) == 0
    assert call(w=1 << 62, sinks=1 << 62) in NO_DEVICE and call(scale=0.0) in NO_DEVICE


def test_attention_q4_scratch(qk_lib):
    f = qk_lib.qk_gqa_attention_q4_scratch_bytes
    none = 1 << 62
    assert f(0, 8, 2, 128, 5, none) == 0 and f(1, 8, 2, 128, 1000, none) == 0 and f(8, 8, 2, 128, 1000, none) == 0
    # more than 32 columns: 512 bytes for each key/value head and position that some query sees
    assert f(9, 8, 2, 128, 1000, none) == 512 * 2 * 1009
    assert f(9, 8, 2, 128, 1000, 100) == 512 * 2 * (100 + 8)
    assert f(9, 8, 2, 128, 1000, 100, 30) == 512 * 2 * (100 + 8 + 30)
    assert f(9, 8, 2, 128, 1000, 100, none) == 512 * 2 * 1009
    assert f(9, 8, 2, 128, 1000, 0) == 0 and f(9, 8, 2, 128, 1000, 0, 7) == 512 * 2 * 7
    # few: from 65536 positions of all heads on, partial results of the CTAs
    assert f(1, 8, 2, 128, 32766, none) == 0
    assert 0 < f(1, 8, 2, 128, 32767, none) <= 1 << 20 and 0 < f(8, 8, 2, 128, 10 ** 6, none) <= 4 << 20
    assert f(1, 8, 2, 128, 10 ** 6, 4096, 4) == 0
    # never more than the fp16 rows of all positions, which the binding relies on
    for M in (1, 3, 7, 8, 9, 40, 700):
        for H, Hkv in ((1, 1), (8, 8), (24, 8), (32, 4), (1024, 1024), (1024, 128), (40, 40)):
            for pos0 in (0, 1, 63, 64, 500, 9000, 65536, 10 ** 6, (1 << 30) - 701):
                for window, sinks in ((none, 0), (0, 5), (1, 0), (700, 3), (10 ** 5, 0)):
                    assert 0 <= f(M, H, Hkv, 128, pos0, window, sinks) <= 512 * Hkv * (pos0 + M)
    for bad in ((-1, 8, 2, 128, 0, 1), (1, 8, 3, 128, 0, 1), (1, 8, 2, 64, 0, 1), (1, 8, 2, 128, -1, 1), (1, 8, 2, 128, 0, -1),
                (1, 8, 2, 128, 0, 1, -1), (1, 8, 2, 128, 1 << 30, 1), (1, 18, 2, 128, 0, 1)):
        with pytest.raises(ValueError):
            f(*bad)


def test_sample_refusals(qk_lib):
    f = qk_lib.lib().qk_sample

    def call(x=AT[0], u=AT[1], t=AT[2], lp=AT[3], n=AT[4], M=3, V=10, T=1.0, k=0, p=1.0, mp=0.0):
        return f(x, u, t, lp, n, M, V, T, k, p, mp, None)
    for bad in (dict(M=-1), dict(M=1 << 31), dict(V=0), dict(V=-4), dict(V=(1 << 19) + 1), dict(T=-1.0), dict(T=1e-7),
                dict(T=2e6), dict(T=math.nan), dict(T=math.inf), dict(k=-1), dict(p=-0.1), dict(p=1.5), dict(p=math.nan),
                dict(mp=-0.1), dict(mp=1.1), dict(mp=1e-13), dict(mp=math.nan)):
        assert call(**bad) == SHAPE, bad
    for name in ("x", "u", "t"):
        assert call(**{name: None}) == NULL, name
    for name in ("x", "u", "t", "lp", "n"):
        assert call(**{name: A8}) == ALIGN, name
    assert call(M=0, x=None) == 0
    assert call(lp=None, n=None) in NO_DEVICE and call(V=1 << 19, k=1 << 30, T=0.0) in NO_DEVICE
    assert call(T=1e6, p=0.0, mp=1e-12) in NO_DEVICE


def test_binding_checks_tensor_buffers(qk_lib):
    torch = pytest.importorskip("torch")
    M, L = 3, 16
    q, kv, fr = torch.zeros(M, 4, 128), torch.zeros(M, 2, 128), torch.zeros(64, dtype=torch.float64)
    g, qo = torch.ones(128, dtype=torch.float16), torch.zeros(M, 4, 128, dtype=torch.float16)
    c4, dm = torch.zeros(2, L, 64, dtype=torch.uint8), torch.zeros(2, L, 4, 2, dtype=torch.float16)
    c16 = torch.zeros(2, L, 128, dtype=torch.float16)
    x, u, tok, lp = torch.zeros(M, 10), torch.zeros(M), torch.zeros(M, dtype=torch.int32), torch.zeros(M)

    def append(q=q, k=kv, v=kv, gq=g, gk=g, fr=fr, qo=qo, kc=c16, vc=c16):
        qk_lib.qk_norm_rope_kv_append(q, k, v, gq, gk, 1e-6, fr, qo, kc, vc, M, 4, 2, 128, 128, 0, L, stream=0)

    def append4(k4=c4, kd=dm, v4=c4, vd=dm):
        qk_lib.qk_norm_rope_kv_append_q4(q, kv, kv, g, g, 1e-6, fr, qo, k4, kd, v4, vd, M, 4, 2, 128, 128, 0, L, stream=0)

    def attn(q=qo, k4=c4, kd=dm, out=qo, M=M, scratch=None):
        qk_lib.qk_gqa_attention_q4(q, k4, kd, c4, dm, out, M, 4, 2, 128, 0, L, 0.1, 9, scratch=scratch, stream=0)

    def sample(x=x, u=u, tok=tok, lp=lp, kept=tok):
        qk_lib.qk_sample(x, u, tok, lp, kept, M, 10, stream=0)
    bad = [
        lambda: append(gq=g.float()), lambda: append(gk=g[:127]), lambda: append(fr=fr.float()), lambda: append(q=q.half()),
        lambda: append(qo=q), lambda: append(kc=c16[:, :15]), lambda: append(vc=c16.transpose(0, 1)),
        lambda: append(k=kv[:2]), lambda: append4(k4=c4.view(torch.int8)), lambda: append4(kd=dm.float()),
        lambda: append4(v4=c4[:, :, :63]), lambda: append4(vd=dm[:1]),
        lambda: qk_lib.qk_dequant_kv_q4(c4, dm, c16[:, :4], 2, 128, 0, 4, L, stream=0),
        lambda: qk_lib.qk_dequant_kv_q4(c4, dm.float(), c16, 2, 128, 0, 4, L, stream=0),
        lambda: qk_lib.qk_dequant_kv_q4(c4[:1], dm, c16, 2, 128, 0, 4, L, stream=0),
        lambda: attn(out=q), lambda: attn(q=qo[:2]), lambda: attn(kd=dm[:, :15]), lambda: attn(k4=c16),
        lambda: sample(x=x.half()), lambda: sample(x=x[:, :9]), lambda: sample(u=u[:2]), lambda: sample(u=u.double()),
        lambda: sample(tok=tok.long()), lambda: sample(lp=lp.double()), lambda: sample(kept=lp),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    # 33 columns: a scratch that is too small, or of another type
    many = torch.zeros(15, 4, 128, dtype=torch.float16), torch.zeros(17, 4, 128, dtype=torch.float16)
    for scratch in (torch.zeros(64, dtype=torch.uint8), torch.zeros(1 << 16)):
        with pytest.raises(ValueError):
            qk_lib.qk_gqa_attention_q4(many[1], c4, dm, c4, dm, many[1], 17, 4, 2, 128, 0, 17, 0.1, 99, scratch=scratch, stream=0)
    for call in (append, append4, attn, sample):  # host tensors pass the binding; the library refuses them
        with pytest.raises(qk_lib.QKError) as e:
            call()
        assert e.value.status in NO_DEVICE + (-7,)
