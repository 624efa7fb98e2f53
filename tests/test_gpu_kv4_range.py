"""Groups of a 4-bit cache near fp16's largest numbers: each is NaN or d q + m is a finite fp16
number for every q, and attention reads the same row the same way whatever the number of tokens."""
import math

import numpy as np
import pytest

from tests import kv4_reference as ref4
from tests import synth

pytestmark = pytest.mark.gpu

SCALE = 1 / math.sqrt(128)

# (least, greatest, value of the rest) of a group, and whether it is stored as NaN
GROUPS = [
    (60000.0, 66000.0, 61000.0, True),      # a value beyond fp16, d = 400
    (65000.0, 65520.0, 65100.0, True),      # the first number that rounds to infinity
    (-66000.0, -60000.0, -61000.0, True),
    (-65520.0, -65519.0, -65519.5, True),
    (1984.0, 65504.0, 30000.0, False),      # d rounds up to 4236: 15 d + m would be 65524
    (1000.0, 65504.0, 2000.0, False),
    (65472.0, 65519.996, 65500.0, False),   # rounds to 65504
    (-65519.996, -65472.0, -65500.0, False),
    (64000.0, 65519.0, 64100.0, False),
    (32760.0, 65504.0, 40000.0, False),
    (-30000.0, 35400.0, 5.0, False),        # 65400 apart
    (-65504.0, 100.0, 0.0, True),           # 65604 apart: 15 d is no finite fp16 number
    (0.0, 65504.0, 1.0, True),              # d is 4368
    (65504.0, 65504.0, 65504.0, False),
    (-65504.0, -65504.0, -65504.0, False),
]


def _pack(x):
    """The header's rule in fp32: (bytes, dm, NaN groups) of rows [..., D]."""
    b = x.astype(np.float32).reshape(*x.shape[:-1], -1, 32)
    lo, hi = b.min(-1), b.max(-1)
    with np.errstate(over="ignore", invalid="ignore"):
        m = lo.astype(np.float16)
        m32 = m.astype(np.float32)
        d = (np.maximum(hi - m32, np.float32(0)) / np.float32(15)).astype(np.float16)
        nan = ~((lo > -65520) & (hi < 65520) & (d.astype(np.float32) <= 4366))
        top = (15 * d.astype(np.float64) + m32).astype(np.float32)  # 15 d + m with one rounding
    down = ~nan & (top >= 65520)
    d = np.where(down, (d.view(np.uint16) - 1).astype(np.uint16).view(np.float16), d)
    m, d = np.where(nan, np.float16(np.nan), m), np.where(nan, np.float16(np.nan), d)
    with np.errstate(divide="ignore", invalid="ignore"):
        d32 = d.astype(np.float32)[..., None]
        q = np.where(d32 > 0, np.clip(np.rint((b - m.astype(np.float32)[..., None]) / d32), 0, 15), 0).astype(np.uint8)
    q = q.reshape(x.shape)
    return q[..., 0::2] | (q[..., 1::2] << 4), np.stack([d, m], -1), nan, down


def _rows(Dh):
    """A row for each of GROUPS [n][Dh] in its first and last group, and ordinary values between."""
    rng = synth.rng_for(601, Dh)
    x = rng.standard_normal((len(GROUPS), Dh)).astype(np.float32)
    for i, (lo, hi, rest, _) in enumerate(GROUPS):
        for at in (0, Dh - 32):
            x[i, at: at + 32] = rest
            x[i, at + 3], x[i, at + 29] = lo, hi
    return x


def _dev(a, cuda):
    import torch
    a = np.ascontiguousarray(a)
    return (torch.from_numpy(a.view(np.uint16)).to(cuda).view(torch.float16) if a.dtype == np.float16
            else torch.from_numpy(a).to(cuda))


def _append(qk, cuda, k, v, half, n_rot):
    import torch
    M, Hkv, Dh = v.shape
    z = lambda t, *s: torch.zeros(*s, dtype=t, device=cuda)  # noqa: E731
    f = _dev(np.zeros(max(1, n_rot // 2)), cuda)  # no turn
    c = [z(torch.uint8, Hkv, M, Dh // 2), z(torch.float16, Hkv, M, Dh // 32, 2), z(torch.uint8, Hkv, M, Dh // 2),
         z(torch.float16, Hkv, M, Dh // 32, 2)]
    qk.qk_norm_rope_kv_append_q4(z(torch.float32, M, Hkv, Dh), _dev(k, cuda), _dev(v, cuda), None, None, 1e-6, f,
                                 z(torch.float16, M, Hkv, Dh), *c, M, Hkv, Hkv, Dh, n_rot, 0, M,
                                 layout=qk.QK_ROPE_HALF if half else qk.QK_ROPE_INTERLEAVED)
    return c


@pytest.mark.parametrize("Dh,half,whole", [(128, True, True), (128, False, True), (64, True, True), (96, False, False),
                                           (320, True, False), (32, False, True)])
def test_groups_at_the_limits(qk_lib, cuda, Dh, half, whole):
    """To the bit by the header's rule (a value in two lanes' and in one lane's reach, k as it is
    after a turn by 0), NaN where it says so, and otherwise finite as fp16 at every level."""
    x = np.stack([_rows(Dh), _rows(Dh)[::-1]], 1)  # [row][head][Dh]
    k4, kd, v4, vd = _append(qk_lib, cuda, x, x, half, Dh if whole else 0)
    q4, dm, nan, down = _pack(x.transpose(1, 0, 2))
    assert down.any() and [bool(n) for n in nan[0, :, 0]] == [g[3] for g in GROUPS]
    for got4, gotd in ((k4, kd), (v4, vd)):
        got4, gotd = got4.cpu().numpy(), gotd.cpu().numpy()
        assert np.array_equal(np.isnan(gotd), np.isnan(dm))
        fine = ~nan
        assert np.array_equal(gotd[fine].view(np.uint16), dm[fine].view(np.uint16))
        b = lambda a: a.reshape(*nan.shape, 16)  # noqa: E731
        assert np.array_equal(b(got4)[fine], b(q4)[fine])
        for level in (0, 15):  # of the ends
            with np.errstate(over="ignore", invalid="ignore"):
                end = (level * gotd[..., 0].astype(np.float64) + gotd[..., 1]).astype(np.float16)
            assert np.isfinite(end[fine]).all()
        # half a step, or, where d was rounded (up to half a step of fp16, a whole one down),
        # 15 of those for the greatest value; and the roundings of m and of the value itself
        d = gotd[..., 0].astype(np.float64)[..., None]
        got = ref4.values(got4, gotd).astype(np.float64).reshape(*nan.shape, 32)
        want = x.transpose(1, 0, 2).astype(np.float64).reshape(*nan.shape, 32)
        off = np.abs(got - want)[fine]
        most = np.abs(want).max(-1)[..., None][fine]
        assert (off <= (d / 2 + 15 * d * 2.0 ** -10)[fine] + 2 * most * 2.0 ** -11 + 2.0 ** -23).all()


@pytest.mark.parametrize("row", [i for i, g in enumerate(GROUPS) if not g[3]])
def test_few_tokens_and_chunks_agree_on_such_a_row(qk_lib, cuda, row):
    """A value row at the limits: 1, 3 and 40 queries get what 64 bits say of d q + m.  Three
    roundings of 2^-11 of the largest |v| (weights, d (q - 8) or fp16(d q + m), the output), and
    2^-12 of fp32's."""
    import torch
    rng = synth.rng_for(602, row)
    H, Hkv, L = 4, 2, 200
    x = rng.standard_normal((L, Hkv, 128)).astype(np.float32)
    k = rng.standard_normal((L, Hkv, 128)).astype(np.float32)
    x[5] = _rows(128)[row]
    cache = _append(qk_lib, cuda, k, x, True, 128)
    host = [t.cpu().numpy() for t in cache]
    kk, vv = ref4.exact(*host[:2]), ref4.exact(*host[2:])
    assert np.isfinite(ref4.values(*host[2:])).all()
    for M in (1, 3, 40):
        q = (1.5 * rng.standard_normal((M, H, 128))).astype(np.float16)
        need = qk_lib.qk_gqa_attention_q4_scratch_bytes(M, H, Hkv, 128, L - M, 10 ** 9)
        out = torch.empty(M, H, 128, dtype=torch.float16, device=cuda)
        qk_lib.qk_gqa_attention_q4(_dev(q, cuda), *cache, out, M, H, Hkv, 128, L - M, L, SCALE, 10 ** 9, 0,
                                   scratch=torch.empty(need, dtype=torch.uint8, device=cuda) if need else None)
        got = out.cpu().numpy().astype(np.float64)
        want = ref4.attention(q, kk, vv, H, Hkv, L - M, 10 ** 9, 0, SCALE)
        assert np.isfinite(got).all()
        assert (np.abs(got - want) <= np.abs(vv).max() * (3 * 2.0 ** -11 + 2.0 ** -12)).all()
