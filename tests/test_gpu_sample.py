"""Sampling against the definition in 64 bits (numpy), through the binding.

Tokens and kept counts are whole numbers: they are equal to the definition's
wherever no border lies closer than 2^-30 of the sum to a decision (the kernel's
sums are within that: 8192 threads' shares rounded to 2^-45 each, five a thread,
and weights within 2^-36 of themselves).  Log probabilities are (x - max) / T less log1p of the
kept sum without its largest weight, both at most 0 in fp32: a difference and a
quotient of 2^-24 each, log1p within 2^-23, their sum 2^-24, less than 2^-22 in all;
the sum within 2^-30.
"""
import math

import numpy as np
import pytest

from tests import synth

pytestmark = pytest.mark.gpu

NEAR = 2.0 ** -30


def reference(x, u, T, k=0, p=1.0, mp=0.0):
    """(token, logprob, kept, distance of the nearest border) of one row."""
    T, p, mp = float(np.float32(T)), float(np.float32(p)), float(np.float32(mp))
    x = x.astype(np.float64)
    if np.isnan(x).any() or (x == np.inf).any() or (x == -np.inf).all():
        return -1, math.nan, 0, 1.0
    order = np.lexsort((np.arange(len(x)), -x))
    order = order[x[order] > -np.inf]
    if T == 0:
        return int(order[0]), 0.0, 1, 1.0
    w = np.exp((x[order] - x[order[0]]) / T)
    c = np.cumsum(w.astype(np.longdouble))
    near = []
    n = min(k, len(w)) if k else len(w)
    if p < 1:
        t = p * c[n - 1]
        n_p = int((c < t).sum()) + 1
        near += list(np.abs(c[max(0, n_p - 2): n_p] - t) / c[n - 1])
        n = min(n, n_p)
    if mp > 0:
        n_m = int((w >= mp).sum())
        # relative, as a weight is known to 2^-36 of itself; the largest is 1 exactly
        near += [abs(v - mp) / mp for v in w[max(0, n_m - 1): n_m + 1] if v < 1]
        n = min(n, n_m)
    t = (float(min(max(u, 0.0), 1 - 2.0 ** -24)) if u == u else 0.0) * c[n - 1]
    j = min(n - 1, int((c <= t).sum()))
    if t > 0:
        near += list(np.abs(c[max(0, j - 1): min(j + 1, n - 1)] - t) / c[n - 1])
    return int(order[j]), float(np.log(w[j] / c[n - 1])), n, min([float(v) for v in near] + [1.0])


def _call(qk, cuda, x, u, T, k=0, p=1.0, mp=0.0, offset=0):
    import torch
    M, V = x.shape
    tok = torch.full((M,), -7, dtype=torch.int32, device=cuda)
    kept = torch.full((M,), -7, dtype=torch.int32, device=cuda)
    lp = torch.full((M,), 7.0, device=cuda)
    qk.qk_sample(torch.from_numpy(np.ascontiguousarray(x)).to(cuda), torch.from_numpy(u.astype(np.float32)).to(cuda),
                 tok, lp, kept, M, V, temperature=T, top_k=k, top_p=p, min_p=mp)
    return tok.cpu().numpy(), lp.cpu().numpy(), kept.cpu().numpy()


def _check(qk, cuda, x, u, T, k=0, p=1.0, mp=0.0, exempt=0):
    tok, lp, kept = _call(qk, cuda, x, u, T, k, p, mp)
    close = 0
    for m in range(len(x)):
        t, want, n, near = reference(x[m], float(u[m]), T, k, p, mp)
        if near < NEAR:
            close += 1
            continue
        assert (tok[m], kept[m]) == (t, n), (m, tok[m], t, kept[m], n, near)
        if t < 0 or n == 0:
            assert math.isnan(lp[m])
        else:
            assert abs(lp[m] - want) <= abs(want) * 2.0 ** -22 + 2.0 ** -29, (m, lp[m], want)
    assert close <= exempt
    return tok, lp, kept


def _rows(seed, M, V, spread=2.5, banned=0.0):
    rng = synth.rng_for(seed, M * 1000003 + V)
    x = (spread * rng.standard_normal((M, V))).astype(np.float32)
    if banned:
        x[rng.random((M, V)) < banned] = -np.inf
        x[:, 0] = 1.0
    if V > 20:
        at = rng.integers(0, V, (M, 8))
        np.put_along_axis(x, at, (6 + 6 * rng.random((M, 8))).astype(np.float32), 1)
    return x, rng.random(M).astype(np.float32)


SETTINGS = [(1.0, 0, 1.0, 0.0), (0.8, 40, 0.95, 0.05), (1.0, 0, 0.9, 0.0), (1.3, 0, 0.999, 0.0), (0.6, 0, 1.0, 0.02),
            (1.5, 300, 1.0, 0.0), (2.0, 3000, 0.97, 0.001), (1.0, 1, 1.0, 0.0), (3.0, 0, 0.5, 0.3), (0.3, 7, 0.3, 0.9),
            (0.0, 5, 0.5, 0.5), (1.1, 90, 1.0, 0.003), (1.5, 512, 0.9, 0.0), (1.5, 513, 1.0, 0.01), (5.0, 0, 0.99, 0.0),
            (1.0, 0, 0.0, 0.0), (1.0, 0, 1.0, 1.0), (100.0, 0, 0.7, 0.0)]


@pytest.mark.parametrize("T,k,p,mp", SETTINGS)
@pytest.mark.parametrize("M,V", [(5, 1), (7, 2), (3, 5), (9, 33), (40, 1000), (3, 4097), (2, 16385), (3, 128256)])
def test_sample(qk_lib, cuda, M, V, T, k, p, mp):
    x, u = _rows(501, M, V, banned=0.03 if V > 4 else 0.0)
    _check(qk_lib, cuda, x, u, T, k, p, mp, exempt=1 if V > 10000 else 0)


@pytest.mark.parametrize("T,k,p,mp", SETTINGS[:5])
def test_sample_longest_rows(qk_lib, cuda, T, k, p, mp):
    x, u = _rows(502, 2, 524288)
    _check(qk_lib, cuda, x, u, T, k, p, mp, exempt=1)


@pytest.mark.parametrize("M,V", [(500, 3001), (160, 2047), (80, 9000), (37, 12001), (18, 40001), (2000, 50)])
def test_sample_many_rows(qk_lib, cuda, M, V):
    """Every number of CTAs a row; rows that start off 16-byte boundaries."""
    x, u = _rows(503, M, V)
    _check(qk_lib, cuda, x, u, 0.9, 60, 0.9, 0.01)
    _check(qk_lib, cuda, x, u, 1.1, 0, 1.0, 0.0, exempt=1)


def test_a_row_is_the_same_in_any_call(qk_lib, cuda):
    x, u = _rows(504, 600, 8191)
    for s in ((1.0, 0, 1.0, 0.0), (0.9, 0, 0.9, 0.0), (1.0, 50, 1.0, 0.0)):
        whole = _call(qk_lib, cuda, x, u, *s)
        again = _call(qk_lib, cuda, x, u, *s)
        parts = [np.concatenate(v) for v in zip(*(_call(qk_lib, cuda, x[a:b], u[a:b], *s)
                                                  for a, b in ((0, 1), (1, 9), (9, 60), (60, 600))))]
        for a, b, c in zip(whole, again, parts):
            assert np.array_equal(a, b) and np.array_equal(a, c)


@pytest.mark.parametrize("V", [1, 3, 700, 2049, 5000, 128256])
def test_equal_logits(qk_lib, cuda, V):
    """All equal: the order is the tokens', and every border falls between two of them."""
    u = np.array([0.0, 0.1, 0.5, 0.77, 0.99999994], np.float32)
    x = np.full((len(u), V), -3.25, np.float32)
    for T, k, p, mp in ((1.0, 0, 1.0, 0.0), (0.7, 0, 0.333, 0.0), (1.0, (V + 1) // 2, 1.0, 0.5), (1.0, 0, 0.5, 1.0)):
        tok, lp, kept = _call(qk_lib, cuda, x, u, T, k, p, mp)
        n = min(k or V, int(np.ceil(float(np.float32(p)) * (k or V))) if p < 1 else V)
        assert (kept == n).all()
        want = np.floor(u.astype(np.float64) * n).astype(int)
        assert np.array_equal(tok, want), (tok, want)
        assert np.abs(lp + np.log(n)).max() <= 2.0 ** -20


@pytest.mark.parametrize("step", [1.0, 0.25, 0.03125])
@pytest.mark.parametrize("T,k,p,mp", SETTINGS[:9])
def test_ties(qk_lib, cuda, step, T, k, p, mp):
    """Logits on a grid: thousands of equal ones at every border."""
    x, u = _rows(505, 4, 30000)
    x = (np.round(x / step) * step).astype(np.float32)
    _check(qk_lib, cuda, x, u, T, k, p, mp, exempt=1)


@pytest.mark.parametrize("T,k,p,mp", SETTINGS[:7])
def test_logits_of_fewer_bits(qk_lib, cuda, T, k, p, mp):
    """Logits that were fp16 or bf16: many equal ones, and many in the middle between two bins."""
    x, u = _rows(514, 8, 30000)
    x[4:] = x[4:].astype(np.float16)
    bits = x[:4].view(np.uint32)
    x[:4] = ((bits + 0x7FFF + ((bits >> 16) & 1)) & 0xFFFF0000).view(np.float32)
    _check(qk_lib, cuda, x, u, T, k, p, mp)


def test_zeros_of_both_signs_are_equal(qk_lib, cuda):
    x = np.zeros((1, 64), np.float32)
    x[0, ::2] = -0.0
    for i in range(0, 64, 7):
        tok, _, kept = _call(qk_lib, cuda, x, np.array([(i + 0.5) / 64], np.float32), 1.0)
        assert tok[0] == i and kept[0] == 64
    assert _call(qk_lib, cuda, x, np.zeros(1, np.float32), 0.0)[0][0] == 0


def test_every_token_by_its_share(qk_lib, cuda):
    """A sweep of u over a small row finds each token between its borders."""
    p = np.array([0.05, 0.4, 0.1, 0.25, 0.2])
    x = np.log(p).astype(np.float32)
    u = ((np.arange(1000) + 0.5) / 1000).astype(np.float32)
    tok, lp, kept = _check(qk_lib, cuda, np.tile(x, (1000, 1)), u, 1.0)
    assert np.array_equal(np.bincount(tok, minlength=5), (p * 1000).astype(int)) and (kept == 5).all()


def test_random_numbers_out_of_range(qk_lib, cuda):
    x, _ = _rows(506, 1, 300)
    u = np.array([0.0, -1.0, -np.inf, np.nan, 1.0, 2.0, np.inf, 0.99999994], np.float32)
    for s in ((1.0, 0, 1.0, 0.0), (1.0, 20, 0.9, 0.0)):
        tok = _call(qk_lib, cuda, np.tile(x, (len(u), 1)), u, *s)[0]
        assert (tok[:4] == tok[0]).all() and (tok[4:] == tok[7]).all() and tok[0] != tok[7]
        assert tok[0] == x[0].argmax()


@pytest.mark.parametrize("T,k,p,mp", [(1.3, 0, 1.0, 0.0), (0.5, 0, 1.0, 0.0), (20.0, 0, 1.0, 0.0), (1.0, 0, 0.9999, 0.0),
                                      (0.1, 3000, 1.0, 0.0), (0.1, 3000, 0.95, 0.0), (0.3, 2411, 1.0, 0.04),
                                      (0.05, 15000, 0.999, 0.0), (2.0, 9000, 1.0, 0.0), (0.4, 20001, 0.9, 0.0)])
def test_the_ends_of_rows(qk_lib, cuda, T, k, p, mp):
    """Random numbers near 1, where thousands of tokens share a little of the sum, and a
    top_k among tokens whose weights are 0 in every sum.  Weights there can be as small as the
    distance that counts as near: by the definition alone 12 of the rows are at T 0.5, one at
    1.3 and none elsewhere."""
    x, _ = _rows(512, 40, 20000)
    u = (1 - 10.0 ** (-0.5 - 6.5 * (np.arange(40) / 40))).astype(np.float32)
    _check(qk_lib, cuda, x, u, T, k, p, mp, exempt={0.5: 12, 1.3: 1}.get(T, 0))


def test_rows_without_an_answer(qk_lib, cuda):
    x, u = _rows(507, 8, 5000)
    x[0, 4999], x[1, 0], x[2] = np.nan, np.inf, -np.inf
    x[3, :-1] = -np.inf
    x[4] = np.nan
    x[5, 1:] = -np.inf
    for s in ((1.0, 0, 1.0, 0.0), (0.0, 0, 1.0, 0.0), (0.8, 50, 0.9, 0.1)):
        tok, _, kept = _check(qk_lib, cuda, x, u, *s)
        assert list(tok[:6]) == [-1, -1, -1, 4999, -1, 0] and list(kept[:6]) == [0, 0, 0, 1, 0, 1]


def test_extreme_logits(qk_lib, cuda):
    rng = synth.rng_for(508, 0)
    u = rng.random(40).astype(np.float32)
    big = rng.choice(np.array([3.4e38, -3.4e38, 1e30, -1e30, 0.0], np.float32), (40, 900))
    close = (1e6 + np.arange(900) % 7 * 0.0625)[None].repeat(40, 0).astype(np.float32)
    tiny = (1e-38 * rng.standard_normal((40, 900))).astype(np.float32)
    wide = (60 * rng.standard_normal((40, 900))).astype(np.float32)
    for x in (big, close, tiny, wide):
        for s in ((1.0, 0, 1.0, 0.0), (0.5, 0, 0.9, 0.0), (1e-6, 30, 1.0, 0.0), (1e6, 0, 0.8, 0.1), (2.0, 400, 0.99, 1e-12)):
            _check(qk_lib, cuda, x, u, *s, exempt=40 if x is not wide else 0)


def test_outputs_that_are_not_wanted(qk_lib, cuda):
    import torch
    x, u = _rows(509, 3, 2000)
    want = _call(qk_lib, cuda, x, u, 0.9, 30)
    tok = torch.zeros(3, dtype=torch.int32, device=cuda)
    xd, ud = torch.from_numpy(x).to(cuda), torch.from_numpy(u).to(cuda)
    qk_lib.qk_sample(xd, ud, tok, None, None, 3, 2000, 0.9, 30)
    assert np.array_equal(tok.cpu().numpy(), want[0])
    qk_lib.qk_sample(xd, ud, tok, None, None, 0, 2000)
    for bad in (dict(token=ud.view(torch.int32)), dict(kept=tok), dict(logprob=xd.view(-1)[:3])):
        with pytest.raises(qk_lib.QKError) as e:
            qk_lib.qk_sample(xd, ud, bad.get("token", tok), bad.get("logprob"), bad.get("kept"), 3, 2000)
        assert e.value.status == -7
    # nothing but the rows' own places is written
    guard = torch.full((16,), -9, dtype=torch.int32, device=cuda)
    qk_lib.qk_sample(xd, ud, guard, None, None, 3, 2000)
    assert (guard[3:] == -9).all()


def test_more_than_2_31_logits(qk_lib, cuda):
    """Rows behind 2^31 logits are as in a call of their own."""
    import torch
    M, V = 17000, 128256
    g = torch.Generator(device=cuda).manual_seed(513)
    x = torch.empty(M, V, device=cuda)
    for i in range(0, M, 1000):
        x[i: i + 1000].normal_(generator=g)
    u = torch.rand(M, generator=g, device=cuda)
    tok, kept = (torch.full((M,), -7, dtype=torch.int32, device=cuda) for _ in range(2))
    lp = torch.empty(M, device=cuda)
    qk_lib.qk_sample(x, u, tok, lp, kept, M, V, 0.8, 40, 0.95, 0.05)
    rows = torch.tensor([0, 16743, 16744, 16745, M - 1], device=cuda)
    t2, k2, lp2 = torch.empty(5, dtype=torch.int32, device=cuda), torch.empty(5, dtype=torch.int32, device=cuda), torch.empty(
        5, device=cuda)
    qk_lib.qk_sample(x[rows], u[rows], t2, lp2, k2, 5, V, 0.8, 40, 0.95, 0.05)
    assert torch.equal(tok[rows], t2) and torch.equal(kept[rows], k2) and (tok >= 0).all()
    qk_lib.qk_sample(x, u, tok, None, None, M, V, 0.0)
    assert torch.equal(tok[rows].long(), x[rows].argmax(1))
    del x
    torch.cuda.empty_cache()


def test_sample_in_a_graph_with_new_numbers(qk_lib, cuda):
    """A captured call follows the logits and the random numbers that its buffers hold."""
    import torch
    x, u = _rows(510, 4, 128256)
    xd, ud = torch.zeros(4, 128256, device=cuda), torch.zeros(4, device=cuda)
    tok = torch.zeros(4, dtype=torch.int32, device=cuda)
    kept, lp = torch.zeros_like(tok), torch.zeros(4, device=cuda)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        qk_lib.qk_sample(xd, ud, tok, lp, kept, 4, 128256, 0.9, 0, 0.95, 0.0)
    for i in range(3):
        y, v = np.roll(x, i, 0), np.roll(u, 2 * i)
        xd.copy_(torch.from_numpy(y))
        ud.copy_(torch.from_numpy(v.copy()))
        graph.replay()
        torch.cuda.synchronize()
        want = _call(qk_lib, cuda, y, v, 0.9, 0, 0.95, 0.0)
        assert np.array_equal(tok.cpu().numpy(), want[0]) and np.array_equal(kept.cpu().numpy(), want[2])
