"""Sums of long rows of equal logits far below the largest: what an addition rounds off must not
add up.  The definition has a closed form here, in 64 bits: weights 1 and n times w.  And zeros
of either sign in the settings."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu


def _call(qk, cuda, x, u, T, k=0, p=1.0):
    import torch
    M, V = len(u), x.numel()
    rows = x.to(cuda).expand(M, V).contiguous()
    tok, kept = (torch.full((M,), -7, dtype=torch.int32, device=cuda) for _ in range(2))
    qk.qk_sample(rows, torch.from_numpy(u).to(cuda), tok, None, kept, M, V, temperature=T, top_k=k, top_p=p)
    return tok.cpu().numpy(), kept.cpu().numpy()


# x of the many: weights just above 2^-24 and 2^-25 (half a step of 1), of the middle of a step, and large ones
@pytest.mark.parametrize("x", [-16.635532, -16.64, -17.04, -17.32868, -15.0, -12.0, -0.3, -1e-3])
@pytest.mark.parametrize("V,M", [(128256, 5), (128256, 200), (524288, 3), (20000, 300)])
def test_many_equal_logits_far_below_the_largest(qk_lib, cuda, x, V, M):
    """A row's tokens, and how many top_p keeps, by the closed form; but where a border lies
    so close to a decision that the sums' errors decide: V additions of 3 2^-48, 2^-29.7 for
    the threads' shares (8192 of them, five sums each, 2^-45) and the weights' 2^-36."""
    import torch
    near = V * 3 * 2.0 ** -48 + 2.0 ** -29.7 + 2.0 ** -36
    at = V // 3  # the largest
    row = torch.full((V,), x, dtype=torch.float32)
    row[at] = 0.0
    w = math.exp(float(np.float32(x)))
    S = 1 + (V - 1) * w
    u = np.linspace(1 / S, 1, M + 2)[1:-1].astype(np.float32)  # all in the tail
    tok, kept = _call(qk_lib, cuda, row, u, 1.0)
    assert (kept == V).all()
    place = (u.astype(np.float64) * S - 1) / w  # of the others: the first one whose sum exceeds u S
    j = np.floor(place).astype(np.int64)
    want = np.where(j < at, j, j + 1)
    clear = np.minimum(place - j, j + 1 - place) * w / S >= near
    assert np.array_equal(tok[clear], want[clear]), np.abs(tok - want)[clear].max()
    # top_p in the tail: n - 1 of the others, the first sum that reaches top_p S
    for p in (np.float32(1 / S + 0.5 * (1 - 1 / S)), np.float32(0.99999)):
        if p * S <= 1:
            continue
        n = (float(p) * S - 1) / w
        if min(n - math.floor(n), math.ceil(n) - n) * w / S < near:
            continue
        tok, kept = _call(qk_lib, cuda, row, u[:3] * 0, 1.0, p=float(p))
        assert (tok == at).all() and (kept == 1 + math.ceil(n)).all(), (kept, n)


def test_zeros_of_either_sign(qk_lib, cuda):
    """A top_p, min_p or temperature of -0 is 0."""
    import torch
    x = torch.from_numpy(np.random.default_rng(603).standard_normal((4, 3000)).astype(np.float32)).to(cuda)
    u = torch.tensor([0.0, 0.3, 0.6, 0.9], device=cuda)
    for kw in (dict(top_p=0.0), dict(top_p=0.0, top_k=40), dict(temperature=0.0), dict(min_p=0.0, top_p=0.9)):
        got = []
        for sign in (1.0, -1.0):
            tok, kept = (torch.full((4,), -7, dtype=torch.int32, device=cuda) for _ in range(2))
            lp = torch.full((4,), 7.0, device=cuda)
            qk_lib.qk_sample(x, u, tok, lp, kept, 4, 3000, **{n: v * sign if v == 0 else v for n, v in kw.items()})
            got.append((tok, lp, kept))
        for a, b in zip(*got):
            assert torch.equal(a, b), kw
        if "min_p" not in kw:
            assert bool((got[1][2] == 1).all()) and torch.equal(got[1][0].long(), x.argmax(1))
