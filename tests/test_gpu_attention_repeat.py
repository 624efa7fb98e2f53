"""A chunk's attention repeats its bits whatever ran on the SMs before.  With 3, 5
or 7 heads a key/value head a query tile's 128 rows are not all queries; what the
others hold (rests of earlier kernels in shared memory) must not reach a decision
that queries share with them."""
import numpy as np
import pytest

from tests import synth

pytestmark = pytest.mark.gpu

D = 128


@pytest.mark.parametrize("H,Hkv,M,pos0,window", [(24, 8, 1023, 3001, 10 ** 9), (24, 8, 500, 2000, 700), (5, 1, 400, 1000, 10 ** 9),
                                                 (14, 2, 300, 1500, 10 ** 9), (6, 2, 60, 4000, 10 ** 9)])
def test_window_chunks_repeat_their_bits_after_other_kernels(qk_lib, cuda, H, Hkv, M, pos0, window):
    import torch
    rng = synth.rng_for(420, M)
    L = pos0 + M
    q, k, v = (torch.from_numpy((a * rng.standard_normal((n, h, D))).astype(np.float16)).to(cuda)
               for a, n, h in ((1.5, M, H), (1.0, Hkv, L), (1.0, Hkv, L)))
    out = [torch.empty(M, H, D, dtype=torch.float16, device=cuda) for _ in range(12)]
    junk = torch.empty(1 << 24, device=cuda)
    for i, o in enumerate(out):
        qk_lib.qk_gqa_attention_window(q, k.view(Hkv, L, D), v.view(Hkv, L, D), o, M, H, Hkv, D, pos0, L, D ** -0.5, window, 3)
        # what other kernels leave behind: large and small values, infinities
        junk.uniform_(-10.0 ** (3 * i), 10.0 ** (3 * i))
        junk.copy_(junk.flip(0) * (float("inf") if i % 3 == 2 else 1.0))
        junk.cumsum(0)
    torch.cuda.synchronize()
    for i, o in enumerate(out):
        assert torch.equal(o, out[0]), (i, int((o != out[0]).sum()))
