"""RMSNorm in front of a linear whose K the decode GEMV can stage without the norm
and not with it (gamma takes shared memory beside x): the tensor-core GEMM runs
it, and the scratch for its normalized activations is asked for."""
import numpy as np
import pytest

import oracle
from tests import synth

QT = {"q4k": oracle.Q4K, "q6k": oracle.Q6K}
EPS = 1e-5

# format, gate/up, M, K that fits with gamma, K that fits without it alone
EDGES = [("q4k", False, 1, 27136, 27392), ("q4k", False, 1, 27136, 35840), ("q4k", False, 2, 11264, 11520),
         ("q4k", False, 8, 11264, 12288), ("q4k", False, 8, 11264, 12800), ("q6k", False, 1, 6400, 6656),
         ("q6k", False, 1, 6400, 6912), ("q6k", False, 1, 20480, 22528), ("q6k", False, 8, 4608, 4864),
         ("q4k", True, 1, 26368, 26624), ("q4k", True, 5, 10752, 11008), ("q4k", True, 8, 10752, 12032)]


@pytest.mark.parametrize("qtype,gateup,M,below,K", EDGES)
def test_scratch_is_asked_for(qk_lib, qtype, gateup, M, below, K):
    assert qk_lib.qk_uses_gemv(qtype, M, K, gateup) and qk_lib.qk_uses_gemv(qtype, M, below, gateup)
    assert qk_lib.qk_rmsnorm_scratch_bytes(qtype, M, below, gateup) == 0
    assert qk_lib.qk_rmsnorm_scratch_bytes(qtype, M, K, gateup) == 2 * M * K


def test_problems_without_a_gemv_plan_ask_for_it(qk_lib):
    """The norm never makes a problem fit: no scratch means a plan without the norm too."""
    for qtype, gateup in (("q4k", False), ("q6k", False), ("q4k", True)):
        for M in (1, 2, 8, 9):
            for K in range(256, 256 * 150, 256):
                need = qk_lib.qk_rmsnorm_scratch_bytes(qtype, M, K, gateup)
                assert need in (0, 2 * M * K)
                assert need or qk_lib.qk_uses_gemv(qtype, M, K, gateup)


@pytest.mark.gpu
@pytest.mark.parametrize("qtype,gateup,M,below,K", EDGES)
def test_rmsnorm_at_the_edge(qk_lib, cuda, qtype, gateup, M, below, K):
    """Right through the caller's scratch, which is not written past its size, and
    through the library's own; without scratch the call is refused."""
    import torch
    from tests.test_gpu_parity import _dev, _x_dev, check_close, gamma_vec
    N = 40
    rng = synth.rng_for(240 + M, K)
    W = [synth.weights(rng, qtype, N, K) for _ in range(1 + gateup)]
    x, g = synth.activations(rng, M, K), gamma_vec(rng, K)
    y = torch.full((M, N), float("nan"), dtype=torch.float16 if gateup else torch.float32, device=cuda)
    p = dict(qtype=qtype, blocks=_dev(W[0], cuda), x_f16=_x_dev(x, cuda), y=y, M=M, N=N, K=K)
    if gateup:
        p["up_blocks"] = _dev(W[1], cuda)
        ref = oracle.rmsnorm_gateup_swiglu(W[0], W[1], x, g, EPS, N, K)
    else:
        ref = oracle.rmsnorm_matmul(QT[qtype], W[0], x, g, EPS, N, K)
    gd = _x_dev(g, cuda)
    what = "rmsnorm %s M%d K%d" % (qtype, M, K)
    guard = torch.full((M * K + 64,), 7.0, dtype=torch.float16, device=cuda)
    qk_lib.qk_rmsnorm_matmul_batch([p], gd, EPS, guard)
    qk_lib.qk_get_device_status()
    check_close(y.float().cpu().numpy().astype(np.float64), ref, what)
    assert (guard[M * K:] == 7).all() and not (guard[:M * K] == 7).all()
    first = y.clone()
    y.fill_(float("nan"))
    qk_lib.qk_rmsnorm_matmul_batch_static([p], gd, EPS)
    qk_lib.qk_get_device_status()
    assert torch.equal(y, first)
    with pytest.raises(qk_lib.QKError) as e:
        qk_lib.qk_rmsnorm_matmul_batch([p], gd, EPS, None)
    assert e.value.status == -1
