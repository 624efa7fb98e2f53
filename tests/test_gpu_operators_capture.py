"""Every operator's first call of a process inside a graph capture: what a first
call sets up (kernel attributes, tensor maps, how many clusters fit) happens
while capturing, a kernel that starts early follows a memset node, and the
replays give what the same calls give outside a graph."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

_CHILD = r"""
import sys, numpy as np, torch
sys.path.insert(0, sys.argv[1])
import quantized_q4_matmul_gb300 as qk
from tests import synth
dev = torch.device("cuda", 0)
rng = synth.rng_for(301, 0)
H, Hkv, D, L, K, V = 8, 4, 128, 700, 512, 5000
f32 = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).to(dev)
M = 300
res, delta = f32(M, K), f32(M, K)
gamma = f32(K).half()
w = torch.from_numpy(synth.q4k_weights(rng, 96, K)).to(dev)
q, k, v = f32(M, H, D), f32(M, Hkv, D), f32(M, Hkv, D)
freq = torch.from_numpy(np.asarray(qk.qk_rope_inv_freq(64, theta=10000.0))).to(dev)
logits = f32(3, V)
tokens = torch.tensor([5, -1, V - 1], dtype=torch.int32, device=dev)
outs = dict(res=torch.zeros(M, K, device=dev), xhat=torch.zeros(M, K, dtype=torch.float16, device=dev),
            xq=torch.zeros(1, K, dtype=torch.int8, device=dev), xd=torch.zeros(1, K // 32, device=dev),
            y=torch.zeros(1, 96, device=dev), q16=torch.zeros(M, H, D, dtype=torch.float16, device=dev),
            kc=torch.zeros(Hkv, L, D, dtype=torch.float16, device=dev),
            vc=torch.zeros(Hkv, L, D, dtype=torch.float16, device=dev),
            a=torch.zeros(M, H, D, dtype=torch.float16, device=dev),
            few=torch.zeros(5, H, D, dtype=torch.float16, device=dev),
            none=torch.ones(7, H, D, dtype=torch.float16, device=dev),
            one=torch.zeros(1, H, D, dtype=torch.float16, device=dev), lp=torch.zeros(3, device=dev),
            ent=torch.zeros(3, device=dev), ids=torch.zeros(3, 4, dtype=torch.int32, device=dev),
            tlp=torch.zeros(3, 4, device=dev))
o = outs

def calls():
    qk.qk_add_rmsnorm(res, delta, gamma, 1e-5, o["res"], o["xhat"], M, K)
    qk.qk_add_rmsnorm_q8(res, delta, gamma, 1e-5, None, o["xq"], o["xd"], 1, K)
    qk.qk_matmul_batch_q8([dict(qtype="q4k", blocks=w, x_q8=o["xq"], x_d=o["xd"], y=o["y"], M=1, N=96, K=K)])
    qk.qk_rope_kv_append(q, k, v, freq, o["q16"], o["kc"], o["vc"], M, H, Hkv, D, 64, 0, L, qk.QK_ROPE_HALF)
    s = D ** -0.5
    qk.qk_gqa_attention_window(o["q16"], o["kc"], o["vc"], o["none"], 7, H, Hkv, D, 0, L, s, 0, 0)
    qk.qk_gqa_attention_window(o["q16"], o["kc"], o["vc"], o["a"], M, H, Hkv, D, 0, L, s, 100, 4)
    qk.qk_gqa_attention_window(o["q16"], o["kc"], o["vc"], o["few"], 5, H, Hkv, D, M - 5, L, s, 10 ** 6, 0)
    qk.qk_gqa_attention_window(o["q16"], o["kc"], o["vc"], o["one"], 1, H, Hkv, D, M - 1, L, s, 64, 4)
    qk.qk_logprobs(logits, tokens, o["lp"], o["ent"], 4, o["ids"], o["tlp"], 3, V)

stream = torch.cuda.Stream()
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph, stream=stream):
    calls()
for t in outs.values():
    t.zero_()
for _ in range(2):
    graph.replay()
torch.cuda.synchronize()
replayed = {n: t.clone() for n, t in outs.items()}
for t in outs.values():
    t.fill_(1)
calls()
torch.cuda.synchronize()
for n, t in outs.items():
    a, b = replayed[n], t
    if n in ("kc", "vc"):  # rows past the prompt keep what was there
        a, b = a[:, :M], b[:, :M]
    assert torch.equal(torch.nan_to_num(a.float(), nan=-7.0), torch.nan_to_num(b.float(), nan=-7.0)), n
assert bool((replayed["none"] == 0).all()) and bool(torch.isnan(replayed["lp"][1]))
assert qk.lib().qk_get_device_status(None) == 0
print("ok")
"""


def test_first_calls_inside_a_capture(qk_lib, cuda):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", _CHILD, root], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stdout[-2000:] + r.stderr[-3000:]
