"""The operators of a decode loop together: prompt and tokens appended with their head
norms to a 4-bit cache, attention over it, the LM head's product, a sampled token that
is the next one's input; in one stream, in two at once, and from graphs."""
import math
import os
import subprocess
import sys

import numpy as np
import pytest

from tests import kv4_reference as ref4
from tests import synth
from tests.test_gpu_sample import NEAR, reference

pytestmark = pytest.mark.gpu

H, HKV, D, V, L, EPS = 8, 2, 128, 2000, 160, 1e-6
SCALE = D ** -0.5
NONE = 10 ** 9


class _Loop:
    """A one-layer model: a token's q, k and v are rows of three tables, its logits the
    attention's output times a Q4_K matrix."""

    def __init__(self, qk, cuda, seed):
        import torch
        self.qk, self.cuda = qk, cuda
        rng = synth.rng_for(seed, 0)
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(cuda)  # noqa: E731
        self.tables = [dev(rng.standard_normal((V, h, D)).astype(np.float32)) for h in (H, HKV, HKV)]
        self.gammas = [dev((1 + 0.2 * rng.standard_normal(D)).astype(np.float16)) for _ in range(2)]
        self.freq = dev(500000.0 ** (-np.arange(0, D, 2) / D))
        self.head = dev(synth.q4k_weights(rng, V, H * D))
        self.u = dev(rng.random(64).astype(np.float32))
        self.prompt = dev(rng.integers(0, V, 60))
        self.reset()

    def reset(self):
        import torch
        z = lambda t, *s: torch.zeros(*s, dtype=t, device=self.cuda)  # noqa: E731
        self.cache = [z(torch.uint8, HKV, L, D // 2), z(torch.float16, HKV, L, D // 32, 2), z(torch.uint8, HKV, L, D // 2),
                      z(torch.float16, HKV, L, D // 32, 2)]
        self.q16, self.out = z(torch.float16, 60, H, D), z(torch.float16, 60, H, D)
        self.logits = z(torch.float32, 1, V)
        self.token, self.kept, self.lp = z(torch.int32, 1), z(torch.int32, 1), z(torch.float32, 1)
        self.scratch = z(torch.uint8, self.qk.qk_gqa_attention_q4_scratch_bytes(60, H, HKV, D, 0, NONE))
        self.made = z(torch.int32, 64)

    def step(self, tokens, pos0, n, window=NONE, sinks=0, top_k=50, top_p=0.9):
        """Tokens (a device tensor) at pos0 ..; the n-th token follows."""
        qk, M = self.qk, len(tokens)
        q, k, v = (t[tokens.long()] for t in self.tables)
        qk.qk_norm_rope_kv_append_q4(q, k, v, *self.gammas, EPS, self.freq, self.q16, *self.cache, M, H, HKV, D, D, pos0, L,
                                     layout=qk.QK_ROPE_HALF)
        qk.qk_gqa_attention_q4(self.q16, *self.cache, self.out, M, H, HKV, D, pos0, L, SCALE, window, sinks,
                               scratch=self.scratch)
        qk.qk_matmul_q4k(self.head, self.out[M - 1], self.logits, 1, V, H * D)
        qk.qk_sample(self.logits, self.u[n: n + 1].clone(), self.token, self.lp, self.kept, 1, V, 0.7, top_k, top_p)
        self.made[n: n + 1] = self.token

    def run(self, steps=10):
        self.step(self.prompt, 0, 0)
        for n in range(1, steps):
            self.step(self.token.clone(), 59 + n, n, 40, 4)
        return self.made


def test_generation_step_by_step(qk_lib, cuda):
    """Each step against numpy in 64 bits, from what the step before left on the device.
    Attention within its own tolerance (2^-10 and twice 2^-12 of the largest |v|); the token
    equal, where the logits are the device's; its log probability beside qk_logprobs'."""
    import torch
    m = _Loop(qk_lib, cuda, 501)
    for n in range(12):
        tokens = m.prompt if n == 0 else m.token.clone()
        pos0, window, sinks = (0, NONE, 0) if n == 0 else (59 + n, 40, 4)
        m.step(tokens, pos0, n, window, sinks, *((0, 1.0) if n % 3 == 2 else (50, 0.9)))
        M = len(tokens)
        q16 = m.q16[:M].cpu().numpy()
        k, v = ref4.values(m.cache[0].cpu().numpy(), m.cache[1].cpu().numpy()), ref4.values(
            m.cache[2].cpu().numpy(), m.cache[3].cpu().numpy())
        # the new rows are within half a step d of what was appended, and d's and m's roundings
        want = m.tables[2][tokens.long()].cpu().numpy().transpose(1, 0, 2)
        d = np.repeat(m.cache[3].cpu().numpy()[:, pos0: pos0 + M, :, 0].astype(np.float64), 32, -1)
        assert (np.abs(v[:, pos0: pos0 + M] - want) <= d * 0.51 + np.abs(want).max() * 2.0 ** -9).all()
        exact = ref4.attention(q16, k, v, H, HKV, pos0, window, sinks, SCALE)
        err = np.abs(m.out[:M].cpu().numpy() - exact).max()
        assert err <= np.abs(v).max() * (2.0 ** -10 + 2.0 ** -11), (n, err)
        x = m.logits[0].cpu().numpy()
        k_, p_ = (0, 1.0) if n % 3 == 2 else (50, 0.9)
        t, lp, kept, near = reference(x, float(m.u[n]), 0.7, k_, p_)
        if near >= NEAR:
            assert (int(m.token[0]), int(m.kept[0])) == (t, kept)
            assert abs(float(m.lp[0]) - lp) <= abs(lp) * 2.0 ** -22 + 2.0 ** -29
        if n % 3 == 2:
            # all tokens kept at temperature 0.7: log softmax of logits / 0.7.  qk_logprobs of fp32
            # x / 0.7 (2^-24 of |x / 0.7| each) is off by its own lse's fp32 too: 2^-20 of both
            y = (m.logits / 0.7).contiguous()
            other = torch.zeros(1, device=cuda)
            qk_lib.qk_logprobs(y, m.token, other, None, 0, None, None, 1, V)
            assert abs(float(other[0]) - float(m.lp[0])) <= 2.0 ** -20 * (float(y.abs().max()) + abs(lp) + 1)


def test_two_loops_at_once(qk_lib, cuda):
    """Two loops on two streams, a step of one between the steps of the other: as alone."""
    import torch
    loops = [_Loop(qk_lib, cuda, s) for s in (502, 503)]
    want = [m.run().clone() for m in loops]
    torch.cuda.synchronize()
    for m in loops:
        m.reset()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in loops]
    for n in range(10):
        for m, s in zip(loops, streams):
            with torch.cuda.stream(s):
                if n == 0:
                    m.step(m.prompt, 0, 0)
                else:
                    m.step(m.token.clone(), 59 + n, n, 40, 4)
    torch.cuda.synchronize()
    for m, w in zip(loops, want):
        assert torch.equal(m.made, w)


def test_graphs_of_long_attention_at_once(qk_lib, cuda):
    """Two captured calls that split positions over all SMs and join through scratches of
    their own, replayed on two streams: each as alone, every time."""
    import torch
    n = 40000
    rng = synth.rng_for(504, 0)
    q4, dm = ref4.random_cache(rng, 4, n)
    c4, cd = torch.from_numpy(q4).to(cuda), torch.from_numpy(dm).to(cuda)
    calls = []
    for i in range(2):
        q = torch.from_numpy((1.5 * rng.standard_normal((1, 8, D))).astype(np.float16)).to(cuda)
        out = torch.zeros_like(q)
        scratch = torch.zeros(qk_lib.qk_gqa_attention_q4_scratch_bytes(1, 8, 4, D, n - 1 - i, NONE), dtype=torch.uint8,
                              device=cuda)
        assert len(scratch)

        def call(q=q, out=out, scratch=scratch, pos0=n - 1 - i):
            qk_lib.qk_gqa_attention_q4(q, c4, cd, c4, cd, out, 1, 8, 4, D, pos0, n, SCALE, NONE, 0, scratch=scratch)
        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(5):
                call()
        calls.append((graph, out, out.clone(), torch.cuda.Stream(), call))  # call holds q and the scratch
    torch.cuda.synchronize()
    for _ in range(20):
        for graph, out, _, s, _ in calls:
            with torch.cuda.stream(s):
                out.fill_(math.nan)
                graph.replay()
    torch.cuda.synchronize()
    for _, out, want, _, _ in calls:
        assert torch.equal(out, want)


_CHILD = r"""
import sys, numpy as np, torch
sys.path.insert(0, sys.argv[1])
import quantized_q4_matmul_gb300 as qk
from tests import kv4_reference as ref4
from tests import synth
dev = torch.device("cuda", 0)
rng = synth.rng_for(505, 0)
H, Hkv, D, L, V, M = 8, 4, 128, 9000, 5000, 300
f32 = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).to(dev)
q, k, v, gamma = f32(M, H, D), f32(M, Hkv, D), f32(M, Hkv, D), f32(D).half()
freq = torch.from_numpy(np.asarray(qk.qk_rope_inv_freq(64, theta=10000.0))).to(dev)
cache = [torch.from_numpy(a).to(dev) for a in ref4.random_cache(rng, Hkv, L) + ref4.random_cache(rng, Hkv, L)]
logits, u = f32(5, V), torch.rand(5, device=dev)
z = lambda t, *s: torch.zeros(*s, dtype=t, device=dev)
f16, i32 = torch.float16, torch.int32
o = dict(q16=z(f16, M, H, D), kc=z(f16, Hkv, L, D), vc=z(f16, Hkv, L, D), q4=z(f16, M, H, D), rows=z(f16, Hkv, M, D),
         chunk=z(f16, M, H, D), one=z(f16, 1, H, D), two=z(f16, 2, H, D), nine=z(f16, 9, H, D), sixteen=z(f16, 16, H, D),
         long=z(f16, 1, H, D), longs=z(f16, 3, H, D), none=torch.ones(3, H, D, dtype=f16, device=dev), tok=z(i32, 5),
         lp=z(torch.float32, 5), kept=z(i32, 5), tok2=z(i32, 5), lp2=z(torch.float32, 5), kept2=z(i32, 5))
scratch = z(torch.uint8, max(qk.qk_gqa_attention_q4_scratch_bytes(M, H, Hkv, D, 0, 10 ** 9),
                             qk.qk_gqa_attention_q4_scratch_bytes(3, H, Hkv, D, L - 3, 10 ** 9)))

def attn(out, m, pos0, window=10 ** 9, sinks=0):
    qk.qk_gqa_attention_q4(o["q4"], *cache, out, m, H, Hkv, D, pos0, L, D ** -0.5, window, sinks, scratch=scratch)

def calls():
    qk.qk_norm_rope_kv_append(q, k, v, gamma, gamma, 1e-6, freq, o["q16"], o["kc"], o["vc"], M, H, Hkv, D, 64, 0, L)
    qk.qk_norm_rope_kv_append_q4(q, k, v, gamma, None, 1e-6, freq, o["q4"], *cache, M, H, Hkv, D, 64, 0, L, qk.QK_ROPE_HALF)
    qk.qk_dequant_kv_q4(cache[0], cache[1], o["rows"], Hkv, D, 0, M, L)
    attn(o["chunk"], M, 0, 100, 4)
    attn(o["one"], 1, M - 1)
    attn(o["two"], 2, M - 2, 50, 3)
    attn(o["nine"], 9, M - 9)
    attn(o["sixteen"], 16, M - 16)
    attn(o["long"], 1, L - 1)
    attn(o["longs"], 3, L - 3)
    attn(o["none"], 3, 0, 0)
    qk.qk_sample(logits, u, o["tok"], o["lp"], o["kept"], 5, V, 0.8, 40, 0.95)
    qk.qk_sample(logits, u, o["tok2"], o["lp2"], o["kept2"], 5, V, 1.1, 0, 0.9)

torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
    calls()
for t in o.values():
    t.zero_()
for _ in range(2):
    graph.replay()
torch.cuda.synchronize()
replayed = {n: t.clone() for n, t in o.items()}
for t in o.values():
    t.zero_()
calls()
torch.cuda.synchronize()
for n, t in o.items():
    assert torch.equal(replayed[n], t), n
assert bool((o["none"] == 0).all()) and bool((o["long"] != 0).any()) and bool((o["kept2"] > 0).all())
assert qk.lib().qk_get_device_status(None) == 0
print("ok")
"""


def test_first_calls_inside_a_capture(qk_lib, cuda):
    """What a first call of a process sets up (kernel attributes, how many clusters fit,
    tables) happens while capturing."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", _CHILD, root], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stdout[-2000:] + r.stderr[-3000:]
