"""The operators of a decoder step around its quantized linears: cases, plain forms and the library's calls.

  norm    residual addition + RMSNorm, output fp16 or int8 with a scale per 32 values
  q8mm    y = x . W^T for x already in int8 (one token), W in Q4_K / Q6_K
  rope    rotary positions on q and k, and the new k / v rows into the KV cache
  attn    grouped-query attention over the cache with a sliding window and sink tokens
  logp    log probabilities of given tokens, entropy and top alternatives from the LM head's logits

``own`` False: elementary torch operations.  ``own`` True: the calls of quantized_q4_matmul_gb300.
"""
import math

import torch

own = False

EPS = 1e-5
# Bytes of a 256-weight super-block.
BLOCK = {"q4k": 144, "q6k": 210}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # a decode step's norm: one row, all latency
        dict(name="norm one token", op="norm", M=1, K=4096, res32=False, q8=False),
        # a long prompt's norm with the residual stream in fp32: HBM
        dict(name="norm prompt", op="norm", M=2048, K=8192, res32=True, q8=False),
        # a ragged chunk into int8 activations
        dict(name="norm int8 chunk", op="norm", M=333, K=2560, res32=False, q8=True),
        # a decode step's q, k, v projections from one int8 x, in one call
        dict(name="int8 q, k, v", op="q8mm", K=4096, q4k=4096, q4k_b=1024, q6k=1024),
        # the tied LM head: 215 MB of weights for one token
        dict(name="int8 LM head", op="q8mm", K=2048, q4k=0, q4k_b=0, q6k=128256),
        # a decode step far into a long context
        dict(name="rope one token", op="rope", M=1, H=24, Hkv=8, D=128, n_rot=128, half=False, banded=True, pos0=31000,
             L_max=32768),
        # a prompt; part of the head rotates, the rest passes through
        dict(name="rope prompt", op="rope", M=2048, H=32, Hkv=8, D=128, n_rot=96, half=True, banded=False, pos0=5,
             L_max=4096),
        # a decode step: 4096 recent positions and 4 sinks of 20001 cached ones
        dict(name="attention one token", op="attn", M=1, H=24, Hkv=8, pos0=20000, window=4096, sinks=4),
        # a prompt with a short window
        dict(name="attention prompt", op="attn", M=2048, H=24, Hkv=8, pos0=0, window=512, sinks=4),
        # a chunk of a long prompt after 4000 cached positions, ragged at both ends
        dict(name="attention long chunk", op="attn", M=4095, H=24, Hkv=8, pos0=4001, window=2048, sinks=16),
        # a decode step's logits, a fiftieth of the vocabulary banned
        dict(name="log-probs one token", op="logp", M=1, V=128256, top=5, banned=0.02),
        # scoring a prompt
        dict(name="log-probs prompt", op="logp", M=1024, V=128256, top=20, banned=0.0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


_HEADS = ((24, 8), (32, 8), (32, 4), (8, 8), (6, 2), (4, 1))


def draw(rng):
    op = rng.choice(("norm", "q8mm", "rope", "attn", "logp"))
    if op == "norm":
        return dict(op=op, M=_log_int(rng, 1, 2048), K=32 * _log_int(rng, 4, 256), res32=rng.random() < 0.5,
                    q8=rng.random() < 0.5)
    if op == "q8mm":
        return dict(op=op, K=256 * rng.randint(1, 24), q4k=_log_int(rng, 1, 40000),
                    q4k_b=_log_int(rng, 1, 3000) if rng.random() < 0.5 else 0,
                    q6k=_log_int(rng, 1, 20000) if rng.random() < 0.5 else 0)
    if op == "rope":
        H, Hkv = rng.choice(_HEADS)
        D = rng.choice((64, 80, 128, 256))
        M = 1 if rng.random() < 0.3 else _log_int(rng, 2, 2048)
        pos0 = rng.choice((0, _log_int(rng, 1, 30000)))
        return dict(op=op, M=M, H=H, Hkv=Hkv, D=D, n_rot=rng.choice((D, 2 * rng.randint(1, D // 2))),
                    half=rng.random() < 0.5, banded=rng.random() < 0.5, pos0=pos0, L_max=pos0 + M + rng.randint(0, 500))
    if op == "attn":
        H, Hkv = rng.choice(_HEADS)
        M = 1 if rng.random() < 0.35 else _log_int(rng, 2, 3000)
        return dict(op=op, M=M, H=min(H, 24), Hkv=Hkv if H <= 24 else 8, pos0=rng.choice((0, _log_int(rng, 1, 20000))),
                    window=_log_int(rng, 1, 3000), sinks=rng.choice((0, _log_int(rng, 1, 80))))
    return dict(op=op, M=_log_int(rng, 1, 800), V=_log_int(rng, 500, 150000), top=rng.randint(1, 32),
                banned=rng.choice((0.0, 0.05)))


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _weights(g, kind, N, K):
    """Random super-blocks [N][K / 256][bytes]: uniform quants, |d| near 1e-4."""
    nb = K // 256
    w = torch.randint(0, 256, (N, nb, BLOCK[kind]), generator=g, device="cuda", dtype=torch.uint8)
    d = (_randn(g, N, nb, 2).abs() * 1e-4).half().view(torch.uint8)  # [N][nb][4]
    if kind == "q4k":
        w[:, :, :4] = d
    else:
        w[:, :, 192:208] = torch.randint(-32, 64, (N, nb, 16), generator=g, device="cuda", dtype=torch.int8).view(
            torch.uint8)
        w[:, :, 208:] = d[:, :, :2]
    return w


def _inv_freq(n_rot, banded):
    """Radians per position of each pair: theta^(-2i / n_rot), or with its long wavelengths stretched 8 times."""
    f = 500000.0 ** (-torch.arange(0, n_rot, 2, dtype=torch.float64) / n_rot)
    if banded:
        turns = 8192 * f / (2 * math.pi)
        keep = ((turns - 1.0) / (4.0 - 1.0)).clamp(0.0, 1.0)
        f = (1 - keep) * f / 8.0 + keep * f
    return f


def _problems(c):
    return [(kind, c[key]) for key, kind in (("q4k", "q4k"), ("q4k_b", "q4k"), ("q6k", "q6k")) if c[key] > 0]


def prepare(case, seed):
    g, c = _gen(seed), dict(case)
    s = {"c": c}
    if c["op"] == "norm":
        M, K = c["M"], c["K"]
        loud = 1.0 + 15.0 * (torch.rand(K, generator=g, device="cuda") < 0.01)  # a few channels carry large values
        res = _randn(g, M, K) * loud
        s["res"] = res if c["res32"] else res.half()
        s["delta"] = _randn(g, M, K) * 0.3
        s["gamma"] = (1 + 0.1 * _randn(g, K)).half()
        s["res_out"] = torch.empty_like(s["res"])
        s["xhat"] = torch.empty(M, K, dtype=torch.float16, device="cuda")
        s["xq"] = torch.empty(M, K, dtype=torch.int8, device="cuda")
        s["xd"] = torch.empty(M, K // 32, dtype=torch.float32, device="cuda")
    elif c["op"] == "q8mm":
        K = c["K"]
        x = _randn(g, K // 32, 32)
        s["xd"] = (x.abs().amax(1) / 127).contiguous()
        s["xq"] = torch.round(x / s["xd"][:, None]).to(torch.int8).view(1, K)
        s["w"] = [_weights(g, kind, N, K) for kind, N in _problems(c)]
        s["y"] = [torch.empty(1, N, device="cuda") for _, N in _problems(c)]
        s["xd"] = s["xd"].view(1, K // 32)
    elif c["op"] == "rope":
        M, H, Hkv, D, L = c["M"], c["H"], c["Hkv"], c["D"], c["L_max"]
        s["q"], s["k"], s["v"] = _randn(g, M, H, D), _randn(g, M, Hkv, D), _randn(g, M, Hkv, D)
        s["kc"], s["vc"] = _randn(g, Hkv, L, D).half(), _randn(g, Hkv, L, D).half()
        s["qo"] = torch.empty(M, H, D, dtype=torch.float16, device="cuda")
        s["inv_freq"] = _inv_freq(c["n_rot"], c["banded"]).cuda()
    elif c["op"] == "attn":
        M, H, Hkv, n = c["M"], c["H"], c["Hkv"], c["pos0"] + c["M"]
        s["q"] = (1.5 * _randn(g, M, H, 128)).half()
        s["kc"], s["vc"] = _randn(g, Hkv, n + 3, 128).half(), _randn(g, Hkv, n + 3, 128).half()
        s["out"] = torch.empty(M, H, 128, dtype=torch.float16, device="cuda")
    else:
        M, V = c["M"], c["V"]
        x = 2.5 * _randn(g, M, V)
        peak = torch.randint(0, V, (M,), generator=g, device="cuda")
        rows = torch.arange(M, device="cuda")
        if c["banned"] > 0:
            x[torch.rand(M, V, generator=g, device="cuda") < c["banned"]] = -math.inf
        # the model's own choice, from unsure to sure, and the token that is scored: the choice in half of the rows
        x[rows, peak] = 8 + 6 * torch.rand(M, generator=g, device="cuda")
        other = torch.randint(0, V, (M,), generator=g, device="cuda")
        s["tok"] = torch.where(torch.rand(M, generator=g, device="cuda") < 0.5, peak, other).to(torch.int32)
        s["x"] = x
        s["lp"], s["ent"] = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
        s["ids"] = torch.empty(M, c["top"], dtype=torch.int32, device="cuda")
        s["tlp"] = torch.empty(M, c["top"], device="cuda")
    return s


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------
def _plain_norm(s, c):
    h = s["res"].float() + s["delta"]
    r = 1.0 / torch.sqrt((h * h).mean(1, keepdim=True) + EPS)
    x = (h * r * s["gamma"].float()).half()
    if not c["q8"]:
        return h.to(s["res"].dtype), x
    b = x.float().view(c["M"], -1, 32)
    d = b.abs().amax(2, keepdim=True) / 127.0
    t = torch.where(d > 0, b / d, torch.zeros_like(b)).double()
    q = torch.trunc(t + torch.copysign(torch.full_like(t, 0.5), t))  # ties away from zero
    return h.to(s["res"].dtype), (q.float() * d).half().view(c["M"], -1)


def _plain_weights(w, kind):
    """fp32 weights [N][K] of the packed blocks."""
    N, nb = w.shape[:2]
    if kind == "q4k":
        d = w[:, :, 0:4].contiguous().view(torch.float16).float()  # d, dmin
        b = w[:, :, 4:16].int()
        sc = torch.cat([b[:, :, 0:4] & 63, (b[:, :, 8:12] & 15) | ((b[:, :, 0:4] >> 6) << 4)], 2)
        mn = torch.cat([b[:, :, 4:8] & 63, (b[:, :, 8:12] >> 4) | ((b[:, :, 4:8] >> 6) << 4)], 2)
        qs = w[:, :, 16:].view(N, nb, 4, 1, 32)
        q = torch.cat([qs & 15, qs >> 4], 3).view(N, nb, 8, 32).float()
        w32 = (d[:, :, 0:1] * sc.float())[..., None] * q - (d[:, :, 1:2] * mn.float())[..., None]
    else:
        d = w[:, :, 208:210].contiguous().view(torch.float16).float()
        sc = w[:, :, 192:208].contiguous().view(torch.int8).float()
        ql = w[:, :, :128].view(N, nb, 2, 2, 32)
        qh = w[:, :, 128:192].view(N, nb, 2, 1, 32)
        low = torch.cat([ql & 15, ql >> 4], 3)                                             # four 32s of each half
        high = torch.cat([qh & 3, (qh >> 2) & 3, (qh >> 4) & 3, qh >> 6], 3)
        q = (low | (high << 4)).view(N, nb, 16, 16).float() - 32.0
        w32 = (d * sc)[..., None] * q
    return w32.view(N, nb * 256)


def _plain_q8mm(s, c):
    x = (s["xq"].view(-1, 32).float() * s["xd"].view(-1, 1)).view(-1)
    return [_plain_weights(w, kind) @ x for w, (kind, _) in zip(s["w"], _problems(c))]


def _plain_rotate(x, cos, sin, n_rot, half):
    """x [M][heads][D] fp32 with its first n_rot dimensions turned."""
    if half:
        a, b = x[..., : n_rot // 2], x[..., n_rot // 2: n_rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = x[..., 0:n_rot:2], x[..., 1:n_rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, x[..., n_rot:]], -1)


def _plain_rope(s, c):
    M, p = c["M"], c["pos0"]
    angle = torch.arange(p, p + M, device="cuda", dtype=torch.float64)[:, None] * s["inv_freq"]
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    s["kc"][:, p: p + M] = _plain_rotate(s["k"], cos, sin, c["n_rot"], c["half"]).half().transpose(0, 1)
    s["vc"][:, p: p + M] = s["v"].half().transpose(0, 1)
    return _plain_rotate(s["q"], cos, sin, c["n_rot"], c["half"]).half(), s["kc"], s["vc"]


def _seen(c):
    """(sinks, first): the call's queries see positions 0 .. sinks - 1 and some of first .. pos0 + M - 1."""
    first = max(0, c["pos0"] - c["window"] + 1)
    return min(c["sinks"], first), first


def _plain_attn(s, c):
    M, H, Hkv, p = c["M"], c["H"], c["Hkv"], c["pos0"]
    G = H // Hkv
    sinks, first = _seen(c)
    at = torch.cat([torch.arange(sinks, device="cuda"), torch.arange(first, p + M, device="cuda")])
    k, v = s["kc"][:, at].float(), s["vc"][:, at].float()
    q = s["q"].float().view(M, Hkv, G, 128).permute(1, 2, 0, 3).reshape(Hkv, G * M, 128)
    z = (q @ k.transpose(1, 2)).view(Hkv, G, M, -1) * (1 / math.sqrt(128))
    i = torch.arange(p, p + M, device="cuda")[:, None]
    z = z.masked_fill(~((at <= i) & ((at > i - c["window"]) | (at < c["sinks"]))), -math.inf)
    e = torch.exp(z - z.amax(-1, keepdim=True))
    o = (e / e.sum(-1, keepdim=True)).view(Hkv, G * M, -1) @ v
    return o.view(Hkv, G, M, 128).permute(2, 0, 1, 3).reshape(M, H, 128).half()


def _plain_logp(s, c):
    x = s["x"]
    m = x.amax(1, keepdim=True)
    z = x - m
    e = torch.exp(z)
    S = e.sum(1, keepdim=True)
    log_s = torch.log(S)
    lp = z.gather(1, s["tok"].long()[:, None]) - log_s
    ent = log_s - torch.where(e > 0, e * z, torch.zeros_like(e)).sum(1, keepdim=True) / S
    # order by value, then by the lower index: one integer key
    b = x.view(torch.int32)
    key = torch.where(b < 0, b ^ 0x7FFFFFFF, b).long() * 2**32 + (2**32 - 1 - torch.arange(c["V"], device="cuda"))
    ids = 2**32 - 1 - (torch.topk(key, c["top"], 1).values & (2**32 - 1))
    return lp.view(-1), ent.view(-1), ids.to(torch.int32), z.gather(1, ids) - log_s


# ---------------------------------------------------------------------------
# The library's calls
# ---------------------------------------------------------------------------
def _own(s, c):
    import quantized_q4_matmul_gb300 as qk
    if c["op"] == "norm":
        if not c["q8"]:
            qk.qk_add_rmsnorm(s["res"], s["delta"], s["gamma"], EPS, s["res_out"], s["xhat"], c["M"], c["K"])
            return s["res_out"], s["xhat"]
        qk.qk_add_rmsnorm_q8(s["res"], s["delta"], s["gamma"], EPS, s["res_out"], s["xq"], s["xd"], c["M"], c["K"])
        return s["res_out"], (s["xq"].view(c["M"], -1, 32) * s["xd"][..., None]).half().view(c["M"], -1)
    if c["op"] == "q8mm":
        qk.qk_matmul_batch_q8([dict(qtype=kind, blocks=w, x_q8=s["xq"], x_d=s["xd"], y=y, M=1, N=N, K=c["K"])
                               for (kind, N), w, y in zip(_problems(c), s["w"], s["y"])])
        return [y.view(-1) for y in s["y"]]
    if c["op"] == "rope":
        qk.qk_rope_kv_append(s["q"], s["k"], s["v"], s["inv_freq"], s["qo"], s["kc"], s["vc"], c["M"], c["H"], c["Hkv"],
                             c["D"], c["n_rot"], c["pos0"], c["L_max"],
                             layout=qk.QK_ROPE_HALF if c["half"] else qk.QK_ROPE_INTERLEAVED)
        return s["qo"], s["kc"], s["vc"]
    if c["op"] == "attn":
        qk.qk_gqa_attention_window(s["q"], s["kc"], s["vc"], s["out"], c["M"], c["H"], c["Hkv"], 128, c["pos0"],
                                   c["pos0"] + c["M"] + 3, 1 / math.sqrt(128), c["window"], c["sinks"])
        return s["out"]
    qk.qk_logprobs(s["x"], s["tok"], s["lp"], s["ent"], c["top"], s["ids"], s["tlp"], c["M"], c["V"])
    return s["lp"], s["ent"], s["ids"], s["tlp"]


def run(state):
    c = state["c"]
    if own:
        return _own(state, c)
    return {"norm": _plain_norm, "q8mm": _plain_q8mm, "rope": _plain_rope, "attn": _plain_attn,
            "logp": _plain_logp}[c["op"]](state, c)


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] == "norm":
        r = 4 if c["res32"] else 2
        return {"bytes": c["M"] * c["K"] * (2 * r + 4 + (1 + 4 / 32 if c["q8"] else 2)) + 2 * c["K"],
                "flops": 6 * c["M"] * c["K"]}
    if c["op"] == "q8mm":
        K = c["K"]
        return {"bytes": sum(N * (K // 256) * BLOCK[kind] + 4 * N for kind, N in _problems(c)) + K + K // 8,
                "flops": sum(2 * N * K for _, N in _problems(c))}
    if c["op"] == "rope":
        n = c["M"] * (c["H"] + 2 * c["Hkv"]) * c["D"]
        return {"bytes": 6 * n + 4 * c["n_rot"], "flops": 3 * c["M"] * (c["H"] + c["Hkv"]) * c["n_rot"]}
    if c["op"] == "attn":
        M, p = c["M"], c["pos0"]
        sinks, first = _seen(c)
        pairs = 0
        for i in range(p, p + M):
            lo = max(0, i - c["window"] + 1)
            pairs += i + 1 - lo + min(c["sinks"], lo)
        return {"bytes": 4 * M * c["H"] * 128 + (sinks + p + M - first) * c["Hkv"] * 128 * 4,
                "flops": 4 * 128 * c["H"] * pairs}
    return {"bytes": 4 * c["M"] * c["V"] + c["M"] * (12 + 8 * c["top"]), "flops": 5 * c["M"] * c["V"]}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_block_weights(w, kind):
    """Weights of packed blocks [n][bytes] in 64 bits, one output position at a time from the block format."""
    w = w.long()

    def half(lo):
        return (w[:, lo] | (w[:, lo + 1] << 8)).to(torch.int16).view(torch.float16).double()

    out = torch.empty(w.shape[0], 256, dtype=torch.float64, device=w.device)
    if kind == "q4k":
        for j in range(8):  # sub-block of 32
            if j < 4:
                sc, mn = w[:, 4 + j] % 64, w[:, 8 + j] % 64
            else:
                sc = w[:, 8 + j] % 16 + 16 * (w[:, j] // 64)
                mn = w[:, 8 + j] // 16 + 16 * (w[:, 4 + j] // 64)
            byte = w[:, 16 + 32 * (j // 2): 48 + 32 * (j // 2)]
            q = byte // 16 if j % 2 else byte % 16
            out[:, 32 * j: 32 * j + 32] = (half(0) * sc)[:, None] * q - (half(2) * mn)[:, None]
        return out
    for j in range(8):  # 32 weights: half j // 4, quarter j % 4
        h, r = j // 4, j % 4
        byte = w[:, 64 * h + 32 * (r % 2): 64 * h + 32 * (r % 2) + 32]
        low = byte // 16 if r >= 2 else byte % 16
        high = (w[:, 128 + 32 * h: 160 + 32 * h] // 4**r) % 4
        sc = w[:, 192 + 2 * j: 194 + 2 * j]
        sc = torch.where(sc > 127, sc - 256, sc).repeat_interleave(16, 1)
        out[:, 32 * j: 32 * j + 32] = half(208)[:, None] * sc * (low + 16 * high - 32)
    return out


def _exact_q8mm(s, c):
    x = s["xq"].double().view(-1) * s["xd"].double().view(-1).repeat_interleave(32)
    ys = []
    for (kind, N), w in zip(_problems(c), s["w"]):
        y = torch.empty(N, dtype=torch.float64, device="cuda")
        rows = max(1, 2**24 // c["K"])
        for a in range(0, N, rows):
            part = w[a: a + rows]
            y[a: a + rows] = _exact_block_weights(part.reshape(-1, BLOCK[kind]), kind).view(part.shape[0], c["K"]).mv(x)
        ys.append(y)
    return ys


def _exact_norm(s, c):
    h = s["res"].double() + s["delta"].double()
    x = h * (h.square().sum(1, keepdim=True) / c["K"] + EPS).rsqrt() * s["gamma"].double()
    if not c["q8"]:
        return h, x
    b = x.half().double().unflatten(1, (-1, 32))  # the int8 values are those of the fp16 activations
    d = b.abs().max(2, keepdim=True).values / 127
    q = torch.where(d > 0, (b / d).abs() + 0.5, 0.0).floor() * b.sign()
    return h, (q * d).flatten(1)


def _exact_rope(s, c):
    n, p = c["n_rot"], c["pos0"]
    kc, vc = s["kc"].double(), s["vc"].double()
    f = _inv_freq(n, c["banded"]).cuda()
    w = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                    torch.arange(p, p + c["M"], device="cuda").double().outer(f)).unsqueeze(1)

    def turn(x):
        x = x.double().clone()
        first = slice(0, n // 2) if c["half"] else slice(0, n, 2)
        second = slice(n // 2, n) if c["half"] else slice(1, n, 2)
        z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * w
        x[..., first], x[..., second] = z.real, z.imag
        return x

    kc[:, p: p + c["M"]] = turn(s["k"]).permute(1, 0, 2)
    vc[:, p: p + c["M"]] = s["v"].double().permute(1, 0, 2)
    return turn(s["q"]), kc, vc


def _exact_attn(s, c):
    M, H, Hkv, p = c["M"], c["H"], c["Hkv"], c["pos0"]
    out = torch.empty(M, H, 128, dtype=torch.float64, device="cuda")
    for a in range(0, M, 256):  # 256 queries against every position that one of them may see
        b = min(M, a + 256)
        lo = max(0, p + a - c["window"] + 1)
        n = p + b
        pos = torch.arange(lo, n, device="cuda")
        pos = torch.cat([torch.arange(min(c["sinks"], lo), device="cuda"), pos])
        back = torch.arange(p + a, n, device="cuda")[:, None] - pos
        hidden = (back < 0) | ((back >= c["window"]) & (pos >= c["sinks"]))
        for h in range(H):
            k, v = s["kc"][h * Hkv // H, pos].double(), s["vc"][h * Hkv // H, pos].double()
            z = s["q"][a:b, h].double() @ k.T / 128**0.5
            z[hidden] = -math.inf
            out[a:b, h] = torch.softmax(z, 1) @ v
    return out


def _exact_logp(s, c):
    lp, ent, ids, tlp = [], [], [], []
    for a in range(0, c["M"], 64):
        p = torch.log_softmax(s["x"][a: a + 64].double(), 1)
        lp.append(p.gather(1, s["tok"][a: a + 64].long()[:, None])[:, 0])
        ent.append(-torch.special.xlogy(p.exp(), p.exp()).sum(1))
        order = s["x"][a: a + 64].sort(dim=1, descending=True, stable=True).indices[:, : c["top"]]
        ids.append(order.to(torch.int32))
        tlp.append(p.gather(1, order))
    return torch.cat(lp), torch.cat(ent), torch.cat(ids), torch.cat(tlp)


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "q8mm": _exact_q8mm, "rope": _exact_rope, "attn": _exact_attn,
            "logp": _exact_logp}[case["op"]](s, s["c"])
