"""The operators of a decoder step with a 4-bit KV cache, from the QKV projections' outputs to the next token:
cases, plain forms and the library's calls.

  append  RMSNorm of each q and k head, rotary positions, and the new k / v rows into the KV cache (fp16 or 4 bits)
  attn4   grouped-query attention over the 4-bit cache, with an optional sliding window and sinks
  sample  a token from logits and a given random number: temperature, top-k, top-p, min-p

``own`` False: elementary torch operations.  ``own`` True: the calls of quantized_q4_matmul_gb300.

The 4-bit cache holds a head's row of one position in groups of 32 values: v = d q + m with q in 0 .. 15, d and m fp16;
byte j of a group has value 2j in its low and 2j + 1 in its high half.  m is the group's least value rounded to fp16, d
the fp16 nearest to (greatest value - m) / 15, q the nearest to (x - m) / d.
"""
import math
import struct

import torch

own = False

EPS = 1e-6
LOG_NONE = 1 << 30  # a window that no sequence here reaches: plain causal attention


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # a decode step far into a long context, fp16 cache: all latency
        dict(name="append one token", op="append", q4=False, M=1, H=24, Hkv=8, D=128, n_rot=128, half=True, q_norm=True,
             k_norm=True, pos0=31000, L_max=32768),
        # a prompt into an fp16 cache, ragged, the end of each head not turning
        dict(name="append prompt", op="append", q4=False, M=2047, H=32, Hkv=4, D=128, n_rot=96, half=False, q_norm=True,
             k_norm=True, pos0=5, L_max=4096),
        # a decode step with a 4-bit cache
        dict(name="append 4-bit one token", op="append", q4=True, M=1, H=24, Hkv=8, D=128, n_rot=128, half=True,
             q_norm=True, k_norm=True, pos0=300, L_max=512),
        # a ragged chunk of a model without the norms, into a 4-bit cache
        dict(name="append 4-bit chunk", op="append", q4=True, M=333, H=32, Hkv=8, D=64, n_rot=64, half=False, q_norm=False,
             k_norm=False, pos0=77, L_max=1000),
        # a long prompt into a 4-bit cache: HBM
        dict(name="append 4-bit prompt", op="append", q4=True, M=4095, H=24, Hkv=8, D=128, n_rot=128, half=True, q_norm=True,
             k_norm=True, pos0=0, L_max=4200),
        # a decode step early in a conversation: latency
        dict(name="attention 4-bit short", op="attn4", M=1, H=32, Hkv=8, pos0=500, window=LOG_NONE, sinks=0),
        # a decode step at the end of a long document: the cache's bytes
        dict(name="attention 4-bit long", op="attn4", M=1, H=24, Hkv=8, pos0=65535, window=LOG_NONE, sinks=0),
        # a few drafted tokens checked at once, with a sliding window and sinks
        dict(name="attention 4-bit draft", op="attn4", M=5, H=24, Hkv=8, pos0=20001, window=8192, sinks=4),
        # a chunk of a prompt after cached positions
        dict(name="attention 4-bit chunk", op="attn4", M=1023, H=24, Hkv=8, pos0=7001, window=LOG_NONE, sinks=0),
        # a decode step's token with the usual settings of a chat
        dict(name="sample one token", op="sample", M=1, V=128256, T=0.8, top_k=40, top_p=0.95, min_p=0.05, banned=0.02),
        # nucleus sampling of several continuations at once
        dict(name="sample nucleus", op="sample", M=64, V=128256, T=1.0, top_k=0, top_p=0.9, min_p=0.0, banned=0.0),
        # the whole distribution of many rows
        dict(name="sample all", op="sample", M=512, V=128256, T=1.3, top_k=0, top_p=1.0, min_p=0.0, banned=0.0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


_HEADS = ((24, 8), (32, 8), (32, 4), (8, 8), (6, 2), (4, 1))


def draw(rng):
    op = rng.choice(("append", "append", "attn4", "attn4", "sample"))
    if op == "append":
        H, Hkv = rng.choice(_HEADS)
        q4 = rng.random() < 0.6
        D = rng.choice((32, 64, 96, 128, 256) if q4 else (64, 72, 80, 128, 256))
        M = 1 if rng.random() < 0.3 else _log_int(rng, 2, 1500)
        pos0 = rng.choice((0, _log_int(rng, 1, 2000 if q4 else 20000)))
        return dict(op=op, q4=q4, M=M, H=H, Hkv=Hkv, D=D, n_rot=rng.choice((D, D, 2 * rng.randint(0, D // 2))),
                    half=rng.random() < 0.5, q_norm=rng.random() < 0.7, k_norm=rng.random() < 0.7, pos0=pos0,
                    L_max=pos0 + M + rng.randint(0, 300))
    if op == "attn4":
        H, Hkv = rng.choice(_HEADS)
        kind = rng.random()
        M = 1 if kind < 0.35 else _log_int(rng, 2, 16) if kind < 0.6 else _log_int(rng, 17, 600)
        pos0 = rng.choice((0, _log_int(rng, 1, 60000 if M == 1 else 20000 if M <= 16 else 6000)))
        window = rng.choice((LOG_NONE, _log_int(rng, 1, 8000)))
        return dict(op=op, M=M, H=min(H, 24), Hkv=Hkv if H <= 24 else 8, pos0=pos0, window=window,
                    sinks=0 if window == LOG_NONE else rng.choice((0, _log_int(rng, 1, 80))))
    return dict(op=op, M=_log_int(rng, 1, 300), V=_log_int(rng, 500, 150000),
                T=0.0 if rng.random() < 0.1 else round(math.exp(rng.uniform(math.log(0.3), math.log(3.0))), 3),
                top_k=rng.choice((0, _log_int(rng, 1, 400))), top_p=rng.choice((1.0, round(rng.uniform(0.2, 0.99), 3))),
                min_p=rng.choice((0.0, 0.0, round(rng.uniform(0.005, 0.3), 4))), banned=rng.choice((0.0, 0.05)))


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _f32(x):
    """The value that a C float argument holds."""
    return struct.unpack("f", struct.pack("f", x))[0]


def _cache4(g, Hkv, L, D):
    """A cache that holds quantized rows: bytes [Hkv][L][D / 2] and (d, m) fp16 [Hkv][L][D / 32][2]."""
    q4 = torch.randint(0, 256, (Hkv, L, D // 2), generator=g, device="cuda", dtype=torch.uint8)
    dm = torch.empty(Hkv, L, D // 32, 2, device="cuda")
    dm[..., 0] = 0.2 + 0.15 * torch.rand(Hkv, L, D // 32, generator=g, device="cuda")
    dm[..., 1] = -7.5 * dm[..., 0] + 0.3 * _randn(g, Hkv, L, D // 32)
    return q4, dm.half()


def prepare(case, seed):
    g, c = _gen(seed), dict(case)
    s = {"c": c}
    if c["op"] == "append":
        M, H, Hkv, D, L = c["M"], c["H"], c["Hkv"], c["D"], c["L_max"]
        s["q"], s["k"], s["v"] = 3 * _randn(g, M, H, D), 2 * _randn(g, M, Hkv, D), _randn(g, M, Hkv, D)
        s["q_gamma"] = (1 + 0.2 * _randn(g, D)).half() if c["q_norm"] else None
        s["k_gamma"] = (1 + 0.2 * _randn(g, D)).half() if c["k_norm"] else None
        f = 500000.0 ** (-torch.arange(0, c["n_rot"], 2, dtype=torch.float64) / max(1, c["n_rot"]))
        s["inv_freq"] = f.cuda()
        s["qo"] = torch.empty(M, H, D, dtype=torch.float16, device="cuda")
        if c["q4"]:
            s["k4"], s["kdm"] = _cache4(g, Hkv, L, D)
            s["v4"], s["vdm"] = _cache4(g, Hkv, L, D)
            s["k16"] = torch.empty(Hkv, L, D, dtype=torch.float16, device="cuda")
            s["v16"] = torch.empty(Hkv, L, D, dtype=torch.float16, device="cuda")
        else:
            s["kc"], s["vc"] = _randn(g, Hkv, L, D).half(), _randn(g, Hkv, L, D).half()
    elif c["op"] == "attn4":
        M, H, Hkv, n = c["M"], c["H"], c["Hkv"], c["pos0"] + c["M"]
        s["q"] = (1.5 * _randn(g, M, H, 128)).half()
        s["k4"], s["kdm"] = _cache4(g, Hkv, n + 3, 128)
        s["v4"], s["vdm"] = _cache4(g, Hkv, n + 3, 128)
        s["out"] = torch.empty(M, H, 128, dtype=torch.float16, device="cuda")
        # what a program keeps for the longest call of many tokens: fp16 rows of the positions that it sees
        sinks, first = _seen(c)
        s["scratch"] = torch.empty(2 * Hkv * (sinks + n - first) * 128, dtype=torch.float16, device="cuda")
    else:
        M, V = c["M"], c["V"]
        x = 2.5 * _randn(g, M, V)
        if c["banned"] > 0:
            x[torch.rand(M, V, generator=g, device="cuda") < c["banned"]] = -math.inf
        # a few likely tokens in each row, from sure to unsure
        at = torch.randint(0, V, (M, 12), generator=g, device="cuda")
        x.scatter_(1, at, 6 + 7 * torch.rand(M, 12, generator=g, device="cuda"))
        s["x"] = x
        s["u"] = torch.rand(M, generator=g, device="cuda")
        s["token"] = torch.empty(M, dtype=torch.int32, device="cuda")
        s["kept"] = torch.empty(M, dtype=torch.int32, device="cuda")
        s["lp"] = torch.empty(M, device="cuda")
    return s


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------
def _plain_head_norm(x, gamma):
    if gamma is None:
        return x
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * gamma.float()


def _plain_rotate(x, cos, sin, n_rot, half):
    """x [M][heads][D] fp32 with its first n_rot dimensions turned."""
    if half:
        a, b = x[..., : n_rot // 2], x[..., n_rot // 2: n_rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = x[..., 0:n_rot:2], x[..., 1:n_rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, x[..., n_rot:]], -1)


def _plain_pack(x):
    """x fp32 [..., D] in 4 bits: bytes [..., D / 2] and (d, m) fp16 [..., D / 32, 2]."""
    b = x.unflatten(-1, (-1, 32))
    m = b.amin(-1, keepdim=True).half()
    d = ((b.amax(-1, keepdim=True) - m.float()).clamp(min=0) / 15).half()
    q = torch.where(d > 0, torch.round((b - m.float()) / d.float()).clamp(0, 15), 0.0).to(torch.uint8)
    return (q[..., 0::2] | (q[..., 1::2] << 4)).flatten(-2), torch.cat([d, m], -1)


def _plain_unpack(q4, dm):
    """fp32 values of packed rows."""
    b = q4.unflatten(-1, (-1, 16))
    q = torch.stack([b & 15, b >> 4], -1).flatten(-2).float()
    return (q * dm[..., 0:1].float() + dm[..., 1:2].float()).flatten(-2)


def _plain_append(s, c):
    M, p = c["M"], c["pos0"]
    angle = torch.arange(p, p + M, device="cuda", dtype=torch.float64)[:, None] * s["inv_freq"]
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    q = _plain_rotate(_plain_head_norm(s["q"], s["q_gamma"]), cos, sin, c["n_rot"], c["half"]).half()
    k = _plain_rotate(_plain_head_norm(s["k"], s["k_gamma"]), cos, sin, c["n_rot"], c["half"])
    if not c["q4"]:
        s["kc"][:, p: p + M] = k.half().transpose(0, 1)
        s["vc"][:, p: p + M] = s["v"].half().transpose(0, 1)
        return q, s["kc"], s["vc"]
    s["k4"][:, p: p + M], s["kdm"][:, p: p + M] = _plain_pack(k.transpose(0, 1))
    s["v4"][:, p: p + M], s["vdm"][:, p: p + M] = _plain_pack(s["v"].transpose(0, 1))
    return q, _plain_unpack(s["k4"], s["kdm"]).half(), _plain_unpack(s["v4"], s["vdm"]).half()


def _seen(c):
    """(sinks, first): the call's queries see positions 0 .. sinks - 1 and some of first .. pos0 + M - 1."""
    first = max(0, c["pos0"] - c["window"] + 1)
    return min(c["sinks"], first), first


def _plain_attn4(s, c):
    M, H, Hkv, p = c["M"], c["H"], c["Hkv"], c["pos0"]
    G = H // Hkv
    sinks, first = _seen(c)
    at = torch.cat([torch.arange(sinks, device="cuda"), torch.arange(first, p + M, device="cuda")])
    k, v = _plain_unpack(s["k4"][:, at], s["kdm"][:, at]), _plain_unpack(s["v4"][:, at], s["vdm"][:, at])
    q = s["q"].float().view(M, Hkv, G, 128).permute(1, 2, 0, 3).reshape(Hkv, G * M, 128)
    z = (q @ k.transpose(1, 2)).view(Hkv, G, M, -1) * (1 / math.sqrt(128))
    i = torch.arange(p, p + M, device="cuda")[:, None]
    z = z.masked_fill(~((at <= i) & ((at > i - c["window"]) | (at < c["sinks"]))), -math.inf)
    e = torch.exp(z - z.amax(-1, keepdim=True))
    o = (e / e.sum(-1, keepdim=True)).view(Hkv, G * M, -1) @ v
    return o.view(Hkv, G, M, 128).permute(2, 0, 1, 3).reshape(M, H, 128).half()


def _plain_sample(s, c):
    x = s["x"]
    top, order = torch.sort(x, dim=1, descending=True, stable=True)  # equal logits: the lower token first
    if c["T"] == 0:
        return order[:, 0].to(torch.int32), torch.zeros_like(s["u"]), torch.ones_like(order[:, 0], dtype=torch.int32)
    w = torch.exp((top.double() - top[:, :1].double()) / _f32(c["T"]))
    cum = torch.cumsum(w, 1)
    n = (top > -math.inf).sum(1, keepdim=True)  # banned tokens are never kept
    if c["top_k"] > 0:
        n = n.clamp(max=c["top_k"])
    n_p = (cum < _f32(c["top_p"]) * cum.gather(1, n - 1)).sum(1, keepdim=True) + 1
    if c["top_p"] < 1:
        n = torch.minimum(n, n_p)
    n = torch.minimum(n, (w >= _f32(c["min_p"])).sum(1, keepdim=True))
    total = cum.gather(1, n - 1)
    j = torch.minimum((cum <= s["u"].double()[:, None] * total).sum(1, keepdim=True), n - 1)
    lp = torch.log(w.gather(1, j) / total)
    return order.gather(1, j)[:, 0].to(torch.int32), lp[:, 0].float(), n[:, 0].to(torch.int32)


# ---------------------------------------------------------------------------
# The library's calls
# ---------------------------------------------------------------------------
def _own(s, c):
    import quantized_q4_matmul_gb300 as qk
    if c["op"] == "append":
        sizes = (c["M"], c["H"], c["Hkv"], c["D"], c["n_rot"], c["pos0"], c["L_max"])
        layout = qk.QK_ROPE_HALF if c["half"] else qk.QK_ROPE_INTERLEAVED
        if not c["q4"]:
            qk.qk_norm_rope_kv_append(s["q"], s["k"], s["v"], s["q_gamma"], s["k_gamma"], EPS, s["inv_freq"], s["qo"],
                                      s["kc"], s["vc"], *sizes, layout=layout)
            return s["qo"], s["kc"], s["vc"]
        qk.qk_norm_rope_kv_append_q4(s["q"], s["k"], s["v"], s["q_gamma"], s["k_gamma"], EPS, s["inv_freq"], s["qo"],
                                     s["k4"], s["kdm"], s["v4"], s["vdm"], *sizes, layout=layout)
        qk.qk_dequant_kv_q4(s["k4"], s["kdm"], s["k16"], c["Hkv"], c["D"], 0, c["L_max"], c["L_max"])
        qk.qk_dequant_kv_q4(s["v4"], s["vdm"], s["v16"], c["Hkv"], c["D"], 0, c["L_max"], c["L_max"])
        return s["qo"], s["k16"], s["v16"]
    if c["op"] == "attn4":
        qk.qk_gqa_attention_q4(s["q"], s["k4"], s["kdm"], s["v4"], s["vdm"], s["out"], c["M"], c["H"], c["Hkv"], 128,
                               c["pos0"], c["pos0"] + c["M"] + 3, 1 / math.sqrt(128), c["window"], c["sinks"],
                               scratch=s["scratch"])
        return s["out"]
    qk.qk_sample(s["x"], s["u"], s["token"], s["lp"], s["kept"], c["M"], c["V"], temperature=c["T"], top_k=c["top_k"],
                 top_p=c["top_p"], min_p=c["min_p"])
    return s["token"], s["lp"], s["kept"]


def run(state):
    c = state["c"]
    if own:
        return _own(state, c)
    return {"append": _plain_append, "attn4": _plain_attn4, "sample": _plain_sample}[c["op"]](state, c)


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] == "append":
        M, H, Hkv, D = c["M"], c["H"], c["Hkv"], c["D"]
        n = M * D
        rows = 2 * Hkv * n
        heads = (H if c["q_norm"] else 0) + (Hkv if c["k_norm"] else 0)
        held = rows * 5 / 8 if c["q4"] else rows * 2
        # the 4-bit cache's values, which the pass returns, are read back and written as fp16
        shown = 2 * Hkv * c["L_max"] * D * (5 / 8 + 2) if c["q4"] else 0
        return {"bytes": 4 * (H * n + rows) + 2 * H * n + held + 4 * c["n_rot"] + shown,
                "flops": 3 * M * (H + Hkv) * c["n_rot"] + 4 * heads * n + (6 * rows if c["q4"] else 0)}
    if c["op"] == "attn4":
        M, p = c["M"], c["pos0"]
        sinks, first = _seen(c)
        pairs = 0
        for i in range(p, p + M):
            lo = max(0, i - c["window"] + 1)
            pairs += i + 1 - lo + min(c["sinks"], lo)
        return {"bytes": 4 * M * c["H"] * 128 + (sinks + p + M - first) * c["Hkv"] * 2 * 80,
                "flops": 4 * 128 * c["H"] * pairs}
    return {"bytes": 4 * c["M"] * c["V"] + 16 * c["M"], "flops": 4 * c["M"] * c["V"]}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_values(q4, dm):
    """The values of packed rows, one place in a byte after the other."""
    q = torch.empty(*q4.shape[:-1], 2 * q4.shape[-1], dtype=torch.float64, device=q4.device)
    q[..., 0::2] = (q4 % 16).double()
    q[..., 1::2] = (q4 // 16).double()
    d, m = dm.double().unbind(-1)
    return q * d.repeat_interleave(32, -1) + m.repeat_interleave(32, -1)


def _exact_append(s, c):
    n, p, M = c["n_rot"], c["pos0"], c["M"]
    f = torch.tensor([500000.0 ** (-2 * j / n) for j in range(n // 2)], dtype=torch.float64, device="cuda")
    w = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                    torch.arange(p, p + M, device="cuda").double().outer(f)).unsqueeze(1)

    def turn(x, gamma):
        x = x.double().clone()
        if gamma is not None:
            x *= (x.square().sum(-1, keepdim=True) / c["D"] + EPS).rsqrt() * gamma.double()
        first = slice(0, n // 2) if c["half"] else slice(0, n, 2)
        second = slice(n // 2, n) if c["half"] else slice(1, n, 2)
        z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * w
        x[..., first], x[..., second] = z.real, z.imag
        return x

    q, k, v = turn(s["q"], s["q_gamma"]), turn(s["k"], s["k_gamma"]), s["v"].double()
    caches = []
    for x, held in ((k, "k"), (v, "v")):
        x = x.permute(1, 0, 2)
        if not c["q4"]:
            cache = s[held + "c"].double()
            cache[:, p: p + M] = x
        else:
            cache = _exact_values(s[held + "4"], s[held + "dm"])
            lo = torch.stack([y.min(-1).values for y in x.split(32, -1)], -1).to(torch.float16).double()
            hi = torch.stack([y.max(-1).values for y in x.split(32, -1)], -1)
            step = ((hi - lo).clamp(min=0) / 15).to(torch.float16).double()
            lo, step = lo.repeat_interleave(32, -1), step.repeat_interleave(32, -1)
            level = torch.where(step > 0, (x - lo) / step, 0.0).round().clamp(0, 15)
            cache[:, p: p + M] = level * step + lo
        caches.append(cache)
    return q, caches[0], caches[1]


def _exact_attn4(s, c):
    M, H, Hkv, p = c["M"], c["H"], c["Hkv"], c["pos0"]
    out = torch.empty(M, H, 128, dtype=torch.float64, device="cuda")
    for a in range(0, M, 256):  # 256 queries against every position that one of them may see
        b = min(M, a + 256)
        lo = max(0, p + a - c["window"] + 1)
        n = p + b
        pos = torch.cat([torch.arange(min(c["sinks"], lo), device="cuda"), torch.arange(lo, n, device="cuda")])
        back = torch.arange(p + a, n, device="cuda")[:, None] - pos
        hidden = (back < 0) | ((back >= c["window"]) & (pos >= c["sinks"]))
        for g in range(Hkv):
            k, v = _exact_values(s["k4"][g, pos], s["kdm"][g, pos]), _exact_values(s["v4"][g, pos], s["vdm"][g, pos])
            for h in range(g * (H // Hkv), (g + 1) * (H // Hkv)):
                z = s["q"][a:b, h].double() @ k.T / 128**0.5
                z[hidden] = -math.inf
                out[a:b, h] = torch.softmax(z, 1) @ v
    return out


def _exact_sample(s, c):
    tokens, lps, kept = [], [], []
    for x, u in zip(s["x"].double().cpu().unbind(0), s["u"].double().tolist()):
        x, order = torch.sort(x, descending=True, stable=True)
        if c["T"] == 0:
            tokens.append(int(order[0])), lps.append(0.0), kept.append(1)
            continue
        p = ((x[x > -math.inf] - x[0]) / _f32(c["T"])).exp()
        n = min(len(p), c["top_k"]) if c["top_k"] else len(p)
        upto = p.cumsum(0)
        if c["top_p"] < 1:
            n = min(n, 1 + int(torch.searchsorted(upto[:n], _f32(c["top_p"]) * upto[n - 1])))
        n = min(n, int((p >= _f32(c["min_p"])).sum()))
        j = min(n - 1, int(torch.searchsorted(upto[:n], u * upto[n - 1], right=True)))
        tokens.append(int(order[j])), lps.append(float(torch.log(p[j] / upto[n - 1]))), kept.append(n)
    dev = s["x"].device
    return (torch.tensor(tokens, dtype=torch.int32, device=dev), torch.tensor(lps, dtype=torch.float64, device=dev),
            torch.tensor(kept, dtype=torch.int32, device=dev))


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attn4": _exact_attn4, "sample": _exact_sample}[case["op"]](s, s["c"])
