"""Integers that a C argument cannot hold are refused by the binding: ctypes takes them modulo
2^32 or 2^64, so that a top_k of 2^32 + 1 would be 1 and a window of 2^64 nothing (no GPU needed)."""
import pytest


def _calls(qk, torch):
    M, L = 3, 16
    f16 = torch.float16
    q, kv, fr = torch.zeros(M, 4, 128), torch.zeros(M, 2, 128), torch.zeros(64, dtype=torch.float64)
    g, qo, out = torch.ones(128, dtype=f16), torch.zeros(M, 4, 128, dtype=f16), torch.zeros(M, 4, 128, dtype=f16)
    k4, v4 = (torch.zeros(2, L, 64, dtype=torch.uint8) for _ in range(2))
    kd, vd = (torch.zeros(2, L, 4, 2, dtype=f16) for _ in range(2))
    kc, vc = (torch.zeros(2, L, 128, dtype=f16) for _ in range(2))
    x, u, tok = torch.zeros(M, 10), torch.zeros(M), torch.zeros(M, dtype=torch.int32)
    scratch = torch.zeros(64, dtype=torch.uint8)
    return {
        "rope": lambda pos0=0, layout=0: qk.qk_rope_kv_append(q, kv, kv, fr, qo, kc, vc, M, 4, 2, 128, 128, pos0, L,
                                                              layout=layout, stream=0),
        "append": lambda pos0=0, layout=0: qk.qk_norm_rope_kv_append(q, kv, kv, g, g, 1e-6, fr, qo, kc, vc, M, 4, 2, 128, 128,
                                                                     pos0, L, layout=layout, stream=0),
        "append4": lambda pos0=0, layout=0: qk.qk_norm_rope_kv_append_q4(q, kv, kv, g, g, 1e-6, fr, qo, k4, kd, v4, vd, M, 4, 2,
                                                                         128, 128, pos0, L, layout=layout, stream=0),
        "dequant": lambda pos0=0: qk.qk_dequant_kv_q4(k4, kd, kc, 2, 128, pos0, M, L, stream=0),
        "attention": lambda pos0=0: qk.qk_gqa_attention(qo, kc, vc, q, M, 4, 2, 128, pos0, L, 0.1, stream=0),
        "window": lambda pos0=0, window=5, sinks=0: qk.qk_gqa_attention_window(qo, kc, vc, out, M, 4, 2, 128, pos0, L, 0.1, window,
                                                                               sinks, stream=0),
        "attention4": lambda pos0=0, window=5, sinks=0: qk.qk_gqa_attention_q4(qo, k4, kd, v4, vd, out, M, 4, 2, 128, pos0, L, 0.1,
                                                                               window, sinks, scratch=scratch, stream=0),
        "scratch": lambda M=40, H=8, pos0=0, window=5, sinks=0: qk.qk_gqa_attention_q4_scratch_bytes(M, H, 2, 128, pos0, window,
                                                                                                     sinks),
        "logprobs": lambda top_n=0: qk.qk_logprobs(x, None, None, u, top_n, None, None, M, 10, stream=0),
        "sample": lambda top_k=0: qk.qk_sample(x, u, tok, None, None, M, 10, top_k=top_k, stream=0),
    }


WRAP = {"pos0": 1 << 64, "window": 1 << 64, "sinks": 1 << 64, "layout": 1 << 32, "top_k": 1 << 32, "top_n": 1 << 32, "M": 1 << 64, "H": 1 << 64}


@pytest.mark.parametrize("name,arg", [("rope", "pos0"), ("rope", "layout"), ("append", "pos0"), ("append", "layout"),
                                      ("append4", "pos0"), ("append4", "layout"), ("dequant", "pos0"), ("attention", "pos0"),
                                      ("window", "pos0"), ("window", "window"), ("window", "sinks"), ("attention4", "pos0"),
                                      ("attention4", "window"), ("attention4", "sinks"), ("scratch", "M"), ("scratch", "H"),
                                      ("scratch", "pos0"), ("scratch", "window"), ("scratch", "sinks"), ("sample", "top_k"),
                                      ("logprobs", "top_n")])
def test_integers_that_do_not_fit(qk_lib, name, arg):
    torch = pytest.importorskip("torch")
    call = _calls(qk_lib, torch)[name]
    for v in (WRAP[arg], WRAP[arg] + 1, -WRAP[arg] + 1, WRAP[arg] // 2, -WRAP[arg] // 2 - 1, 10 ** 30):
        with pytest.raises(ValueError) as e:
            call(**{arg: v})
        assert "does not fit" in str(e.value), (name, arg, v)


def test_the_largest_that_fit(qk_lib):
    """They reach the library: a top_k or window of any size up to there is "all"."""
    torch = pytest.importorskip("torch")
    calls = _calls(qk_lib, torch)
    no_device = (-4, -6, -8)
    for name, args in (("sample", dict(top_k=(1 << 31) - 1)), ("window", dict(window=(1 << 63) - 1, sinks=(1 << 63) - 1)),
                       ("attention4", dict(window=(1 << 63) - 1, sinks=(1 << 63) - 1))):
        with pytest.raises(qk_lib.QKError) as e:
            calls[name](**args)
        assert e.value.status in no_device, name
    assert calls["scratch"](window=(1 << 63) - 1) == 512 * 2 * 40
