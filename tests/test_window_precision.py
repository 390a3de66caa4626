"""How far f32 rows under a window may be from the definition in 64 bits: the
2-norm of the difference over that of the result, which the header states and the
tolerances of single elements (1e-5 + 1e-4 |ref|) do not reach.

Prompts.  An accumulator of the tensor cores that took j times 64 tokens is some
j 1.3e-7 of the result off, and f32 logits, weights and sums leave 3e-7 to 5e-7
beside that.  It is emptied every 384 tokens, so 6 x 1.3e-7 and 5e-7 together, the
root of their squares, are 0.93e-6: the header's 1e-6.  Emptied every 512 tokens it
is 1.15e-6, and 1.6e-6 after 768.
"""
import math

import pytest

from tests.test_prefill import lib  # noqa: F401  (fixture)

gpu = pytest.mark.gpu
BLOCK = 16


@pytest.fixture(autouse=True)
def _built(request):
    if "gpu" in request.keywords:
        request.getfixturevalue("lib")


def quantised(gen, kv, pages, dim, mean):
    """A cache of quantised N(mean, 1) vectors."""
    import torch
    x = torch.randn((pages, kv, BLOCK, dim), device="cuda", generator=gen) + mean
    amax = x.abs().amax(-1, keepdim=True)
    words = torch.empty((pages, kv, BLOCK, dim // 4 + 1), dtype=torch.int32, device="cuda")
    words[..., :-1] = (x * (127.0 / amax)).round_().to(torch.int8).view(torch.int32)
    words[..., -1] = (amax / 127.0).view(torch.int32)[..., 0]
    return words


def dense(words, head, tokens):
    import torch
    x = words[:, head]
    vectors = x[..., :-1].contiguous().view(torch.int8).double() * x[..., -1:].contiguous().view(torch.float32).double()
    return vectors.flatten(0, 1)[:tokens]


def off(got, q, kc, vc, places, tokens, window, sinks):
    """2-norm of the difference over that of the result; q, got: [rows, H, D], rows at `places` of one sequence."""
    import torch
    kv, dim, per = kc.shape[1], q.shape[2], q.shape[1] // kc.shape[1]
    t, wrong, all_ = torch.arange(tokens, device="cuda")[None], 0.0, 0.0
    sees = (t <= places[:, None]) & ((t > places[:, None] - window) | (t < sinks))
    for g in range(kv):
        k, v = dense(kc, g, tokens), dense(vc, g, tokens)
        for h in range(g * per, (g + 1) * per):
            z = (q[:, h].double() @ k.T * dim ** -0.5).masked_fill_(~sees, -math.inf)
            want = torch.softmax(z, -1) @ v
            wrong += float((got[:, h].double() - want).square().sum())
            all_ += float(want.square().sum())
    return math.sqrt(wrong / all_)


@gpu
@pytest.mark.parametrize("mean", [0.0, 1.0])
@pytest.mark.parametrize("window", [64, 300, 384, 500, 700, 760, 1024, 1500, 2048, 6000])
@pytest.mark.parametrize("H,Hk,D", [(16, 1, 256), (8, 2, 128), (8, 2, 64)])
def test_prompts(H, Hk, D, window, mean):
    import torch
    import int8_paged_kv_gb300 as pk
    rows, sinks = 1024, 4
    tokens = rows + window + 100
    gen = torch.Generator(device="cuda").manual_seed(D + window)
    pages = -(-tokens // BLOCK)
    kc, vc = quantised(gen, Hk, pages, D, 0.0), quantised(gen, Hk, pages, D, mean)
    q = torch.randn((rows, H, D), device="cuda", generator=gen)
    i32 = dict(dtype=torch.int32, device="cuda")
    got = pk.pa_q8_window_prefill(torch.empty_like(q), q, kc, vc, torch.arange(pages, **i32)[None].contiguous(),
                                  torch.tensor([tokens], **i32), torch.tensor([0, rows], **i32), num_kv_heads=Hk,
                                  block_size=BLOCK, window=window, num_sinks=sinks, scale=D ** -0.5)
    at = torch.arange(0, rows, 8, device="cuda")
    assert off(got[at], q[at], kc, vc, tokens - rows + at, tokens, window, sinks) <= 1e-6
