"""How far f32 rows under a window may be from the definition in 64 bits: the
2-norm of the difference over that of the result, which the header states and the
tolerances of single elements (1e-5 + 1e-4 |ref|) do not reach.

Prompts.  An accumulator of the tensor cores that took j times 64 tokens is some
j 1.3e-7 of the result off, and f32 logits, weights and sums leave 3e-7 to 5e-7
beside that.  It is emptied every 384 tokens, so 6 x 1.3e-7 and 5e-7 together, the
root of their squares, are 0.93e-6: the header's 1e-6.  Emptied every 512 tokens it
is 1.15e-6, and 1.6e-6 after 768.

Single tokens.  A warp adds the products of 32 tokens to an f32 sum, one after the
other.  A rounding is off by 2^-24 / sqrt(3) (root mean square) of the power of two at or
below the sum, which is 0.7 of the sum on average: 2.4e-8 of it.  With T tokens, T / 32
sums that grow evenly (V with a mean) have T / 96 times its square, sums that walk (V
around zero) T / 64: 3.0e-9 sqrt(T) at most.  The weights' own sum has 4 additions per 32
tokens in each of 8 parts: 2.4e-8 sqrt(T / 24 / 8) = 1.8e-9 sqrt(T).  Together below 4e-9
sqrt(T).
  Beside that stand the logits.  An error of theirs moves the result by as much of it (both
are sums of the same weights over values without order).  One is D / 16 steps of the
tensor cores, each of which cuts 17 terms of either sign at 2^-25 of the power of two at or
below their largest and the sum at 2^-23: 2^-23 sqrt(17 / 3 / 16 + 7 / 32) = 9.0e-8 of the
logits' spread, taken as large in every step as at the end.  To that come q in 22 bits
(0.7e-7), three products (0.4e-7), the distance to the largest, a number of up to 8
(0.7e-7), and its power of two (1e-7): 1.5e-7 together.  With normal q and K the logits that
have the weight lie around 1 with a spread of 1, so their mean square is 2:
sqrt(2) sqrt(D / 16 (9.0e-8)^2 + (1.5e-7)^2).
  Sums left to the tensor cores would lose about 1e-7 of themselves with every 16 tokens.
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


@gpu
@pytest.mark.parametrize("mean", [0.0, 1.0])
@pytest.mark.parametrize("tokens", [100, 2048, 32768])
@pytest.mark.parametrize("H,D,warps", [(4, 64, 12), (8, 128, 12), (4, 256, 4), (16, 128, 8), (16, 256, 4)])
def test_single_tokens(H, D, warps, tokens, mean):
    """As many sequences (of the same pages) as the GPU has streams of warps: each walks a whole window."""
    import torch
    import int8_paged_kv_gb300 as pk
    S = warps * torch.cuda.get_device_properties(0).multi_processor_count
    gen = torch.Generator(device="cuda").manual_seed(D + tokens)
    pages = -(-tokens // BLOCK)
    kc, vc = quantised(gen, 1, pages, D, 0.0), quantised(gen, 1, pages, D, mean)
    q = torch.randn((S, H, D), device="cuda", generator=gen)
    i32 = dict(dtype=torch.int32, device="cuda")
    got = pk.pa_q8_window_decode(torch.empty_like(q), q, kc, vc, torch.arange(pages, **i32)[None].repeat(S, 1),
                                 torch.full((S,), tokens, **i32), num_kv_heads=1, block_size=BLOCK, window=tokens,
                                 scale=D ** -0.5)
    at = torch.arange(0, S, S // 32, device="cuda")
    logits = math.sqrt(2 * (D / 16 * 9.0e-8 ** 2 + 1.5e-7 ** 2))
    bound = math.hypot(logits, 4e-9 * math.sqrt(tokens))
    assert off(got[at], q[at], kc, vc, torch.full_like(at, tokens - 1), tokens, tokens, 0) <= bound


@gpu
@pytest.mark.parametrize("window", [368, 376, 379, 380, 384, 385, 760, 768, 769])
@pytest.mark.parametrize("H,Hk,D", [(16, 1, 256), (8, 2, 128), (8, 2, 64)])
def test_prompts_where_the_first_sums_begin(H, Hk, D, window):
    """Windows at which the workspace gets room for sums and accumulators are first emptied into them; what
    stands behind a workspace of the size asked for stays."""
    import torch
    import int8_paged_kv_gb300 as pk
    rows, tokens = 200, 1000
    gen = torch.Generator(device="cuda").manual_seed(D + window)
    pages = -(-tokens // BLOCK)
    kc, vc = quantised(gen, Hk, pages, D, 0.0), quantised(gen, Hk, pages, D, 0.0)
    q = torch.randn((rows, H, D), device="cuda", generator=gen)
    i32 = dict(dtype=torch.int32, device="cuda")
    need = pk.pa_q8_window_prefill_workspace_size(rows, 1, H, Hk, D, BLOCK, pages, window, 0, q.dtype)
    memory = torch.full((need + (1 << 20),), 0xA5, dtype=torch.uint8, device="cuda")
    got = pk.pa_q8_window_prefill(torch.empty_like(q), q, kc, vc, torch.arange(pages, **i32)[None].contiguous(),
                                  torch.tensor([tokens], **i32), torch.tensor([0, rows], **i32), num_kv_heads=Hk,
                                  block_size=BLOCK, window=window, scale=D ** -0.5, workspace=memory[:need])
    at = torch.arange(rows, device="cuda")
    assert off(got, q, kc, vc, tokens - rows + at, tokens, window, 0) <= 1e-6
    assert bool((memory[need:] == 0xA5).all())
