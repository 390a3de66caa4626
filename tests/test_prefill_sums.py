"""f32 rows: what the tensor cores' accumulators lose between two additions to the
f32 sums.

An MMA adds 16 products, one for each of 16 tokens, to the accumulator.  All 17 terms
are aligned to the largest exponent and cut, toward zero, two bits below the
accumulator's last (2^-25 of the power of two at or below it), and the sum is cut at
its last bit; H100s are published to add like that, and the losses measured on a
GB300 (1e-7 of the accumulator a step) agree.  On average each of the 17 loses half
of 2^-25, the sum three eighths of 2^-23: 2.5 x 2^-23 together.  The products of the
weights' low parts have either sign and lose nothing on average but the sum's 0.375 x
2^-23.

An accumulator that has nearly all of its weight from its first job on keeps that size
for the 15 jobs of 4 + 4 steps up to its flush: 60 x 2.875 x 2^-23 = 2.06e-5 at most
(an accumulator just above a power of two).  What adds up beside it, the weights' two
parts (2^-22) and the logits' rounding (some 2^-22, of either sign from token to
token), is below 2^-20.  In the 2-norm over some 10^5 elements the steps' spread
averages out.  With flushes half as often 31 jobs, not 15, would lose as much.
"""
import numpy as np
import pytest

from tests.test_prefill import Case, _clean, lib  # noqa: F401  (fixtures)

gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("H,Hk,D", [(16, 8, 128), (16, 8, 64), (16, 1, 256)])
def test_first_tokens_that_dominate(H, Hk, D):
    """64 tokens with logits of about 7 in front of 4136 with logits around 0; V with a mean."""
    import torch
    from tests.gpu_helpers import device_status
    ctx, rows = 4200, 600
    c = Case(H, Hk, D, 16, [ctx], [rows], seed=D)
    value = c.vc[..., :-1].contiguous().view(torch.int8)
    c.vc[..., :-1] = (value // 2 + 60).to(torch.int8).view(torch.int32)          # codes -4 .. 123
    first = c.bt[0, :4].long()
    key = c.kc[first][..., :-1].contiguous().view(torch.int8)
    words = c.kc[first]
    words[..., :-1] = (key // 4 + 80).to(torch.int8).view(torch.int32)           # K of about 1.9 in every dimension
    c.kc[first] = words
    c.q.mul_(0.3).add_(7 / (1.9 * D ** 0.5))
    got = c.run().double()
    k, v = (x[c.bt[0].long()].permute(1, 0, 2, 3).reshape(Hk, -1, D // 4 + 1)[:, :ctx] for x in (c.kc, c.vc))
    k, v = (x[..., :-1].contiguous().view(torch.int8).double() * x[..., -1:].contiguous().view(torch.float32).double()
            for x in (k, v))
    at = torch.arange(0, rows, 10, device="cuda")
    q = c.q[at].double().view(len(at), Hk, H // Hk, D)
    z = torch.einsum("ighd,gtd->ight", q, k) * c.w.scale
    seen = torch.arange(ctx, device="cuda")[None] < ctx - (rows - 1 - at)[:, None]
    p = torch.softmax(z.masked_fill(~seen[:, None, None], -np.inf), -1)
    assert 0.5 < float(p[..., :64].sum(-1).mean()) < 0.99
    want = torch.einsum("ight,gtd->ighd", p, v).reshape(len(at), H, D)
    off = float((got[at] - want).norm() / want.norm())
    assert off <= 60 * 2.875 * 2.0 ** -23 + 2.0 ** -20
    assert device_status() == 0
