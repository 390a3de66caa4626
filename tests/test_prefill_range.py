"""Prompt attention at the ends of its ranges: many sequences, rows far apart, q of any magnitude, many heads on
one kv head.  Tolerances: those of test_prefill.py."""
import numpy as np
import pytest

from tests.test_prefill import Case, _clean, check, lib  # noqa: F401  (fixtures)

gpu = pytest.mark.gpu


@gpu
def test_as_many_sequences_as_are_allowed():
    """65,535 sequences of one row each, over four contexts: the decode's result within two f32 bounds."""
    import torch
    import int8_paged_kv_gb300 as pk
    from tests.gpu_helpers import device_status
    S = 65535
    c = Case(8, 2, 64, 16, [1, 7, 16, 33], [1] * 4, seed=3)
    at = torch.arange(S, device="cuda") % 4
    q = torch.randn((S, 8, 64), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    bt, cl = c.bt[at].contiguous(), c.cl[at].contiguous()
    starts = torch.arange(S + 1, dtype=torch.int32, device="cuda")
    kw = dict(num_kv_heads=2, block_size=16, scale=0.125)
    got = pk.pa_q8_prefill(torch.full_like(q, float("nan")), q, c.kc, c.vc, bt, cl, starts, **kw)
    ref = pk.pa_q8_decode(torch.full_like(q, float("nan")), q, c.kc, c.vc, bt, cl, **kw)
    assert bool(((got - ref).abs() <= 2 * (1e-5 + 1e-4 * ref.abs())).all()) and device_status() == 0
    with pytest.raises(pk.PaQ8Error, match="unsupported"):
        pk.pa_q8_prefill(got, q, c.kc, c.vc, bt.repeat(2, 1), cl.repeat(2), torch.zeros(2 * S + 1, dtype=torch.int32, device="cuda"),
                         **kw)


@gpu
def test_rows_past_32bit_offsets():
    """Rows 65,536 elements apart, 4.6e9 in all (9.2 GB each of q and out): the same bits as packed rows."""
    import torch
    c = Case(8, 2, 128, 16, [70000], [70000], "float16", seed=4)
    packed = c.run()
    q = torch.empty((70000, 65536), dtype=torch.float16, device="cuda")
    out = torch.empty_like(q)
    q[:, 1024:2048] = c.q.reshape(70000, 1024)
    c.run(q=q[:, 1024:2048].unflatten(1, (8, 128)), out=out[:, 4096:5120].unflatten(1, (8, 128)))
    assert torch.equal(out[:, 4096:5120].reshape(-1), packed.reshape(-1))


@gpu
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("power", [20, 60, 110])
def test_large_queries(power, dtype):
    """Logits so large that one token has all weight: its V.  Rows whose two largest logits are closer than f32
    can tell (2^-18 of them, with D terms and two parts of q) are left out."""
    c = Case(8, 2, 128, 16, [300], [300], dtype, seed=5)
    c.q *= 2.0 ** power
    got = c.run().float().cpu().numpy().astype(np.float64)
    want, top = c.want()
    from tests.helpers import dense_context
    k = dense_context(c.ok, c.w.block_tables, 0, 300, 128)
    q = c.q.float().cpu().numpy().astype(np.float64)
    clear = np.zeros(q.shape[:2], dtype=bool)
    for h in range(8):
        z = q[:, h] @ k[:, h // 4].T
        z[np.triu_indices(300, 1)] = -np.inf
        two = np.sort(z, axis=1)[:, -2:]
        clear[:, h] = (two[:, 1] - two[:, 0] > 2.0 ** -18 * np.abs(two[:, 1]))
    assert clear.mean() > 0.99
    check(got[clear], want[clear], top[clear], dtype)


@gpu
def test_4096_heads_on_one():
    c = Case(4096, 1, 64, 16, [70, 9], [3, 9], "bfloat16", seed=7)
    c.checked("4096 heads")
