"""Prompt attention over tables that name pages that do not exist, or that are
much wider than the contexts.  Tolerances: those of test_prefill.py; where
logits are of size z, their f32 rounding grows with z, so the absolute part of
the bound takes the factor of f32_units (value size 1, logit size z)."""
import numpy as np
import pytest

from tests.helpers import dense_context
from tests.test_prefill import TYPES, Case, _clean, check, lib  # noqa: F401  (fixtures)

gpu = pytest.mark.gpu


def plain(q, kc, vc, bt, lens, starts, scale, dim, block):
    """The definition in 64 bits; tokens on pages that do not exist are zero vectors."""
    T, H, D = q.shape
    out, top = np.full((T, H, D), np.nan), np.zeros((T, H, D))
    hk, pages = kc.shape[1], kc.shape[0]
    here = np.where(bt < pages, bt, 0)
    for s in range(len(lens)):
        lo, hi, c = int(starts[s]), int(starts[s + 1]), int(lens[s])
        if hi <= lo:
            continue
        lost = (bt[s] >= pages)[np.arange(c) // block]
        k = np.where(lost[:, None, None], 0.0, dense_context(kc, here, s, c, dim))
        v = np.where(lost[:, None, None], 0.0, dense_context(vc, here, s, c, dim))
        for h in range(H):
            g = h // (H // hk)
            z = q[lo:hi, h].astype(np.float64) @ k[:, g].T * scale
            sees = c - (hi - 1 - np.arange(lo, hi))
            z[np.arange(c)[None, :] >= sees[:, None]] = -np.inf
            m = z.max(axis=1, initial=-np.inf, keepdims=True)
            p = np.exp(z - np.where(np.isinf(m), 0.0, m))
            l = p.sum(axis=1, keepdims=True)
            out[lo:hi, h] = p @ v[:, g] / np.where(l == 0, 1.0, l)
            top[lo:hi, h] = np.abs(v[:, g]).max(axis=0)
    return out, top


def low_logits(c):
    """K of positive codes around 80 and rows of q around -1: every logit is strongly negative."""
    import torch
    codes = c.kc[..., :-1].contiguous().view(torch.int8)
    c.kc[..., :-1] = (codes // 4 + 80).to(torch.int8).view(torch.int32)
    c.ok[...] = c.kc.cpu().numpy().view(np.uint32)
    c.q.copy_(0.3 * c.q - 1)


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D,B,low", [(64, 16, True), (128, 16, False), (128, 16, True), (128, 4, True), (256, 32, True)])
def test_tokens_on_pages_that_do_not_exist_are_zero_vectors(D, B, low, dtype):
    """A page inside a context, the first one, one at the end, runs that fill tiles of 64 and 128 tokens, a
    whole table, among tokens of any logits and of strongly negative ones: what the rows that see them get."""
    import int8_paged_kv_gb300 as pk
    from tests.gpu_helpers import dev_u32, device_status, f32_units
    c = Case(8, 2, D, B, [500, 140, 400, 200], [500, 140, 130, 200], dtype, seed=D + B)
    if low:
        low_logits(c)
    clean = c.run()
    assert device_status() == 0
    bt = c.w.block_tables.copy()
    gone = c.w.num_blocks
    bt[0, 64 // B:128 // B] = gone                      # a job of 64 tokens
    bt[0, 160 // B] = 0xFFFFFFFF
    bt[0, 256 // B:384 // B] = 1 << 31                  # a tile of 128
    bt[0, 499 // B] = gone + 5
    bt[1] = gone                                        # nothing left
    bt[2, 0] = gone
    got = c.run(bt=dev_u32(bt))
    assert device_status() == pk.PA_Q8_DEV_BAD_BLOCK
    want, top = plain(c.q.float().cpu().numpy(), c.ok, c.ov, bt, c.w.context_lens, c.starts, c.w.scale, D, B)
    got = got.float().cpu().numpy().astype(np.float64)
    check(got, want, top, dtype, units=f32_units(1, 1.9 * np.sqrt(D)) if low else 1.0)
    assert not got[500:640].any()
    assert np.array_equal(got[770:], clean.float().cpu().numpy()[770:])


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_pieces_without_a_page(D, dtype):
    """A long context cut into pieces, some of which have no page at all."""
    import int8_paged_kv_gb300 as pk
    from tests.gpu_helpers import dev_u32, device_status, f32_units
    c = Case(8, 2, D, 16, [9000, 6000], [5, 5], dtype, seed=D)
    low_logits(c)
    bt = c.w.block_tables.copy()
    bt[0, :200] = 0xFFFFFFFF
    bt[0, 350::3] = c.w.num_blocks
    bt[1, 7:] = c.w.num_blocks
    got = c.run(bt=dev_u32(bt))
    assert device_status() == pk.PA_Q8_DEV_BAD_BLOCK
    want, top = plain(c.q.float().cpu().numpy(), c.ok, c.ov, bt, c.w.context_lens, c.starts, c.w.scale, D, 16)
    check(got.float().cpu().numpy().astype(np.float64), want, top, dtype, units=f32_units(1, 1.9 * np.sqrt(D)))


def widened(c, width):
    """The case's tables, `width` pages wide; entries behind a sequence's pages name no page."""
    from tests.gpu_helpers import dev_u32
    bt = np.full((c.w.block_tables.shape[0], width), 0xFFFFFFFF, dtype=np.uint32)
    bt[:, :c.w.block_tables.shape[1]] = c.w.block_tables
    return dev_u32(bt)


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_short_prompts_behind_wide_tables(D, dtype):
    """Tables for 131,072 tokens: room for pieces in the plan, no context long enough for one, the same bits."""
    import torch
    from tests.gpu_helpers import device_status
    lens = [64, 64, 1, 500, 0, 33, 64, 128]
    c = Case(32, 8, D, 16, lens, [64, 64, 1, 64, 0, 33, 7, 100], dtype, seed=D)
    narrow = c.run()
    got = c.run(bt=widened(c, 8192))
    assert torch.equal(got, narrow) and device_status() == 0


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_long_and_short_contexts_behind_wide_tables(D, dtype):
    """Pieces of the long one, the short ones whole."""
    from tests.gpu_helpers import device_status
    c = Case(8, 2, D, 16, [20000, 40, 700], [9, 40, 130], dtype, seed=D)
    c.checked("wide", bt=widened(c, 65536))
    assert device_status() == 0


def test_size_of_a_wide_tables_plan(lib):  # noqa: F811
    """What the header says: at most some 170 MB of records, 10 to 20 MB of sums."""
    import ctypes
    from int8_paged_kv_gb300 import _binding
    for D in (64, 128, 256):
        for dtype in (0, 1, 2):
            for rows in (1, 8, 512, 4096, 32768):
                for seqs in (1, 8, 64):
                    n = _binding.lib().pa_q8_prefill_workspace_size(ctypes.c_int64(rows), seqs, 32, 8, D, 16, 1 << 16, dtype)
                    assert 0 < n <= 190e6
