"""What pa_q8_prefill asks for as workspace (host side; no device is touched)."""
import ctypes

import pytest

F32, F16, BF16 = 0, 1, 2


@pytest.fixture(scope="module")
def size():
    from int8_paged_kv_gb300 import _binding, build
    build.build()
    L = _binding.lib()

    def ask(rows, seqs, H, Hk, D, B, Nb, dtype):
        n = L.pa_q8_prefill_workspace_size(ctypes.c_int64(rows), seqs, H, Hk, D, B, Nb, dtype)
        assert n > 0
        return n
    return ask


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_16_bit_rows_keep_no_sums(size, D, dtype):
    """Only f32 rows add their accumulators to f32 sums, 128 rows x head size per accumulator and SM.  A large
    batch of whole prompts needs a few KB of lists, whatever the table's width."""
    wide, narrow = size(32768, 8, 32, 8, D, 16, 8192, dtype), size(32768, 8, 32, 8, D, 16, 64, dtype)
    assert wide == narrow < 1 << 20
    sums = 152 * (1 if D == 256 else 2) * 128 * D * 4
    lists = size(32768, 8, 32, 8, D, 16, 64, F32)
    assert size(32768, 8, 32, 8, D, 16, 8192, F32) == lists + sums
