"""ctypes binding of libpa_q8.so -- argument marshalling only.

Every function here checks dtypes / devices / shapes of torch tensors,
passes their ``data_ptr()`` and the current CUDA stream to the C entry
point of the same name, and turns a negative status into an exception.
All arithmetic happens in the library's CUDA kernels; there is no fallback:
without the compiled library every call raises.
"""
from __future__ import annotations

import ctypes
import os
import threading

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpa_q8.so")
HEADER = os.path.join(os.path.dirname(_HERE), "include", "pa_q8.h")

PA_Q8_KERNEL_AUTO = 0
PA_Q8_KERNEL_CUDA_CORE = 1
PA_Q8_KERNEL_TENSOR_CORE = 2
PA_Q8_KERNEL_TCGEN05 = 3
PA_Q8_DEV_BAD_BLOCK = 0x1
PA_Q8_DEV_BAD_SLOT = 0x2
PA_Q8_DEV_WAIT_TIMEOUT = 0x4
PA_Q8_DEV_BAD_SEQ = 0x8
PA_Q8_DEV_NO_BLOCK = 0x10
PA_Q8_DEV_BAD_ROWS = 0x20
PA_Q8_F32 = 0
PA_Q8_F16 = 1
PA_Q8_BF16 = 2

_lock = threading.Lock()
_lib = None


class PaQ8Error(RuntimeError):
    def __init__(self, fn: str, status: int, text: str):
        super().__init__(f"{fn}: {text} (status {status})")
        self.status = status


class DecodeOptions(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_int), ("partition_tokens", ctypes.c_int)]


def lib() -> ctypes.CDLL:
    """Load libpa_q8.so (built by int8_paged_kv_gb300.build); raise if absent."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m int8_paged_kv_gb300.build` (no CPU fallback exists)")
        L = ctypes.CDLL(LIB_PATH)
        P, i32, i64, u32, f32, sz = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_uint32,
                                     ctypes.c_float, ctypes.c_size_t)
        L.pa_q8_version.restype = i32
        L.pa_q8_version.argtypes = []
        L.pa_q8_status_string.restype = ctypes.c_char_p
        L.pa_q8_status_string.argtypes = [i32]
        L.pa_q8_reshape_and_cache.restype = i32
        L.pa_q8_reshape_and_cache.argtypes = [P, P, P, P, P, i64, i64, i64, i32, i32, i32, i64, P]
        dec = [P, P, P, P, P, P, i32, i32, i32, i32, i32, i32, i64, f32, P, sz, P]
        L.pa_q8_decode.restype = i32
        L.pa_q8_decode.argtypes = dec
        L.pa_q8_decode_ex.restype = i32
        L.pa_q8_decode_ex.argtypes = dec + [ctypes.POINTER(DecodeOptions)]
        L.pa_q8_decode_rows.restype = i32
        L.pa_q8_decode_rows.argtypes = ([P, P, P, P, P, P, i32, i32, i32, i32, i32, i32, i32, i64, f32,
                                         P, sz, P, ctypes.POINTER(DecodeOptions)])
        L.pa_q8_decode_append.restype = i32
        L.pa_q8_decode_append.argtypes = ([P, P, P, P, i64, i64, P, P, P, P, i32, i32, i32, i32, i32, i32,
                                           i32, i64, f32, P, sz, P, ctypes.POINTER(DecodeOptions)])
        L.pa_q8c_cache_words.restype = sz
        L.pa_q8c_cache_words.argtypes = [i64, i32, i32]
        L.pa_q8c_append.restype = i32
        L.pa_q8c_append.argtypes = [P, P, i64, i64, P, P, P, i64, i32, i32, i64, i32, P]
        L.pa_q8c_decode.restype = i32
        L.pa_q8c_decode.argtypes = [P, P, P, P, P, i32, i32, i32, i32, i64, f32, P, sz, P,
                                    ctypes.POINTER(DecodeOptions)]
        L.pa_q8c_decode_workspace_size.restype = sz
        L.pa_q8c_decode_workspace_size.argtypes = [i32, i32, i32, i32, i64, ctypes.POINTER(DecodeOptions)]
        L.pa_f32_reshape_and_cache.restype = i32
        L.pa_f32_reshape_and_cache.argtypes = [P, P, P, P, P, i64, i64, i64, i32, i32, i32, i64, P]
        L.pa_f32_decode.restype = i32
        L.pa_f32_decode.argtypes = dec + [ctypes.POINTER(DecodeOptions)]
        L.pa_f32_decode_workspace_size.restype = sz
        L.pa_f32_decode_workspace_size.argtypes = [i32] * 6 + [ctypes.POINTER(DecodeOptions)]
        L.pa_q8_decode_rows_workspace_size.restype = sz
        L.pa_q8_decode_rows_workspace_size.argtypes = [i32] * 7 + [ctypes.POINTER(DecodeOptions)]
        L.pa_q8_decode_workspace_size.restype = sz
        L.pa_q8_decode_workspace_size.argtypes = [i32] * 6
        L.pa_q8_decode_workspace_size_ex.restype = sz
        L.pa_q8_decode_workspace_size_ex.argtypes = [i32] * 6 + [ctypes.POINTER(DecodeOptions)]
        L.pa_q8_decode_plan.restype = i32
        L.pa_q8_decode_plan.argtypes = [i32] * 6 + [ctypes.POINTER(DecodeOptions),
                                                    ctypes.POINTER(i32), ctypes.POINTER(i32),
                                                    ctypes.POINTER(i32), ctypes.POINTER(i64)]
        L.pa_q8_prefill.restype = i32
        L.pa_q8_prefill.argtypes = [P, P, i32, i64, i64, P, P, P, P, P, i64, i32, i32, i32, i32, i32, i32, i64, f32,
                                    P, sz, P]
        L.pa_q8_prefill_workspace_size.restype = sz
        L.pa_q8_prefill_workspace_size.argtypes = [i64] + [i32] * 7
        for copy in (L.pa_q8_copy_blocks, L.pa_f32_copy_blocks):
            copy.restype = i32
            copy.argtypes = [P, P, P, P, i64, i32, i32, i32, i64, P]
        L.pa_q8_pool_workspace_size.restype = sz
        L.pa_q8_pool_workspace_size.argtypes = [i32, i64, i32]
        L.pa_q8_pool_init.restype = i32
        L.pa_q8_pool_init.argtypes = [P, P, P, i64, P]
        L.pa_q8_extend_seqs.restype = i32
        L.pa_q8_extend_seqs.argtypes = [P] * 7 + [i32] * 4 + [i64, P, sz, P]
        L.pa_q8_fork_seqs.restype = i32
        L.pa_q8_fork_seqs.argtypes = [P] * 9 + [i32] * 4 + [i64, P, sz, P]
        L.pa_q8_free_seqs.restype = i32
        L.pa_q8_free_seqs.argtypes = [P] * 6 + [i32] * 4 + [i64, P]
        L.pa_q8_compact_blocks.restype = i32
        L.pa_q8_compact_blocks.argtypes = [P] * 7 + [i64, i32, i32, i32, i64, P, sz, P]
        L.pa_q8_device_status.restype = i32
        L.pa_q8_device_status.argtypes = [ctypes.POINTER(u32), i32, P]
        L.pa_q8_selftest_wait_timeout.restype = i32
        L.pa_q8_selftest_wait_timeout.argtypes = [u32, P]
        _lib = L
        return L


def pa_q8_status_string(status: int) -> str:
    return lib().pa_q8_status_string(int(status)).decode()


def pa_q8_version() -> int:
    return int(lib().pa_q8_version())


def _check(fn: str, rc: int) -> None:
    if rc != 0:
        raise PaQ8Error(fn, rc, pa_q8_status_string(rc))


def _stream(stream):
    import torch
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return ctypes.c_void_p(stream)
    return ctypes.c_void_p(stream.cuda_stream)


def _cuda(t, dtype, name):
    """Device pointer of a CUDA tensor; u32 buffers may also be int32 (same bits)."""
    import torch
    ok = (torch.uint32, torch.int32) if dtype is torch.uint32 else (dtype,)
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype not in ok:
        raise TypeError(f"{name} must be a CUDA tensor of dtype {dtype}")
    return ctypes.c_void_p(t.data_ptr())


def _opts(kernel: int, partition_tokens: int):
    return ctypes.byref(DecodeOptions(int(kernel), int(partition_tokens)))


def _allocate(need, like, stream):
    """`need` bytes on the device of the tensor `like`, from the pool of the
    stream that will use them: torch gives a stream's memory away again behind
    the work queued there, so what is freed once a call has queued its work
    needs no event, and no other stream's work is pending on it."""
    import torch
    if stream is None:
        return torch.empty(need, dtype=torch.uint8, device=like.device)
    if not isinstance(stream, torch.cuda.Stream):
        handle = stream if isinstance(stream, int) else stream.cuda_stream
        # 0 and 1: the legacy default stream (an ExternalStream(0) is a new stream)
        stream = (torch.cuda.default_stream(like.device) if handle in (0, 1)
                  else torch.cuda.ExternalStream(handle, device=like.device))
    with torch.cuda.stream(stream):
        return torch.empty(need, dtype=torch.uint8, device=like.device)


def pa_q8_reshape_and_cache(key, value, key_cache, value_cache, slot_mapping, *, num_kv_heads: int,
                            head_size: int, block_size: int, num_blocks: int | None = None,
                            stream=None) -> None:
    """Quantise rows of `key`/`value` into the caches.

    key/value: float32 CUDA tensors whose first dimension is the token and
    whose rows hold num_kv_heads * head_size contiguous floats; rows may be
    further apart (e.g. K/V column slices of fused QKV rows): the row stride
    is taken from the tensor.  Caches: uint32 [num_blocks, Hk, B, D/4 + 1].
    """
    import torch
    for t, n in ((key, "key"), (value, "value")):
        if t.dim() < 2 or t.stride(-1) != 1:
            raise ValueError(f"{n} rows must be contiguous in their last dimension")
        inner = t[0] if t.dim() > 2 else None
        if inner is not None and not inner.is_contiguous():
            raise ValueError(f"{n} must be [T, Hk, D] with contiguous rows")
    T = int(slot_mapping.numel())
    if key.shape[0] != T or value.shape[0] != T:
        raise ValueError("key/value rows must match slot_mapping")
    nb = int(key_cache.shape[0]) if num_blocks is None else int(num_blocks)
    rc = lib().pa_q8_reshape_and_cache(
        _cuda(key, torch.float32, "key"), _cuda(value, torch.float32, "value"),
        _cuda(key_cache, torch.uint32, "key_cache"), _cuda(value_cache, torch.uint32, "value_cache"),
        _cuda(slot_mapping, torch.uint32, "slot_mapping"), T, int(key.stride(0)),
        int(value.stride(0)), int(num_kv_heads), int(head_size), int(block_size), nb, _stream(stream))
    _check("pa_q8_reshape_and_cache", rc)


def pa_q8_decode_workspace_size(num_seqs, num_heads, num_kv_heads, head_size, block_size,
                                max_blocks_per_seq, *, kernel: int = 0,
                                partition_tokens: int = 0) -> int:
    return int(lib().pa_q8_decode_workspace_size_ex(int(num_seqs), int(num_heads), int(num_kv_heads),
                                                    int(head_size), int(block_size),
                                                    int(max_blocks_per_seq),
                                                    _opts(kernel, partition_tokens)))


def pa_q8_decode_plan(num_seqs, num_heads, num_kv_heads, head_size, block_size, max_blocks_per_seq,
                      *, kernel: int = 0, partition_tokens: int = 0) -> dict:
    k, pt, np_ = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
    nc = ctypes.c_int64()
    rc = lib().pa_q8_decode_plan(int(num_seqs), int(num_heads), int(num_kv_heads), int(head_size),
                                 int(block_size), int(max_blocks_per_seq),
                                 _opts(kernel, partition_tokens), ctypes.byref(k),
                                 ctypes.byref(pt), ctypes.byref(np_), ctypes.byref(nc))
    _check("pa_q8_decode_plan", rc)
    return {"kernel": k.value, "partition_tokens": pt.value, "num_partitions": np_.value,
            "num_ctas": nc.value}


def pa_q8_decode(out, q, key_cache, value_cache, block_tables, context_lens, *, num_kv_heads: int,
                 block_size: int, scale: float, num_blocks: int | None = None, workspace=None,
                 kernel: int = 0, partition_tokens: int = 0, stream=None):
    """out[S, H, D] = paged int8 attention decode (see include/pa_q8.h).

    workspace: a uint8 CUDA tensor of >= pa_q8_decode_workspace_size bytes;
    allocated here (torch) when None.  Returns `out`.
    """
    import torch
    S, H, D = q.shape
    if out.shape != q.shape or not out.is_contiguous() or not q.is_contiguous():
        raise ValueError("q and out must be contiguous [num_seqs, num_heads, head_size]")
    Nb = int(block_tables.shape[1])
    if block_tables.shape[0] != S or context_lens.numel() != S:
        raise ValueError("block_tables / context_lens do not match num_seqs")
    nb = int(key_cache.shape[0]) if num_blocks is None else int(num_blocks)
    need = pa_q8_decode_workspace_size(S, H, num_kv_heads, D, block_size, Nb, kernel=kernel,
                                       partition_tokens=partition_tokens)
    if workspace is None and need:
        workspace = _allocate(need, q, stream)
    ws_ptr = ctypes.c_void_p(workspace.data_ptr()) if workspace is not None else ctypes.c_void_p(0)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    rc = lib().pa_q8_decode_ex(
        _cuda(out, torch.float32, "out"), _cuda(q, torch.float32, "q"),
        _cuda(key_cache, torch.uint32, "key_cache"), _cuda(value_cache, torch.uint32, "value_cache"),
        _cuda(block_tables, torch.uint32, "block_tables"),
        _cuda(context_lens, torch.uint32, "context_lens"), S, H, int(num_kv_heads), D,
        int(block_size), Nb, nb, float(scale), ws_ptr, ws_bytes, _stream(stream),
        _opts(kernel, partition_tokens))
    _check("pa_q8_decode", rc)
    return out


def pa_q8_decode_rows_workspace_size(num_seqs, num_rows, num_heads, num_kv_heads, head_size,
                                     block_size, max_blocks_per_seq, *, kernel: int = 0,
                                     partition_tokens: int = 0) -> int:
    return int(lib().pa_q8_decode_rows_workspace_size(
        int(num_seqs), int(num_rows), int(num_heads), int(num_kv_heads), int(head_size),
        int(block_size), int(max_blocks_per_seq), _opts(kernel, partition_tokens)))


def pa_q8_decode_rows(out, q, key_cache, value_cache, block_tables, context_lens, *,
                      num_kv_heads: int, block_size: int, scale: float,
                      num_blocks: int | None = None, workspace=None, kernel: int = 0,
                      partition_tokens: int = 0, stream=None):
    """out[S, R, H, D] = causal multi-row decode: row b of sequence s attends
    to the first c - (R - 1 - b) cached tokens (see include/pa_q8.h).
    Returns `out`."""
    import torch
    S, R, H, D = q.shape
    if out.shape != q.shape or not out.is_contiguous() or not q.is_contiguous():
        raise ValueError("q and out must be contiguous [num_seqs, num_rows, num_heads, head_size]")
    Nb = int(block_tables.shape[1])
    if block_tables.shape[0] != S or context_lens.numel() != S:
        raise ValueError("block_tables / context_lens do not match num_seqs")
    nb = int(key_cache.shape[0]) if num_blocks is None else int(num_blocks)
    need = pa_q8_decode_rows_workspace_size(S, R, H, num_kv_heads, D, block_size, Nb, kernel=kernel,
                                            partition_tokens=partition_tokens)
    if workspace is None and need:
        workspace = _allocate(need, q, stream)
    ws_ptr = ctypes.c_void_p(workspace.data_ptr()) if workspace is not None else ctypes.c_void_p(0)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    rc = lib().pa_q8_decode_rows(
        _cuda(out, torch.float32, "out"), _cuda(q, torch.float32, "q"),
        _cuda(key_cache, torch.uint32, "key_cache"), _cuda(value_cache, torch.uint32, "value_cache"),
        _cuda(block_tables, torch.uint32, "block_tables"),
        _cuda(context_lens, torch.uint32, "context_lens"), S, R, H, int(num_kv_heads), D,
        int(block_size), Nb, nb, float(scale), ws_ptr, ws_bytes, _stream(stream),
        _opts(kernel, partition_tokens))
    _check("pa_q8_decode_rows", rc)
    return out


def _rows2d(t, n_rows, name):
    """(tensor, row stride in floats) of new K/V rows given as [S, R, Hk, D]
    / [S, R, Hk * D] (contiguous) or [S * R, Hk * D] (rows may be strided)."""
    if t.dim() == 2:
        if t.shape[0] != n_rows or t.stride(1) != 1:
            raise ValueError(f"{name}: expected [num_seqs * num_rows, num_kv_heads * head_size] rows")
        return t, int(t.stride(0))
    if not t.is_contiguous() or t.shape[0] * t.shape[1] != n_rows:
        raise ValueError(f"{name}: expected contiguous [num_seqs, num_rows, ...] rows")
    return t, int(t[0].numel() // t.shape[1])


def pa_q8_decode_append(out, q, key, value, key_cache, value_cache, block_tables, context_lens, *,
                        num_kv_heads: int, block_size: int, scale: float,
                        num_blocks: int | None = None, workspace=None, kernel: int = 0,
                        partition_tokens: int = 0, stream=None):
    """Append the newest num_rows tokens' K/V (rows of key / value) to the
    caches and decode q [S, R, H, D] over them, in one attention launch (see
    include/pa_q8.h).  Returns `out`."""
    import torch
    S, R, H, D = q.shape
    if out.shape != q.shape or not out.is_contiguous() or not q.is_contiguous():
        raise ValueError("q and out must be contiguous [num_seqs, num_rows, num_heads, head_size]")
    Nb = int(block_tables.shape[1])
    if block_tables.shape[0] != S or context_lens.numel() != S:
        raise ValueError("block_tables / context_lens do not match num_seqs")
    k2, ks = _rows2d(key, S * R, "key")
    v2, vs = _rows2d(value, S * R, "value")
    nb = int(key_cache.shape[0]) if num_blocks is None else int(num_blocks)
    need = pa_q8_decode_rows_workspace_size(S, R, H, num_kv_heads, D, block_size, Nb, kernel=kernel,
                                            partition_tokens=partition_tokens)
    if workspace is None and need:
        workspace = _allocate(need, q, stream)
    ws_ptr = ctypes.c_void_p(workspace.data_ptr()) if workspace is not None else ctypes.c_void_p(0)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    rc = lib().pa_q8_decode_append(
        _cuda(out, torch.float32, "out"), _cuda(q, torch.float32, "q"),
        _cuda(k2, torch.float32, "key"), _cuda(v2, torch.float32, "value"), ks, vs,
        _cuda(key_cache, torch.uint32, "key_cache"), _cuda(value_cache, torch.uint32, "value_cache"),
        _cuda(block_tables, torch.uint32, "block_tables"),
        _cuda(context_lens, torch.uint32, "context_lens"), S, R, H, int(num_kv_heads), D,
        int(block_size), Nb, nb, float(scale), ws_ptr, ws_bytes, _stream(stream),
        _opts(kernel, partition_tokens))
    _check("pa_q8_decode_append", rc)
    return out


def pa_f32_reshape_and_cache(key, value, key_cache, value_cache, slot_mapping, *, num_kv_heads: int,
                             head_size: int, block_size: int, num_blocks: int | None = None,
                             stream=None) -> None:
    """Copy rows into the f32 caches [num_blocks, Hk, B, D] (see include/pa_q8.h)."""
    import torch
    T = int(slot_mapping.numel())
    if key.dim() != 2 or value.dim() != 2 or key.stride(1) != 1 or value.stride(1) != 1:
        raise ValueError("key/value must be 2-D [num_tokens, >= num_kv_heads * head_size] with unit column stride")
    nb = int(key_cache.shape[0]) if num_blocks is None else int(num_blocks)
    rc = lib().pa_f32_reshape_and_cache(
        _cuda(key, torch.float32, "key"), _cuda(value, torch.float32, "value"),
        _cuda(key_cache, torch.float32, "key_cache"), _cuda(value_cache, torch.float32, "value_cache"),
        _cuda(slot_mapping, torch.uint32, "slot_mapping"), T, int(key.stride(0)), int(value.stride(0)),
        int(num_kv_heads), int(head_size), int(block_size), nb, _stream(stream))
    _check("pa_f32_reshape_and_cache", rc)


def pa_f32_decode_workspace_size(num_seqs, num_heads, num_kv_heads, head_size, block_size,
                                 max_blocks_per_seq, *, partition_tokens: int = 0) -> int:
    return int(lib().pa_f32_decode_workspace_size(int(num_seqs), int(num_heads), int(num_kv_heads),
                                                  int(head_size), int(block_size), int(max_blocks_per_seq),
                                                  _opts(0, partition_tokens)))


def pa_f32_decode(out, q, key_cache, value_cache, block_tables, context_lens, *, num_kv_heads: int,
                  block_size: int, scale: float, num_blocks: int | None = None, workspace=None,
                  partition_tokens: int = 0, stream=None):
    """out[S, H, D] = paged attention decode over the f32 caches.  Returns `out`."""
    import torch
    S, H, D = q.shape
    if out.shape != q.shape or not out.is_contiguous() or not q.is_contiguous():
        raise ValueError("q and out must be contiguous [num_seqs, num_heads, head_size]")
    Nb = int(block_tables.shape[1])
    if block_tables.shape[0] != S or context_lens.numel() != S:
        raise ValueError("block_tables / context_lens do not match num_seqs")
    nb = int(key_cache.shape[0]) if num_blocks is None else int(num_blocks)
    need = pa_f32_decode_workspace_size(S, H, num_kv_heads, D, block_size, Nb,
                                        partition_tokens=partition_tokens)
    if workspace is None and need:
        workspace = _allocate(need, q, stream)
    ws_ptr = ctypes.c_void_p(workspace.data_ptr()) if workspace is not None else ctypes.c_void_p(0)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    rc = lib().pa_f32_decode(
        _cuda(out, torch.float32, "out"), _cuda(q, torch.float32, "q"),
        _cuda(key_cache, torch.float32, "key_cache"), _cuda(value_cache, torch.float32, "value_cache"),
        _cuda(block_tables, torch.uint32, "block_tables"),
        _cuda(context_lens, torch.uint32, "context_lens"), S, H, int(num_kv_heads), D,
        int(block_size), Nb, nb, float(scale), ws_ptr, ws_bytes, _stream(stream), _opts(0, partition_tokens))
    _check("pa_f32_decode", rc)
    return out


def pa_q8c_cache_words(max_t: int, num_kv_heads: int, head_size: int) -> int:
    return int(lib().pa_q8c_cache_words(int(max_t), int(num_kv_heads), int(head_size)))


def pa_q8c_append(key, value, key_cache, value_cache, slot_mapping, *, num_kv_heads: int, head_size: int,
                  max_t: int, num_seqs: int | None = None, stream=None) -> None:
    """Quantise rows into the contiguous caches (u32 [num_seqs, cache_words]);
    slot = sequence * max_t + position (see include/pa_q8.h)."""
    import torch
    T = int(slot_mapping.numel())
    if key.dim() != 2 or value.dim() != 2 or key.stride(1) != 1 or value.stride(1) != 1:
        raise ValueError("key/value must be 2-D [num_tokens, >= num_kv_heads * head_size] with unit column stride")
    ns = int(key_cache.shape[0]) if num_seqs is None else int(num_seqs)
    rc = lib().pa_q8c_append(
        _cuda(key, torch.float32, "key"), _cuda(value, torch.float32, "value"), int(key.stride(0)),
        int(value.stride(0)), _cuda(key_cache, torch.uint32, "key_cache"),
        _cuda(value_cache, torch.uint32, "value_cache"), _cuda(slot_mapping, torch.uint32, "slot_mapping"), T,
        int(num_kv_heads), int(head_size), int(max_t), ns, _stream(stream))
    _check("pa_q8c_append", rc)


def pa_q8c_decode_workspace_size(num_seqs, num_heads, num_kv_heads, head_size, max_t, *,
                                 partition_tokens: int = 0) -> int:
    return int(lib().pa_q8c_decode_workspace_size(int(num_seqs), int(num_heads), int(num_kv_heads),
                                                  int(head_size), int(max_t), _opts(0, partition_tokens)))


def pa_q8c_decode(out, q, key_cache, value_cache, context_lens, *, num_kv_heads: int, max_t: int,
                  scale: float, workspace=None, partition_tokens: int = 0, stream=None):
    """out[S, H, D] = decode over the contiguous caches.  Returns `out`."""
    import torch
    S, H, D = q.shape
    if out.shape != q.shape or not out.is_contiguous() or not q.is_contiguous():
        raise ValueError("q and out must be contiguous [num_seqs, num_heads, head_size]")
    if context_lens.numel() != S:
        raise ValueError("context_lens does not match num_seqs")
    need = pa_q8c_decode_workspace_size(S, H, num_kv_heads, D, max_t, partition_tokens=partition_tokens)
    if workspace is None and need:
        workspace = _allocate(need, q, stream)
    ws_ptr = ctypes.c_void_p(workspace.data_ptr()) if workspace is not None else ctypes.c_void_p(0)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    rc = lib().pa_q8c_decode(
        _cuda(out, torch.float32, "out"), _cuda(q, torch.float32, "q"),
        _cuda(key_cache, torch.uint32, "key_cache"), _cuda(value_cache, torch.uint32, "value_cache"),
        _cuda(context_lens, torch.uint32, "context_lens"), S, H, int(num_kv_heads), D, int(max_t), float(scale),
        ws_ptr, ws_bytes, _stream(stream), _opts(0, partition_tokens))
    _check("pa_q8c_decode", rc)
    return out


_U32 = ()                   # dtypes of u32 buffers (the same bits), and two of torch's calls, once it is loaded
_current_device = _raw_stream = None


def _address(t, dtypes, name, device, numel=-1):
    """Address of a contiguous CUDA tensor of one of the given types on the
    device with this index, with the number of elements asked for."""
    if t.dtype in dtypes and t.get_device() == device and t.is_contiguous() and (numel < 0 or t.numel() == numel):
        return t.data_ptr()
    if t.dtype not in dtypes or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor of dtype {' or '.join(map(str, dtypes))}")
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, the call's other tensors on cuda:{device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} has {t.numel()} elements, expected {numel}")


def _current(t):
    """Index of the tensor's device, which has to be the current one: the
    library queues there."""
    global _U32, _current_device, _raw_stream
    if _current_device is None:
        import torch
        _U32 = (torch.int32, torch.uint32)
        # torch's own short way to the handle, 2 us of a call's 6 to 8; public calls where it is not there
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                              lambda device: torch.cuda.current_stream(device).cuda_stream)
        _current_device = torch.cuda.current_device
    device = t.get_device()
    if device < 0:
        raise TypeError("tensors must be CUDA tensors")
    if device != _current_device():
        raise ValueError(f"tensors are on {t.device}, the current device is cuda:{_current_device()}")
    return device


def _queue(stream, device):
    """The stream's handle (None: the device's current stream)."""
    if stream is None:
        return _raw_stream(device)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _scratch(need, workspace, like, stream):
    """(tensor, address, bytes) of the caller's workspace, or of one allocated
    here; `like`: a tensor on the call's device.  The caller holds the tensor
    until the library has queued its work: its memory is given away when it goes."""
    if workspace is None:
        workspace = _allocate(max(need, 16), like, stream)
    elif workspace.get_device() != like.get_device() or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {like.device}")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _row_type(dtype):
    import torch
    try:
        return {torch.float32: PA_Q8_F32, torch.float16: PA_Q8_F16, torch.bfloat16: PA_Q8_BF16}[dtype]
    except KeyError:
        raise TypeError(f"q and out must be float32, float16 or bfloat16, got {dtype}") from None


def pa_q8_prefill_workspace_size(num_rows, num_seqs, num_heads, num_kv_heads, head_size, block_size,
                                 max_blocks_per_seq, dtype) -> int:
    """Workspace bytes of pa_q8_prefill; dtype: the torch dtype of q."""
    return int(lib().pa_q8_prefill_workspace_size(int(num_rows), int(num_seqs), int(num_heads), int(num_kv_heads),
                                                  int(head_size), int(block_size), int(max_blocks_per_seq),
                                                  _row_type(dtype)))


def pa_q8_prefill(out, q, key_cache, value_cache, block_tables, context_lens, query_starts, *,
                  num_kv_heads: int, block_size: int, scale: float, num_blocks: int | None = None,
                  workspace=None, stream=None):
    """out[T, H, D] = causal attention of packed prompt rows over the int8
    pages (see include/pa_q8.h): rows query_starts[s] .. query_starts[s + 1] - 1
    are the last ones of sequence s's context_lens[s] cached tokens.

    q, out: float32, float16 or bfloat16 (the same), rows may be further apart
    than H * D.  query_starts: u32 [S + 1].  Returns `out`.
    """
    T, H, D = q.shape
    dt = _row_type(q.dtype)
    dev = _current(q)
    if out.dtype != q.dtype or out.shape != q.shape or out.get_device() != dev:
        raise ValueError("out must be a tensor like q")
    for t, name in ((q, "q"), (out, "out")):
        if T and (t.stride(2) != 1 or (H > 1 and t.stride(1) != D)):
            raise ValueError(f"each row of {name} must be contiguous [num_heads, head_size]")
    qs, os_ = (q.stride(0), out.stride(0)) if T > 1 else (H * D, H * D)
    S, Nb = block_tables.shape
    words = key_cache.numel()
    nb = int(key_cache.shape[0]) if num_blocks is None else int(num_blocks)
    if nb * num_kv_heads * block_size * (D // 4 + 1) > words:
        raise ValueError("the caches do not hold num_blocks pages of these sizes")
    u32 = _U32
    L = lib()
    need = L.pa_q8_prefill_workspace_size(T, S, H, num_kv_heads, D, block_size, Nb, dt)
    scratch, ws, ws_bytes = _scratch(need, workspace, q, stream)
    _check("pa_q8_prefill", L.pa_q8_prefill(
        out.data_ptr(), q.data_ptr(), dt, os_, qs, _address(key_cache, u32, "key_cache", dev),
        _address(value_cache, u32, "value_cache", dev, words), _address(block_tables, u32, "block_tables", dev),
        _address(context_lens, u32, "context_lens", dev, S), _address(query_starts, u32, "query_starts", dev, S + 1),
        T, S, H, num_kv_heads, D, block_size, Nb, nb, scale, ws, ws_bytes, _queue(stream, dev)))
    return out


def _copy_blocks(fn, key_cache, value_cache, src_blocks, dst_blocks, dtypes, head_size, num_blocks, stream):
    dev = _current(key_cache)
    if key_cache.dim() != 4 or value_cache.shape != key_cache.shape:
        raise ValueError("key_cache and value_cache must have one shape [num_blocks, num_kv_heads, block_size, ...]")
    nb, hk, bs, _ = key_cache.shape
    if num_blocks is not None:
        if num_blocks > nb:
            raise ValueError("the caches do not hold num_blocks pages")
        nb = int(num_blocks)
    n = src_blocks.numel()
    u32 = _U32
    dtypes = dtypes or u32
    _check(fn, getattr(lib(), fn)(
        _address(key_cache, dtypes, "key_cache", dev), _address(value_cache, dtypes, "value_cache", dev),
        _address(src_blocks, u32, "src_blocks", dev), _address(dst_blocks, u32, "dst_blocks", dev, n),
        n, hk, head_size, bs, nb, _queue(stream, dev)))


def pa_q8_copy_blocks(key_cache, value_cache, src_blocks, dst_blocks, *, num_blocks: int | None = None,
                      stream=None) -> None:
    """Copy page src_blocks[i] to dst_blocks[i] of both q8 caches (0xFFFFFFFF: no pair)."""
    _copy_blocks("pa_q8_copy_blocks", key_cache, value_cache, src_blocks, dst_blocks, None,
                 4 * (key_cache.shape[-1] - 1), num_blocks, stream)


def pa_f32_copy_blocks(key_cache, value_cache, src_blocks, dst_blocks, *, num_blocks: int | None = None,
                       stream=None) -> None:
    """pa_q8_copy_blocks over the f32 caches [num_blocks, Hk, B, D]."""
    import torch
    _copy_blocks("pa_f32_copy_blocks", key_cache, value_cache, src_blocks, dst_blocks, (torch.float32,),
                 key_cache.shape[-1], num_blocks, stream)


def pa_q8_pool_workspace_size(num_seqs: int, num_blocks: int, num_requests: int = 0) -> int:
    return int(lib().pa_q8_pool_workspace_size(int(num_seqs), int(num_blocks), int(num_requests)))


def _pool(block_tables, context_lens, ref_counts, free_blocks, num_free):
    """(device, rows, row length, pages, addresses) of a pool's tensors."""
    dev = _current(block_tables)
    S, Nb = block_tables.shape
    nb = ref_counts.numel()
    u32 = _U32
    return dev, S, Nb, nb, (
        _address(block_tables, u32, "block_tables", dev), _address(context_lens, u32, "context_lens", dev, S),
        _address(ref_counts, u32, "ref_counts", dev), _address(free_blocks, u32, "free_blocks", dev, nb),
        _address(num_free, u32, "num_free", dev, 1))


def pa_q8_pool_init(ref_counts, free_blocks, num_free, *, stream=None) -> None:
    """All pages of the pool free (see include/pa_q8.h)."""
    dev, nb = _current(ref_counts), ref_counts.numel()
    u32 = _U32
    _check("pa_q8_pool_init", lib().pa_q8_pool_init(
        _address(ref_counts, u32, "ref_counts", dev), _address(free_blocks, u32, "free_blocks", dev, nb),
        _address(num_free, u32, "num_free", dev, 1), nb, _queue(stream, dev)))


def pa_q8_extend_seqs(block_tables, context_lens, ref_counts, free_blocks, num_free, seqs, new_lens, *,
                      block_size: int, workspace=None, stream=None) -> None:
    """Grow sequence seqs[i] to new_lens[i] tokens, with pages from the pool."""
    dev, S, Nb, nb, pool = _pool(block_tables, context_lens, ref_counts, free_blocks, num_free)
    n = seqs.numel()
    L = lib()
    u32 = _U32
    scratch, ws, ws_bytes = _scratch(L.pa_q8_pool_workspace_size(S, nb, n), workspace, block_tables, stream)
    _check("pa_q8_extend_seqs", L.pa_q8_extend_seqs(
        *pool, _address(seqs, u32, "seqs", dev), _address(new_lens, u32, "new_lens", dev, n), n, S, Nb,
        block_size, nb, ws, ws_bytes, _queue(stream, dev)))


def pa_q8_fork_seqs(block_tables, context_lens, ref_counts, free_blocks, num_free, parents, children, copy_src,
                    copy_dst, *, block_size: int, workspace=None, stream=None) -> None:
    """Empty rows children[i] become copies of sequences parents[i]; the pages
    to copy, for pa_q8_copy_blocks, go to copy_src / copy_dst."""
    dev, S, Nb, nb, pool = _pool(block_tables, context_lens, ref_counts, free_blocks, num_free)
    n = parents.numel()
    L = lib()
    u32 = _U32
    scratch, ws, ws_bytes = _scratch(L.pa_q8_pool_workspace_size(S, nb, n), workspace, block_tables, stream)
    _check("pa_q8_fork_seqs", L.pa_q8_fork_seqs(
        *pool, _address(parents, u32, "parents", dev), _address(children, u32, "children", dev, n),
        _address(copy_src, u32, "copy_src", dev, n), _address(copy_dst, u32, "copy_dst", dev, n), n, S, Nb,
        block_size, nb, ws, ws_bytes, _queue(stream, dev)))


def pa_q8_free_seqs(block_tables, context_lens, ref_counts, free_blocks, num_free, seqs, *, block_size: int,
                    stream=None) -> None:
    """Empty the rows seqs[i]; pages that no row holds go back to the pool."""
    dev, S, Nb, nb, pool = _pool(block_tables, context_lens, ref_counts, free_blocks, num_free)
    _check("pa_q8_free_seqs", lib().pa_q8_free_seqs(
        *pool, _address(seqs, _U32, "seqs", dev), seqs.numel(), S, Nb, block_size, nb, _queue(stream, dev)))


def pa_q8_compact_blocks(block_tables, context_lens, ref_counts, free_blocks, num_free, move_src, move_dst, *,
                         block_size: int, workspace=None, stream=None) -> None:
    """Renumber the held pages to 0 .. L - 1; the moves, for pa_q8_copy_blocks,
    go to move_src / move_dst (at least num_blocks // 2 entries)."""
    dev, S, Nb, nb, pool = _pool(block_tables, context_lens, ref_counts, free_blocks, num_free)
    n = move_src.numel()
    L = lib()
    u32 = _U32
    scratch, ws, ws_bytes = _scratch(L.pa_q8_pool_workspace_size(S, nb, 0), workspace, block_tables, stream)
    _check("pa_q8_compact_blocks", L.pa_q8_compact_blocks(
        *pool, _address(move_src, u32, "move_src", dev), _address(move_dst, u32, "move_dst", dev, n), n, S, Nb,
        block_size, nb, ws, ws_bytes, _queue(stream, dev)))


def pa_q8_device_status(clear: bool = True, stream=None) -> int:
    bits = ctypes.c_uint32()
    _check("pa_q8_device_status", lib().pa_q8_device_status(ctypes.byref(bits), int(bool(clear)),
                                                              _stream(stream)))
    return int(bits.value)


def pa_q8_selftest_wait_timeout(timeout_us: int, stream=None) -> None:
    _check("pa_q8_selftest_wait_timeout",
           lib().pa_q8_selftest_wait_timeout(int(timeout_us), _stream(stream)))


def header_functions() -> list[str]:
    """Names of the functions include/pa_q8.h declares."""
    import re
    text = open(HEADER).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(pa_(?:q8c?|f32)_[a-z0-9_]+)\s*\(", text)))
