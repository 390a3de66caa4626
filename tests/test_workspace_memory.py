"""The memory that the prompt, window and pool calls take for a workspace
straight from torch's allocator: whose pool it comes from, and that it is held
until the library has queued its work and given back then, once.  With a
stand-in for the library, on CPU tensors; a GPU test takes the way without torch's
private calls.
"""
import os
import subprocess
import sys
import types

import pytest

from tests.test_workspace import NEED

gpu = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CURRENT = 0x900                 # the current stream's handle
EVERY = ["prefill", "window_prefill", "window_decode", "extend", "fork", "compact"]


class Allocator:
    """torch's, with every piece of memory's stream, and what happened in which order."""

    def __init__(self):
        self.live, self.events = {}, []

    def alloc(self, need, handle):
        address = 1 << 40 | (len(self.events) + 1) << 20
        self.live[address] = (need, handle)
        self.events.append(("alloc", address))
        return address

    def delete(self, address):
        del self.live[address]                          # (given back twice: KeyError)
        self.events.append(("delete", address))


class Library:
    """Every size query says NEED; a call notes the live memory among its arguments, and returns `status`."""

    def __init__(self, allocator):
        self.allocator, self.status, self.seen = allocator, 0, []

    def __getattr__(self, name):
        if name.endswith("workspace_size"):
            return lambda *a: NEED

        def call(*args):
            args = [getattr(a, "value", a) for a in args]
            self.seen += [self.allocator.live[a] for a in args if a in self.allocator.live]
            self.allocator.events.append(("call", args[-1]))
            return self.status
        return call


@pytest.fixture
def stand_in(monkeypatch):
    import torch
    from int8_paged_kv_gb300 import _binding
    allocator = Allocator()
    library = Library(allocator)
    for name, value in dict(lib=lambda: library, _current=lambda t: -1, _U32=(torch.int32, torch.uint32), _SIZES={},
                            _raw_stream=lambda device: CURRENT, _raw_alloc=allocator.alloc,
                            _raw_delete=allocator.delete, pa_q8_status_string=str).items():
        monkeypatch.setattr(_binding, name, value)
    return types.SimpleNamespace(library=library, allocator=allocator, binding=_binding)


def call(name, b, **kw):
    import torch

    def i32(*shape):
        return torch.zeros(shape, dtype=torch.int32)
    pool, one, cache, q = (i32(4, 4), i32(4), i32(16), i32(16), i32(1)), i32(1), i32(16, 2, 16, 33), torch.zeros((4, 8, 128))
    sizes = dict(num_kv_heads=2, block_size=16, scale=0.1)
    if name == "prefill":
        b.pa_q8_prefill(q.clone(), q, cache, cache, pool[0], pool[1], i32(5), **sizes, **kw)
    elif name == "window_prefill":
        b.pa_q8_window_prefill(q.clone(), q, cache, cache, pool[0], pool[1], i32(5), window=30, **sizes, **kw)
    elif name == "window_decode":
        b.pa_q8_window_decode(q.clone(), q, cache, cache, pool[0], pool[1], window=30, **sizes, **kw)
    elif name == "extend":
        b.pa_q8_extend_seqs(*pool, one, one, block_size=16, **kw)
    elif name == "fork":
        b.pa_q8_fork_seqs(*pool, one, one, one, one, block_size=16, **kw)
    else:
        b.pa_q8_compact_blocks(*pool, i32(8), i32(8), block_size=16, **kw)


@pytest.mark.parametrize("stream,handle,pool", [
    (None, CURRENT, CURRENT), (0, 0, 0), (1, 1, 0), (64, 64, 64), (types.SimpleNamespace(cuda_stream=128), 128, 128)])
@pytest.mark.parametrize("name", EVERY)
def test_memory_of_the_calls_stream_held_until_it_is_queued(stand_in, name, stream, handle, pool):
    """0 and 1 are the legacy default stream, whose pool is 0's."""
    call(name, stand_in.binding, stream=stream)
    assert stand_in.library.seen == [(NEED, pool)]
    kinds = [e[0] for e in stand_in.allocator.events]
    assert kinds == ["alloc", "call", "delete"] and stand_in.allocator.events[1] == ("call", handle)
    assert not stand_in.allocator.live


@pytest.mark.parametrize("name", EVERY)
def test_memory_comes_back_from_a_refused_call(stand_in, name):
    stand_in.library.status = -1
    with pytest.raises(stand_in.binding.PaQ8Error):
        call(name, stand_in.binding)
    assert [e[0] for e in stand_in.allocator.events] == ["alloc", "call", "delete"]


@pytest.mark.parametrize("name", EVERY)
def test_memory_that_is_not_there_is_not_given_back(stand_in, monkeypatch, name):
    def alloc(need, handle):
        raise MemoryError("full")
    monkeypatch.setattr(stand_in.binding, "_raw_alloc", alloc)
    with pytest.raises(MemoryError, match="full"):
        call(name, stand_in.binding)
    assert not stand_in.allocator.events


@pytest.mark.parametrize("name", EVERY)
def test_no_memory_is_taken_beside_a_workspace(stand_in, name):
    import torch
    call(name, stand_in.binding, workspace=torch.zeros(NEED, dtype=torch.uint8))
    assert [e[0] for e in stand_in.allocator.events] == ["call"]


@pytest.mark.parametrize("lost", ["_raw_alloc", "_raw_delete"])
@pytest.mark.parametrize("name", EVERY)
def test_without_torchs_allocator_calls_a_tensor_is_the_workspace(stand_in, monkeypatch, name, lost):
    import torch
    asked, empty = [], torch.empty

    def noting(*a, **kw):
        t = empty(*a, **kw)
        if kw.get("dtype") is torch.uint8:
            asked.append(t.numel())
            stand_in.allocator.live[t.data_ptr()] = (t.numel(), None)
        return t
    monkeypatch.setattr(torch, "empty", noting)
    monkeypatch.setattr(stand_in.binding, lost, None)
    call(name, stand_in.binding)
    assert asked == [NEED] and stand_in.library.seen == [(NEED, None)] and len(stand_in.allocator.events) == 1


@pytest.mark.parametrize("there", [True, False])
def test_torchs_allocator_calls_are_looked_up(monkeypatch, there):
    import torch
    from int8_paged_kv_gb300 import _binding
    names = ("_cuda_cudaCachingAllocator_raw_alloc", "_cuda_cudaCachingAllocator_raw_delete")
    for name in names:
        if there:
            monkeypatch.setattr(torch._C, name, name, raising=False)
        else:
            monkeypatch.delattr(torch._C, name, raising=False)
    for name in ("_current_device", "_raw_stream", "_raw_alloc", "_raw_delete"):
        monkeypatch.setattr(_binding, name, None)
    monkeypatch.setattr(_binding, "_U32", ())
    with pytest.raises(TypeError, match="CUDA tensors"):
        _binding._current(torch.zeros(1))
    assert (_binding._raw_alloc, _binding._raw_delete) == (names if there else (None, None))


def test_the_order_of_tests_does_not_matter():
    """What an earlier call of the process looked up (torch's calls, for its device) does not reach the tests
    that stand in for the library: they pass behind calls on a GPU as well."""
    code = ("import sys, pytest\n"
            "from int8_paged_kv_gb300 import _binding as b\n"
            "def used(*a):\n"
            "    raise RuntimeError('the allocator of an earlier call')\n"
            "b._raw_alloc = b._raw_delete = used\n"
            "sys.exit(pytest.main(['-q', '-p', 'no:cacheprovider', '-m', 'not gpu', 'tests/test_workspace.py']))\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-2000:]


@gpu
@pytest.mark.parametrize("lost", ["_raw_alloc", "_raw_delete", None])
def test_results_do_not_depend_on_the_allocators_way(monkeypatch, lost):
    import torch
    from int8_paged_kv_gb300 import _binding, build
    build.build()
    from tests.test_window import Window
    c = Window(8, 2, 128, 16, [900, 500, 3000], [100, 50, 300], 600, 5, "bfloat16", seed=90)
    one = Window(8, 2, 128, 16, [900, 500, 3000], [1, 1, 1], 600, 5, seed=91)
    want = [c.run(), one.decode()]
    side = torch.cuda.Stream()
    if lost:
        monkeypatch.setattr(_binding, lost, None)
    for stream in (None, side, side.cuda_stream, 0, 1):
        torch.cuda.synchronize()
        got = [c.run(stream=stream), one.decode(stream=stream)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got)), stream
