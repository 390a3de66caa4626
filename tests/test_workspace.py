"""Workspaces that the binding allocates itself: alive until the library has
queued its work, and from the pool of the stream that the work is queued on,
so that nobody else writes to them while it runs.

On the CPU the library is a stand-in and the tensors are CPU tensors: what is
looked at is the tensor behind the address that the library gets.
"""
import contextlib
import types
import weakref

import pytest

gpu = pytest.mark.gpu
NEED = 4096


class Library:
    """Stands in for libpa_q8.so: every size query says NEED, every call notes whether the workspace lives."""

    def __init__(self, seen):
        self.seen, self.alive = seen, []

    def __getattr__(self, name):
        if name.endswith("workspace_size") or name.endswith("workspace_size_ex"):
            return lambda *a: NEED

        def call(*args):
            addresses = [getattr(a, "value", a) for a in args]
            living = {r().data_ptr(): r.stream for r in self.seen if r() is not None}
            self.alive.append([living[a] for a in addresses if a in living])
            return 0
        return call


class Ref(weakref.ref):
    stream = None


@pytest.fixture
def stand_in(monkeypatch):
    import torch
    from int8_paged_kv_gb300 import _binding
    seen, inside, empty = [], [None], torch.empty

    def noting(*a, **kw):
        t = empty(*a, **kw)
        if kw.get("dtype") is torch.uint8:
            r = Ref(t)
            r.stream = inside[0]
            seen.append(r)
        return t

    @contextlib.contextmanager
    def stream_of(stream):
        before, inside[0] = inside[0], stream
        yield
        inside[0] = before

    library = Library(seen)
    monkeypatch.setattr(_binding, "lib", lambda: library)
    monkeypatch.setattr(_binding, "_current", lambda t: -1)
    monkeypatch.setattr(_binding, "_queue", lambda stream, device: 0)
    monkeypatch.setattr(_binding, "_stream", lambda stream: 0)
    monkeypatch.setattr(_binding, "_cuda", lambda t, dtype, name: t.data_ptr())
    monkeypatch.setattr(_binding, "_U32", (torch.int32, torch.uint32))
    monkeypatch.setattr(torch, "empty", noting)
    monkeypatch.setattr(torch.cuda, "stream", stream_of)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, stream: None)
    return types.SimpleNamespace(library=library, binding=_binding)


def pool_and_caches():
    import torch

    def i32(*shape):
        return torch.zeros(shape, dtype=torch.int32)
    pool = (i32(4, 4), i32(4), i32(16), i32(16), i32(1))
    return i32, pool, i32(16, 2, 16, 33), torch.zeros((4, 8, 128))


def calls(names, b, **kw):
    i32, pool, cache, q = pool_and_caches()
    one, sizes = i32(1), dict(num_kv_heads=2, block_size=16, scale=0.1)
    rows = q[:, None].contiguous()
    every = {
        "prefill": lambda: b.pa_q8_prefill(q.clone(), q, cache, cache, pool[0], pool[1], i32(5), **sizes, **kw),
        "extend": lambda: b.pa_q8_extend_seqs(*pool, one, one, block_size=16, **kw),
        "fork": lambda: b.pa_q8_fork_seqs(*pool, one, one, one, one, block_size=16, **kw),
        "compact": lambda: b.pa_q8_compact_blocks(*pool, i32(8), i32(8), block_size=16, **kw),
        "decode": lambda: b.pa_q8_decode(q.clone(), q, cache, cache, pool[0], pool[1], **sizes, **kw),
        "decode_rows": lambda: b.pa_q8_decode_rows(rows.clone(), rows, cache, cache, pool[0], pool[1], **sizes, **kw),
        "decode_append": lambda: b.pa_q8_decode_append(rows.clone(), rows, q[:, None, :2].contiguous(),
                                                       q[:, None, :2].contiguous(), cache, cache, pool[0], pool[1],
                                                       **sizes, **kw),
        "f32_decode": lambda: b.pa_f32_decode(q.clone(), q, cache, cache, pool[0], pool[1], **sizes, **kw),
        "q8c_decode": lambda: b.pa_q8c_decode(q.clone(), q, cache, cache, pool[1], num_kv_heads=2, max_t=64, scale=0.1,
                                              **kw),
    }
    return every[names]


EVERY = ["prefill", "extend", "fork", "compact", "decode", "decode_rows", "decode_append", "f32_decode", "q8c_decode"]


@pytest.mark.parametrize("name", EVERY)
def test_the_workspace_lives_until_the_call_is_queued(stand_in, name):
    calls(name, stand_in.binding)()
    assert stand_in.library.alive == [[None]]


@pytest.mark.parametrize("name", EVERY)
def test_the_workspace_comes_from_the_streams_own_pool(stand_in, monkeypatch, name):
    import torch
    side = types.SimpleNamespace(cuda_stream=64)
    monkeypatch.setattr(torch.cuda, "Stream", types.SimpleNamespace)
    calls(name, stand_in.binding, stream=side)()
    assert stand_in.library.alive == [[side]]


@pytest.mark.parametrize("handle,default", [(0, True), (1, True), (64, False)])
def test_streams_given_by_their_handle(stand_in, monkeypatch, handle, default):
    """0 and 1 are the legacy default stream, which torch has an object of its own for."""
    import torch
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device: "default")
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device: handle)
    calls("extend", stand_in.binding, stream=handle)()
    assert stand_in.library.alive == [["default" if default else handle]]


def test_no_private_call_of_torch_is_needed(monkeypatch):
    """Without torch's short way to a stream's handle its public functions give it."""
    import torch
    from int8_paged_kv_gb300 import _binding
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.setattr(_binding, "_current_device", None)
    monkeypatch.setattr(_binding, "_raw_stream", None)
    with pytest.raises(TypeError, match="CUDA tensors"):
        _binding._current(torch.zeros(1))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device: types.SimpleNamespace(cuda_stream=100 + device))
    assert _binding._queue(None, 3) == 103 and _binding._queue(7, 3) == 7


@gpu
def test_two_streams_with_work_pending():
    """Calls that leave the workspace to the binding, on two streams at once and behind writes that are
    pending on the current stream to memory that was freed there: workspaces apart, results as alone."""
    import torch
    from int8_paged_kv_gb300 import _binding, build
    build.build()
    from tests.test_prefill import Case
    cs = [Case(8, 2, 128, 16, [3000, 500], [300, 500], t, seed=16 + i) for i, t in enumerate(("float32", "bfloat16"))]
    alone = [c.run() for c in cs]
    need = [_binding.pa_q8_prefill_workspace_size(c.T, 2, 8, 2, 128, 16, c.bt.shape[1], c.q.dtype) for c in cs]
    streams, outs = [torch.cuda.Stream() for _ in cs], [torch.full_like(c.q, float("nan")) for c in cs]
    big = torch.zeros(1 << 28, device="cuda")                            # 1 GB
    asked = []

    class Noting:
        """The library, with the workspace of each prompt call noted."""
        def __getattr__(self, name):
            real = getattr(library, name)
            if name != "pa_q8_prefill":
                return real

            def call(*a):
                asked.append((a[-3], a[-2]))
                return real(*a)
            return call

    library = _binding.lib()
    torch.cuda.synchronize()
    with pytest.MonkeyPatch.context() as patch:
        patch.setattr(_binding, "lib", lambda noting=Noting(): noting)
        for turn in range(8):
            freed = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in need]
            for _ in range(10):
                big.add_(1.0)                                            # some 4 ms on the current stream
            for f in freed:
                f.fill_(0xA5)
            at_freed = [(f.data_ptr(), f.numel()) for f in freed]
            del f, freed
            del asked[:]
            for _ in range(3):
                for c, st, out in zip(cs, streams, outs):
                    c.run(out=out, stream=st)
            spans = {st: {a for k, a in enumerate(asked) if k % 2 == i} for i, st in enumerate(streams)}
            every = [(a, n, i) for i, st in enumerate(streams) for a, n in spans[st]] + [(a, n, 2) for a, n in at_freed]
            for a, n, i in every:
                assert all(i == j or a + n <= b or b + m <= a for b, m, j in every), "workspaces shared between streams"
            torch.cuda.synchronize()
            for a, out in zip(alone, outs):
                assert torch.equal(a, out), turn
                out.fill_(float("nan"))
            torch.cuda.synchronize()


@gpu
def test_streams_by_object_and_by_handle():
    """A stream of torch, its handle, the legacy default stream's two handles, a stream of another library's."""
    import torch
    from int8_paged_kv_gb300 import build
    build.build()
    from tests.test_prefill import Case
    c = Case(8, 2, 128, 16, [3000, 50], [200, 50], "bfloat16", seed=30)
    alone = c.run()
    side = torch.cuda.Stream()
    other = types.SimpleNamespace(cuda_stream=side.cuda_stream)
    for stream in (side, side.cuda_stream, other, torch.cuda.ExternalStream(side.cuda_stream), 0, 1,
                   torch.cuda.default_stream()):
        out = torch.full_like(c.q, float("nan"))
        torch.cuda.synchronize()
        c.run(out=out, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(out, alone), stream
