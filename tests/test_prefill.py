"""Prompt attention over the paged int8 caches (pa_q8_prefill) against a plain
64-bit evaluation of its definition on the same cache words.

Tolerances.  f32 rows keep the library's bound, 1e-5 + 1e-4 |ref|.  f16 and
bf16 rows come back rounded to their type, at most u |ref| off (u = eps / 2:
2^-11, 2^-8), and their softmax weights (times the tokens' V scales) pass the
tensor cores as f16, each at most 2^-11 of itself off.  With W = sum w,
out = sum w V / W then moves by at most 2^-11 sum w |V| / W <= 2^-11 max_t |V_t|
over the tokens seen, rounded once more by the store.  So the bound is
1e-5 + (1e-4 + u) |ref| + 2^-11 (1 + u) max_t |V_t|.
"""
import numpy as np
import pytest

from tests.helpers import dense_context

gpu = pytest.mark.gpu
PAD = 0xFFFFFFFF
UNIT = {"float32": 0.0, "float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}


@pytest.fixture(scope="module")
def lib():
    from int8_paged_kv_gb300 import build
    build.build()
    import oracle
    oracle.build()


def plain(q, kc, vc, bt, lens, starts, scale, dim, block):
    """The definition in 64 bits: (out, largest |V| a row's group can see); q: [T, H, D]."""
    T, H, D = q.shape
    out, top = np.full((T, H, D), np.nan), np.zeros((T, H, D))
    hk = kc.shape[1]
    for s in range(len(lens)):
        lo, hi = int(starts[s]), int(starts[s + 1])
        c = min(int(lens[s]), bt.shape[1] * block)
        if hi <= lo:
            continue
        k = dense_context(kc, bt, s, c, dim)
        v = dense_context(vc, bt, s, c, dim)
        for h in range(H):
            g = h // (H // hk)
            z = q[lo:hi, h].astype(np.float64) @ k[:, g].T * scale
            sees = c - (hi - 1 - np.arange(lo, hi))
            z[np.arange(c)[None, :] >= sees[:, None]] = -np.inf
            m = z.max(axis=1, initial=-np.inf, keepdims=True)
            p = np.exp(z - np.where(np.isinf(m), 0.0, m))
            l = p.sum(axis=1, keepdims=True)
            out[lo:hi, h] = p @ v[:, g] / np.where(l == 0, 1.0, l)
            if c:
                top[lo:hi, h] = np.abs(v[:, g]).max(axis=0)
    return out, top


def check(got, want, top, dtype, what="", units=1.0):
    u = UNIT[dtype]
    tol = 1e-5 * units + (1e-4 + u) * np.abs(want) + (2.0 ** -11 * (1 + u) * top if u else 0.0)
    assert np.all(np.isfinite(got)), f"{what}: non-finite output"
    err = np.abs(got - want)
    worst = np.unravel_index(np.argmax(err / tol), err.shape)
    assert np.all(err <= tol), f"{what}: {int((err > tol).sum())} of {err.size} outside; at {worst} {got[worst]} for {want[worst]}"


class Case:
    """Ragged sequences over a poisoned pool: lens tokens cached, rows of them queried."""

    def __init__(self, H, Hk, D, B, lens, rows, dtype="float32", seed=0, first=0, behind=0, scale_mult=1.0, **kw):
        import torch
        from tests.gpu_helpers import dev_u32, random_case
        w, self.ok, self.ov, self.kc, self.vc = random_case(len(lens), H, Hk, D, B, lens, seed, scale_mult=scale_mult, **kw)
        self.w, self.D, self.B, self.Hk, self.dtype = w, D, B, Hk, dtype
        self.starts = np.concatenate([[0], np.cumsum(rows)]).astype(np.uint32) + np.uint32(first)
        self.T = int(self.starts[-1]) + behind
        rng = np.random.default_rng(seed + 1)
        self.q = torch.from_numpy(rng.standard_normal((self.T, H, D)).astype(np.float32)).cuda().to(getattr(torch, dtype))
        self.bt, self.cl, self.qs = dev_u32(w.block_tables), dev_u32(w.context_lens), dev_u32(self.starts)

    def run(self, q=None, out=None, **kw):
        import torch
        import int8_paged_kv_gb300 as pk
        q = self.q if q is None else q
        out = torch.full_like(q, float("nan")) if out is None else out
        pk.pa_q8_prefill(out, q, self.kc, self.vc, kw.pop("bt", self.bt), kw.pop("cl", self.cl), kw.pop("qs", self.qs),
                         num_kv_heads=self.Hk, block_size=self.B, scale=self.w.scale, num_blocks=self.w.num_blocks, **kw)
        return out

    def want(self, q=None, lens=None):
        q = self.q if q is None else q
        return plain(q.float().cpu().numpy(), self.ok, self.ov, self.w.block_tables,
                     self.w.context_lens if lens is None else lens, self.starts, self.w.scale, self.D, self.B)

    def checked(self, what="", **kw):
        got = self.run(**kw).float().cpu().numpy().astype(np.float64)
        ref, top = self.want()
        lo, hi = int(self.starts[0]), int(self.starts[-1])
        check(got[lo:hi], ref[lo:hi], top[lo:hi], self.dtype, what)
        assert np.all(np.isnan(got[:lo])) and np.all(np.isnan(got[hi:])), f"{what}: rows of no sequence were written"


@pytest.fixture(autouse=True)
def _clean(request):
    if "gpu" not in request.keywords:
        yield
        return
    request.getfixturevalue("lib")
    from tests.gpu_helpers import device_status
    device_status()
    yield


TYPES = ["float32", "float16", "bfloat16"]


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("H,Hk,D,B", [(4, 2, 64, 16), (32, 8, 128, 16), (16, 1, 256, 32), (6, 2, 128, 4),
                                      (5, 5, 64, 1024), (7, 1, 256, 8), (96, 1, 128, 64), (160, 1, 64, 16)])
def test_whole_prompts(H, Hk, D, B, dtype):
    from tests.gpu_helpers import device_status
    lens = [1, 37, 0, 128, 129, 300, 31]
    Case(H, Hk, D, B, lens, lens, dtype, seed=H + D).checked(f"{H}/{Hk} x {D}")
    assert device_status() == 0


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_chunks_behind_a_prefix(D, dtype):
    """Rows that are the last of a longer context: none, one, a few, many; more rows than tokens."""
    from tests.gpu_helpers import device_status
    lens, rows = [700, 1000, 64, 5, 513, 0, 257], [1, 130, 64, 9, 0, 3, 256]
    Case(8, 2, D, 16, lens, rows, dtype, seed=D).checked(f"head size {D}")
    assert device_status() == 0


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", [1, 3, 16, 70])
def test_few_rows_over_long_contexts(rows, dtype):
    """The context is cut into pieces and joined."""
    from tests.gpu_helpers import device_status
    Case(8, 2, 128, 16, [9000, 20011], [rows, rows], dtype, seed=rows).checked(f"{rows} rows")
    assert device_status() == 0


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("H,Hk,rows", [(64, 64, [3, 2]), (64, 32, [200, 150])])
def test_unequal_contexts_of_many_heads(H, Hk, rows, dtype):
    """As many items as SMs, of two lengths: cut finely, joined in an order of their own."""
    import torch
    from tests.gpu_helpers import device_status
    c = Case(H, Hk, 64, 16, [8192, 4096], rows, dtype, seed=Hk)
    c.checked(f"{H}/{Hk} heads")
    assert torch.equal(c.run(), c.run())
    assert device_status() == 0


@gpu
@pytest.mark.parametrize("dtype", TYPES)
def test_long_prompt(dtype):
    Case(4, 1, 128, 32, [2500, 1031], [2500, 900], dtype, seed=3).checked("long prompt")


@gpu
@pytest.mark.parametrize("H,Hk,D,rows,ctx", [(16, 8, 128, 500, 40000), (4, 2, 64, 700, 30000), (16, 1, 256, 400, 30000),
                                             (32, 8, 128, 5000, 9000)])
def test_f32_sums_over_long_contexts(H, Hk, D, rows, ctx):
    """V with a mean, so that every term adds up.  An accumulator of the tensor cores loses half a last
    bit (2^-24 of itself) on average at each of its at most 32 x 8 steps, 1.5e-5 of it in all at most;
    the bound is 2e-5 of the result (2-norm).  Without sums of its
    own, 30,000 tokens are 3,750 steps and more: over 1e-4."""
    import torch
    from tests.gpu_helpers import device_status
    c = Case(H, Hk, D, 16, [ctx, 100], [rows, 100], seed=D)
    words = c.vc.clone()
    codes = words[..., :-1].contiguous().view(torch.int8)
    words[..., :-1] = (codes // 2 + 60).to(torch.int8).view(torch.int32)        # codes -4 .. 123
    c.vc.copy_(words)
    got = c.run().double()
    k, v = (x[c.bt[0].long()].permute(1, 0, 2, 3).reshape(Hk, -1, D // 4 + 1)[:, :ctx] for x in (c.kc, c.vc))
    k, v = (x[..., :-1].contiguous().view(torch.int8).double() * x[..., -1:].contiguous().view(torch.float32).double()
            for x in (k, v))
    at = torch.arange(0, rows, max(1, rows // 60), device="cuda")               # some of the rows
    q = c.q[at].double().view(len(at), Hk, H // Hk, D)
    z = torch.einsum("ighd,gtd->ight", q, k) * c.w.scale
    seen = torch.arange(ctx, device="cuda")[None] < ctx - (rows - 1 - at)[:, None]
    p = torch.softmax(z.masked_fill(~seen[:, None, None], -np.inf), -1)
    want = torch.einsum("ight,gtd->ighd", p, v).reshape(len(at), H, D)
    assert float((got[at] - want).norm() / want.norm()) <= 2e-5
    assert device_status() == 0


@gpu
@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_row_per_sequence_is_the_decode(D):
    """One row per sequence: the definition is pa_q8_decode's."""
    import torch
    import int8_paged_kv_gb300 as pk
    from tests.gpu_helpers import assert_close
    lens = [1, 100, 777, 64, 0, 333]
    c = Case(8, 2, D, 16, lens, [1] * len(lens), seed=D)
    got = c.run().cpu().numpy()
    ref = torch.full_like(c.q, float("nan"))
    pk.pa_q8_decode(ref, c.q, c.kc, c.vc, c.bt, c.cl, num_kv_heads=2, block_size=16, scale=c.w.scale)
    want, _ = c.want()
    assert_close(got, want, "prefill")
    assert_close(ref.cpu().numpy(), want, "decode")


@gpu
@pytest.mark.parametrize("dtype", TYPES)
def test_rows_before_and_behind_the_sequences_stay(dtype):
    Case(8, 2, 128, 16, [50, 200], [50, 77], dtype, seed=5, first=3, behind=130).checked("outer rows")


@gpu
@pytest.mark.parametrize("dtype", TYPES)
def test_strided_rows(dtype):
    """q a column slice of fused QKV rows, out a slice of wider rows."""
    import torch
    c = Case(8, 2, 128, 16, [150, 33], [150, 33], dtype, seed=6)
    fused = torch.randn((c.T, 12 * 128), device="cuda").to(c.q.dtype)
    fused[:, 256:256 + 1024] = c.q.reshape(c.T, -1)
    wide = torch.full((c.T, 1024 + 64), 7.0, device="cuda", dtype=c.q.dtype)
    c.run(q=fused[:, 256:1280].unflatten(1, (8, 128)), out=wide[:, 64:].unflatten(1, (8, 128)))
    assert torch.equal(wide[:, 64:].reshape(c.T, 8, 128), c.run())
    assert bool((wide[:, :64] == 7.0).all())


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("mult", [-1.0, 0.0, 3.0])
def test_softmax_scales(mult, dtype):
    Case(8, 2, 128, 16, [300, 70], [300, 70], dtype, seed=8, scale_mult=mult).checked(f"scale x {mult}")


@gpu
@pytest.mark.parametrize("dtype", TYPES)
def test_value_scales_that_rise_and_fall(dtype):
    """V magnitudes over 12 powers of two along the context, up in one sequence and down in the other;
    errors are relative to the largest V seen, so each row is compared in those units."""
    c = Case(8, 2, 128, 16, [900, 600], [900, 300], dtype, seed=9,
             v_token_mult=lambda p, n: np.where(n == 900, 2.0 ** (12 * p / n), 2.0 ** (-12 * p / n)))
    got = c.run().float().cpu().numpy().astype(np.float64)
    want, top = c.want()
    check(got, want, top, dtype, "value scales", units=np.maximum(1.0, top))


@gpu
@pytest.mark.parametrize("dtype", TYPES)
def test_query_magnitudes(dtype):
    """Rows from 2^-60 to 2^4 (f16: from its smallest normal numbers): tiny ones give the mean of V."""
    import torch
    c = Case(8, 2, 128, 16, [400], [400], dtype, seed=10)
    low = -12 if dtype == "float16" else -60
    c.q *= torch.exp2(torch.linspace(low, 4, 400, device="cuda"))[:, None, None].to(c.q.dtype)
    got = c.run().float().cpu().numpy().astype(np.float64)
    want, top = c.want()
    check(got, want, top, dtype, "query magnitudes", units=16.0)


@gpu
@pytest.mark.parametrize("dtype", TYPES)
def test_zero_vectors(dtype):
    """All-zero K and V vectors carry scale 1.0 and zero codes; a zero q weighs all tokens alike."""
    import torch
    c = Case(8, 2, 128, 16, [200, 90], [200, 90], dtype, seed=11)
    zero = np.random.default_rng(4).random(c.ok.shape[:3]) < 0.1
    for host, dev in ((c.ok, c.kc), (c.ov, c.vc)):
        host[zero] = 0
        host[zero, -1] = np.float32(1.0).view(np.uint32)
        dev.copy_(torch.from_numpy(host.view(np.int32)))
    c.q[5] = 0
    c.checked("zero vectors")


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_what_a_mask_hides_stays_hidden(D, dtype):
    """NaN and infinite scales at later positions of a sequence, behind its end and in a neighbour's
    rows leave the rows that do not see them bit for bit as they were; the rows that see one are not finite."""
    import torch
    c = Case(8, 2, D, 16, [333, 140], [333, 140], dtype, seed=12)
    clean = c.run()
    for cache, bits in ((c.kc, 0x7FC00000), (c.vc, 0x7F800000), (c.vc, 0x7FC00000)):
        keep = cache.clone()
        for s, t in ((0, 200), (1, 139)):
            cache[int(c.w.block_tables[s, t // 16]), :, t % 16, -1] = bits
        cache[int(c.w.block_tables[1, 8]), :, 12:, -1] = bits                  # behind the end, same page
        got = c.run()
        assert torch.equal(got[:200], clean[:200]) and torch.equal(got[333:472], clean[333:472])
        assert not bool(torch.isfinite(got[200:333]).all(-1).any()) and not bool(torch.isfinite(got[472]).all(-1).any())
        cache.copy_(keep)
    # a row of q that is not finite spoils itself alone
    q = c.q.clone()
    q[17], q[300, 3] = float("nan"), float("inf")
    got = c.run(q=q)
    keep = torch.ones(c.T, dtype=torch.bool, device="cuda")
    keep[17] = keep[300] = False
    assert torch.equal(got[keep], clean[keep])
    assert torch.equal(got[300, :3], clean[300, :3]) and torch.equal(got[300, 4:], clean[300, 4:])
    assert bool(torch.isnan(got[17]).all())


@gpu
def test_contexts_longer_than_the_table():
    """context_lens beyond the table's tokens are cut to them, for the rows' places too."""
    import torch
    from tests.gpu_helpers import dev_u32
    c = Case(8, 2, 128, 16, [64, 64], [64, 20], seed=13)
    got = c.run(cl=dev_u32(np.array([10 ** 6, 0xFFFFFFFF], dtype=np.uint32)))
    assert torch.equal(got, c.run())


@gpu
def test_bad_pages_and_bad_bounds_are_flagged():
    import torch
    import int8_paged_kv_gb300 as pk
    from tests.gpu_helpers import dev_u32, device_status
    c = Case(8, 2, 128, 16, [40, 40, 40], [40, 40, 40], seed=14)
    clean = c.run()
    bt = c.w.block_tables.copy()
    bt[1, 1] = 1 << 30
    got = c.run(bt=dev_u32(bt))
    assert device_status() == pk.PA_Q8_DEV_BAD_BLOCK
    assert torch.equal(got[:40], clean[:40]) and torch.equal(got[80:], clean[80:])
    for bad in ([0, 40, 30, 120], [0, 40, 80, 121], [0, 40, 0xFFFFFFFF, 120], [0, 40, 0, 40]):
        got = c.run(qs=dev_u32(np.array(bad, dtype=np.uint32)))
        assert device_status() == pk.PA_Q8_DEV_BAD_ROWS
        assert torch.equal(got[:40], clean[:40])
        assert bool(torch.isnan(got[80:]).all())


@gpu
def test_many_sequences_that_claim_the_same_rows():
    """Bounds that swing up and down over 3000 sequences: only the first one's rows are its own."""
    import torch
    import int8_paged_kv_gb300 as pk
    from tests.gpu_helpers import dev_u32, device_status
    c = Case(8, 2, 64, 16, [64], [64], seed=21)
    S = 3000
    starts = dev_u32(np.array([0, 64] * (S // 2) + [0], dtype=np.uint32))
    got = c.run(bt=c.bt.repeat(S, 1).contiguous(), cl=c.cl.repeat(S), qs=starts)
    assert torch.equal(got, c.run()) and device_status() == pk.PA_Q8_DEV_BAD_ROWS


@gpu
@pytest.mark.parametrize("dtype", TYPES)
def test_captured_and_replayed(dtype):
    """One capture, new lengths, rows and queries in the same buffers: the lengths decide on the device."""
    import torch
    import int8_paged_kv_gb300 as pk
    from tests.gpu_helpers import dev_u32
    c = Case(8, 2, 128, 16, [900, 500, 64], [200, 30, 26], dtype, seed=15)
    ws = torch.empty(pk.pa_q8_prefill_workspace_size(c.T, 3, 8, 2, 128, 16, c.bt.shape[1], c.q.dtype),
                     dtype=torch.uint8, device="cuda")
    out = torch.empty_like(c.q)
    c.run(out=out, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run(out=out, workspace=ws)
    for lens, rows in (([900, 500, 64], [200, 30, 26]), ([10, 480, 0], [5, 250, 0]), ([880, 1, 60], [1, 1, 60])):
        c.cl.copy_(dev_u32(np.array(lens, dtype=np.uint32)))
        c.qs.copy_(dev_u32(np.concatenate([[0], np.cumsum(rows)]).astype(np.uint32)))
        c.q.normal_()
        ws.fill_(0xFF)
        out.fill_(7.0)
        g.replay()
        again = torch.full_like(out, 7.0)
        c.run(out=again)
        assert torch.equal(out, again)


@gpu
def test_streams_of_their_own():
    """Two calls at once, each with its stream and workspace, as alone; workspaces left to the binding."""
    import torch
    cs = [Case(8, 2, 128, 16, [3000, 500], [300, 500], t, seed=16 + i) for i, t in enumerate(("float32", "bfloat16"))]
    alone = [c.run() for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    outs = [torch.full_like(c.q, float("nan")) for c in cs]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, st, out in zip(cs, streams, outs):
            c.run(out=out, stream=st)
    torch.cuda.synchronize()
    for a, b in zip(alone, outs):
        assert torch.equal(a, b)


@gpu
def test_the_same_call_gives_the_same_bits():
    import torch
    c = Case(32, 8, 128, 16, [5000, 700, 90], [40, 700, 90], "bfloat16", seed=18)
    first = c.run()
    for _ in range(5):
        assert torch.equal(c.run(), first)


@gpu
def test_pages_past_32bit_offsets():
    """Pages whose words lie past 2^32: the same bits as from a compact pool."""
    import torch
    import int8_paged_kv_gb300 as pk
    from tests.gpu_helpers import device_status
    H, Hk, D, B = 8, 8, 128, 16
    NB = 1_100_000
    c = Case(H, Hk, D, B, [300, 77], [300, 20], seed=19)
    ids = torch.arange(c.w.num_blocks, device="cuda")
    far = (NB - 1 - ids).to(torch.int32)
    kc = torch.empty((NB, Hk, B, D // 4 + 1), dtype=torch.int32, device="cuda")
    vc = torch.empty_like(kc)
    kc[NB - c.w.num_blocks:], vc[NB - c.w.num_blocks:] = c.kc.flip(0), c.vc.flip(0)
    bt = torch.where(c.bt == -1, c.bt, far[c.bt.clamp(min=0).long()]).contiguous()
    out = torch.full_like(c.q, float("nan"))
    pk.pa_q8_prefill(out, c.q, kc, vc, bt, c.cl, c.qs, num_kv_heads=Hk, block_size=B, scale=c.w.scale)
    assert torch.equal(out, c.run()) and device_status() == 0


@gpu
def test_refusals_of_the_binding():
    import torch
    import int8_paged_kv_gb300 as pk
    c = Case(8, 2, 128, 16, [40], [40], seed=20)
    with pytest.raises(TypeError):
        c.run(q=c.q.double(), out=c.q.double())
    with pytest.raises(ValueError):
        c.run(out=torch.empty_like(c.q, dtype=torch.float16))
    with pytest.raises(ValueError):
        c.run(q=c.q.transpose(1, 2).contiguous().transpose(1, 2))
    with pytest.raises(ValueError):
        c.run(qs=c.qs[:1])
    with pytest.raises(TypeError):
        c.run(bt=c.bt.cpu())
    with pytest.raises(ValueError):
        c.run(bt=torch.cat([c.bt, c.bt], 1)[:, ::2])
    with pytest.raises(pk.PaQ8Error, match="workspace too small"):
        c.run(workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))
    with pytest.raises(pk.PaQ8Error, match="misaligned"):
        flat = torch.empty(c.q.numel() + 1, device="cuda")[1:]
        c.run(q=flat.view(c.q.shape))
    assert c.run(q=c.q[:0], out=c.q[:0]).shape[0] == 0


def test_argument_errors(lib):
    """Status codes of the C entry point, none of which touches a device."""
    import ctypes
    from int8_paged_kv_gb300 import _binding
    L = _binding.lib()
    ok, odd = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10008)

    def call(out=ok, q=ok, dtype=0, os_=1024, qs=1024, kc=ok, bt=ok, T=40, S=2, H=8, Hk=2, D=128, B=16, Nb=4, nb=8):
        return L.pa_q8_prefill(out, q, dtype, os_, qs, kc, ok, bt, ok, ok, T, S, H, Hk, D, B, Nb, nb, 0.1, None, 0, None)

    for kw, code in ((dict(dtype=3), -1), (dict(dtype=-1), -1), (dict(T=-1), -1), (dict(S=0), -1), (dict(Hk=3), -1),
                     (dict(D=96), -2), (dict(B=12), -2), (dict(nb=0), -1), (dict(os_=1023), -1), (dict(qs=1000), -1),
                     (dict(q=None), -1), (dict(bt=None), -1), (dict(q=odd), -3), (dict(out=odd), -3), (dict(kc=odd), -3),
                     (dict(qs=1026), -3), (dict(dtype=1, os_=1028), -3), (dict(H=8194, Hk=2, qs=1 << 21, os_=1 << 21), -2),
                     (dict(T=(1 << 30) + 1), -2)):
        assert call(**kw) == code, kw
    assert call(T=0, q=None) == 0                                     # nothing to do, nothing looked at
    assert L.pa_q8_prefill_workspace_size(40, 2, 8, 2, 128, 16, 4, 0) > 0
    assert L.pa_q8_prefill_workspace_size(40, 2, 8, 2, 100, 16, 4, 0) == 0
    assert L.pa_q8_prefill_workspace_size(40, 2, 8, 2, 128, 16, 4, 3) == 0
