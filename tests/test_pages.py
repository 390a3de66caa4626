"""The page pool (extend, fork, free, compact) and the page copies against a
plain Python model of the pool: lists, one request after the other.  All
values are whole numbers and have to be equal, the free stack's order among
them."""
import numpy as np
import pytest

gpu = pytest.mark.gpu
PAD = 0xFFFFFFFF


@pytest.fixture(scope="module")
def lib():
    from int8_paged_kv_gb300 import build
    build.build()


@pytest.fixture(autouse=True)
def _clean(request):
    if "gpu" in request.keywords:
        request.getfixturevalue("lib")
        import int8_paged_kv_gb300 as pk
        pk.pa_q8_device_status()
    yield


class Model:
    """The pool as its documentation describes it."""

    def __init__(self, rows, width, pages, size):
        self.table = [[0] * width for _ in range(rows)]
        self.lens, self.refs, self.stack = [0] * rows, [0] * pages, list(range(pages))[::-1]
        self.size, self.width, self.flags = size, width, 0

    def held(self, s):
        return -(-self.lens[s] // self.size)

    def extend(self, seqs, new):
        named, want, room = set(), 0, len(self.stack)
        for s, n in zip(seqs, new):
            if s >= len(self.lens) or s in named or n > self.width * self.size:
                self.flags |= 8
                named.add(s)
                continue
            named.add(s)
            if n <= self.lens[s]:
                continue
            need = -(-n // self.size) - self.held(s)
            want += need
            if want > room:
                self.flags |= 16
                continue
            for k in range(need):
                b = self.stack.pop()
                self.table[s][self.held(s) + k] = b
                self.refs[b] = 1
            self.lens[s] = n

    def fork(self, parents, children):
        before = list(self.lens)
        named, src, dst = set(), [], []
        for p, c in zip(parents, children):
            src.append(PAD)
            dst.append(PAD)
            if max(p, c) >= len(before) or p == c or c in named or before[c]:
                self.flags |= 8
                if c < len(before):
                    named.add(c)
                continue
            named.add(c)
            whole, part = divmod(before[p], self.size)
            if part:
                if not self.stack:
                    self.flags |= 16
                    continue
                src[-1], dst[-1] = self.table[p][whole], self.stack.pop()
                self.table[c][whole] = dst[-1]
                self.refs[dst[-1]] = 1
            for j in range(whole):
                self.table[c][j] = self.table[p][j]
                self.refs[self.table[p][j]] += 1
            self.lens[c] = before[p]
        return src, dst

    def free(self, seqs):
        gone = []
        for s in seqs:
            if s >= len(self.lens):
                self.flags |= 8
                continue
            for j in range(self.held(s)):
                b = self.table[s][j]
                self.refs[b] -= 1
                if self.refs[b] == 0:
                    gone.append(b)
            self.lens[s] = 0
        self.stack += sorted(gone)

    def compact(self):
        used = [b for b, r in enumerate(self.refs) if r]
        live = len(used)
        src = [b for b in used if b >= live]
        dst = [b for b in range(live) if not self.refs[b]]
        where = dict(zip(src, dst))
        for s in range(len(self.lens)):
            for j in range(self.held(s)):
                self.table[s][j] = where.get(self.table[s][j], self.table[s][j])
        for a, b in where.items():
            self.refs[b], self.refs[a] = self.refs[a], 0
        self.stack = list(range(live, len(self.refs)))[::-1]
        return src, dst


class Pool:
    """The same pool on the device."""

    def __init__(self, rows, width, pages, size):
        import torch
        import int8_paged_kv_gb300 as pk
        self.size = size
        self.table = torch.zeros((rows, width), dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(rows, dtype=torch.int32, device="cuda")
        self.refs = torch.full((pages,), 77, dtype=torch.int32, device="cuda")
        self.stack = torch.full((pages,), -5, dtype=torch.int32, device="cuda")
        self.count = torch.full((1,), 99, dtype=torch.int32, device="cuda")
        pk.pa_q8_pool_init(self.refs, self.stack, self.count)

    @property
    def all(self):
        return self.table, self.lens, self.refs, self.stack, self.count

    def check(self, m, what=""):
        import int8_paged_kv_gb300 as pk
        assert self.lens.tolist() == m.lens, what
        assert self.table.tolist() == m.table, what
        assert self.refs.tolist() == m.refs, what
        assert self.count.tolist() == [len(m.stack)], what
        assert self.stack[:len(m.stack)].tolist() == m.stack, what
        assert pk.pa_q8_device_status() == m.flags, what
        m.flags = 0


def u32(values):
    import torch
    return torch.from_numpy(np.array(values, dtype=np.uint32).view(np.int32)).cuda()


def as_u32(t):
    return t.cpu().numpy().view(np.uint32).tolist()


def both(pool, m, op, *args):
    """One call on the device and in the model; the pools have to be equal after it."""
    import torch
    import int8_paged_kv_gb300 as pk
    if op == "extend":
        pk.pa_q8_extend_seqs(*pool.all, u32(args[0]), u32(args[1]), block_size=pool.size)
        m.extend(*args)
    elif op == "fork":
        src, dst = u32([5] * len(args[0])), u32([5] * len(args[0]))
        pk.pa_q8_fork_seqs(*pool.all, u32(args[0]), u32(args[1]), src, dst, block_size=pool.size)
        assert (as_u32(src), as_u32(dst)) == m.fork(*args)
    elif op == "free":
        pk.pa_q8_free_seqs(*pool.all, u32(args[0]), block_size=pool.size)
        m.free(*args)
    else:
        n = pool.refs.numel() // 2 + args[0]
        src, dst = torch.empty(n, dtype=torch.int32, device="cuda"), torch.empty(n, dtype=torch.int32, device="cuda")
        pk.pa_q8_compact_blocks(*pool.all, src, dst, block_size=pool.size)
        a, b = m.compact()
        assert as_u32(src) == a + [PAD] * (n - len(a)) and as_u32(dst) == b + [PAD] * (n - len(b))
        assert as_u32(pool.stack)[len(m.stack):] == [PAD] * (pool.refs.numel() - len(m.stack))
    pool.check(m, f"{op} {args}")


@gpu
@pytest.mark.parametrize("rows,width,pages,size", [(6, 9, 40, 4), (1, 1, 1, 16), (40, 30, 700, 16), (300, 5, 9001, 32),
                                                   (9, 64, 513, 1024)])
def test_random_calls(rows, width, pages, size):
    rng = np.random.default_rng(rows)
    pool, m = Pool(rows, width, pages, size), Model(rows, width, pages, size)
    pool.check(m, "init")
    for step in range(40):
        op = ["extend", "extend", "fork", "free", "compact"][int(rng.integers(5))]
        n = int(rng.integers(1, 2 * rows + 2))
        if op == "extend":
            # now and then a row out of range, a row named twice, a length beyond the table
            both(pool, m, op, rng.integers(0, rows + (step % 7 == 0), n).tolist(),
                 np.minimum(rng.integers(0, width * size + 1 + (step % 5 == 0), n),
                            rng.integers(1, width * size + 2, n)).tolist())
        elif op == "fork":
            both(pool, m, op, rng.integers(0, rows + (step % 7 == 0), n).tolist(),
                 rng.integers(0, rows + (step % 7 == 0), n).tolist())
        elif op == "free":
            both(pool, m, op, rng.integers(0, rows + (step % 7 == 0), max(1, n // 4)).tolist())
        else:
            both(pool, m, op, int(rng.integers(3)))


@gpu
def test_more_requests_than_threads():
    """Scans that go on from one sweep of the planning threads to the next."""
    rows = 3000
    rng = np.random.default_rng(1)
    pool, m = Pool(rows, 6, 30000, 4), Model(rows, 6, 30000, 4)
    both(pool, m, "extend", list(range(0, rows, 2)), rng.integers(0, 25, rows // 2).tolist())
    both(pool, m, "fork", list(range(0, rows, 2)), list(range(1, rows, 2)))
    both(pool, m, "fork", list(range(0, rows, 2)) * 2, list(range(1, rows, 2)) * 2)
    both(pool, m, "free", rng.permutation(rows)[:2000].tolist() * 2)
    both(pool, m, "compact", 0)
    both(pool, m, "extend", rng.integers(0, rows, 5000).tolist(), rng.integers(0, 25, 5000).tolist())


@gpu
def test_a_pool_that_runs_out():
    pool, m = Pool(8, 10, 20, 4), Model(8, 10, 20, 4)
    both(pool, m, "extend", [0, 1, 2, 3], [40, 39, 1, 0])                # 20 pages, then one too many
    both(pool, m, "fork", [0, 1, 0], [4, 5, 6])                          # whole pages only: no page needed
    both(pool, m, "extend", [4, 2], [40, 0])
    both(pool, m, "free", [0])
    both(pool, m, "free", [4, 6])
    both(pool, m, "extend", [2, 3, 0, 7], [40, 1, 0xFFFFFFFF, 4])


@gpu
def test_a_page_shared_by_every_row():
    pool, m = Pool(500, 3, 600, 16), Model(500, 3, 600, 16)
    both(pool, m, "extend", [0], [40])
    both(pool, m, "fork", [0] * 499, list(range(1, 500)))
    both(pool, m, "free", list(range(0, 500, 2)))
    both(pool, m, "compact", 0)
    both(pool, m, "free", list(range(500)))


@gpu
def test_rows_freed_by_mistake_are_flagged():
    """A table that names a free page, or a page that does not exist: flagged, counts as they were."""
    import torch
    import int8_paged_kv_gb300 as pk
    pool = Pool(4, 8, 32, 4)
    pk.pa_q8_extend_seqs(*pool.all, u32([0, 1]), u32([32, 32]), block_size=4)
    pool.table[1] = pool.table[0]                                        # row 1 holds row 0's pages by mistake
    pk.pa_q8_free_seqs(*pool.all, u32([0, 1]), block_size=4)
    assert pk.pa_q8_device_status() == pk.PA_Q8_DEV_BAD_BLOCK
    assert pool.refs.tolist() == [0] * 8 + [1] * 8 + [0] * 16
    assert sorted(pool.stack[:24].tolist()) == list(range(8)) + list(range(16, 32)) and pool.count.item() == 24
    pool.table[2, 0], pool.lens[2] = 1 << 20, 4
    for call in (lambda: pk.pa_q8_free_seqs(*pool.all, u32([2]), block_size=4),
                 lambda: pk.pa_q8_compact_blocks(*pool.all, torch.empty_like(pool.stack), torch.empty_like(pool.stack),
                                                 block_size=4)):
        pool.lens[2] = 4
        call()
        assert pk.pa_q8_device_status() == pk.PA_Q8_DEV_BAD_BLOCK
    pool.lens[2] = 3                                                     # part full: the page to copy does not exist
    src, dst = u32([5]), u32([5])
    pk.pa_q8_fork_seqs(*pool.all, u32([2]), u32([3]), src, dst, block_size=4)
    assert pk.pa_q8_device_status() == pk.PA_Q8_DEV_BAD_BLOCK
    assert as_u32(src) == as_u32(dst) == [PAD] and pool.lens.tolist() == [0, 0, 3, 0]


@gpu
@pytest.mark.parametrize("cache", ["q8", "f32"])
@pytest.mark.parametrize("Hk,B,D", [(2, 4, 64), (8, 16, 128), (1, 1024, 256), (3, 32, 64), (64, 64, 128)])
def test_copies(cache, Hk, B, D):
    import torch
    import int8_paged_kv_gb300 as pk
    pages = 41
    last = D // 4 + 1 if cache == "q8" else D
    gen = torch.Generator(device="cuda").manual_seed(D)
    bits = [torch.randint(-2 ** 31, 2 ** 31, (pages, Hk, B, last), dtype=torch.int32, device="cuda", generator=gen)
            for _ in range(2)]
    perm = np.random.default_rng(B).permutation(pages)
    src, dst = perm[:20].astype(np.uint32), perm[20:40].astype(np.uint32)
    src[3] = src[7]                                                      # one source twice
    want = [b.clone() for b in bits]
    for w in want:
        w[torch.from_numpy(dst[5:].astype(np.int64)).cuda()] = w[torch.from_numpy(src[5:].astype(np.int64)).cuda()]
    src[0], dst[1], src[2], dst[2] = PAD, PAD, PAD, PAD                  # no pair
    src[3], dst[4] = pages, pages + 7                                    # no such page
    call = pk.pa_q8_copy_blocks if cache == "q8" else pk.pa_f32_copy_blocks
    views = bits if cache == "q8" else [b.view(torch.float32) for b in bits]
    call(*views, u32(src), u32(dst))
    assert pk.pa_q8_device_status() == pk.PA_Q8_DEV_BAD_BLOCK
    for b, w in zip(bits, want):
        assert torch.equal(b, w)
    call(*views, u32([]), u32([]))
    assert pk.pa_q8_device_status() == 0


@gpu
def test_long_lists_of_copies():
    """More pairs than one round of lookups takes, two thirds of them padding; some ids that do not exist."""
    import torch
    import int8_paged_kv_gb300 as pk
    nb, n = 70001, 69000
    g = torch.Generator(device="cuda").manual_seed(5)
    cache = [torch.randint(-2 ** 31, 2 ** 31 - 1, (nb, 1, 4, 17), dtype=torch.int32, device="cuda", generator=g)
             for _ in range(2)]
    perm = torch.randperm(nb, device="cuda", generator=g).to(torch.int32)
    src, dst = perm[:23000], perm[23000:46000]
    at = torch.randperm(n, device="cuda", generator=g)[:23000]
    lists = [torch.full((n,), -1, dtype=torch.int32, device="cuda") for _ in range(2)]
    lists[0][at], lists[1][at] = src, dst
    want = [c.clone() for c in cache]
    for c in want:
        c[dst.long()] = c[src.long()]
    pk.pa_q8_copy_blocks(*cache, *lists)
    assert all(torch.equal(x, y) for x, y in zip(cache, want)) and pk.pa_q8_device_status() == 0
    lists[0][at[7]] = nb
    pk.pa_q8_copy_blocks(*cache, *lists)
    assert all(torch.equal(x, y) for x, y in zip(cache, want))
    assert pk.pa_q8_device_status() == pk.PA_Q8_DEV_BAD_BLOCK


@gpu
@pytest.mark.parametrize("rows", [3, 700])
def test_rows_freed_many_times_in_one_call(rows):
    """Each row is freed once, wherever the call names it; rows out of range between them are flagged."""
    import torch
    import int8_paged_kv_gb300 as pk
    pool = Pool(rows, 9, rows * 8, 16)
    everyone = torch.arange(rows, dtype=torch.int32, device="cuda")
    pk.pa_q8_extend_seqs(*pool.all, everyone, torch.full_like(everyone, 128), block_size=16)
    assert int(pool.count) == 0
    g = torch.Generator(device="cuda").manual_seed(rows)
    seqs = torch.cat([everyone[: rows - 1].repeat(40), u32([rows, 0xFFFFFFFF])])
    pk.pa_q8_free_seqs(*pool.all, seqs[torch.randperm(len(seqs), device="cuda", generator=g)].contiguous(), block_size=16)
    held = pool.table[rows - 1, :8]
    assert int(pool.count) == (rows - 1) * 8 and pool.lens.tolist() == [0] * (rows - 1) + [128]
    stack = pool.stack[: (rows - 1) * 8]
    assert torch.equal(stack, torch.sort(stack)[0]) and not torch.isin(stack, held).any()
    assert int(pool.refs.sum()) == 8 and bool((pool.refs[held.long()] == 1).all())
    assert pk.pa_q8_device_status() == pk.PA_Q8_DEV_BAD_SEQ


@gpu
def test_copies_past_32bit_offsets():
    """Pages whose words lie past 2^32 (18.6 GB per cache), and a list much longer than the grid."""
    import torch
    import int8_paged_kv_gb300 as pk
    NB, Hk, B, W = 1_100_000, 8, 16, 33
    cache = [torch.empty((NB, Hk, B, W), dtype=torch.int32, device="cuda") for _ in range(2)]
    n = 5000
    src = torch.arange(n, dtype=torch.int32, device="cuda")
    dst = NB - 1 - src
    for k, c in enumerate(cache):
        c[:n].random_()
    pk.pa_q8_copy_blocks(*cache, src, dst)
    assert pk.pa_q8_device_status() == 0
    for c in cache:
        assert torch.equal(c[NB - n:].flip(0), c[:n])


@gpu
def test_captured_and_replayed():
    """A turnover of rows and a fork in one graph, replayed over changing requests."""
    import torch
    import int8_paged_kv_gb300 as pk
    rows, width, pages, size = 12, 8, 80, 4
    pool, m = Pool(rows, width, pages, size), Model(rows, width, pages, size)
    both(pool, m, "extend", list(range(6)), [9, 30, 4, 17, 1, 32])
    ends, new, par, chi = u32([0]), u32([1]), u32([1]), u32([7])
    src, dst = u32([5]), u32([5])
    ws = torch.empty(pk.pa_q8_pool_workspace_size(rows, pages, 1), dtype=torch.uint8, device="cuda")

    def step():
        pk.pa_q8_free_seqs(*pool.all, ends, block_size=size)
        pk.pa_q8_extend_seqs(*pool.all, ends, new, block_size=size, workspace=ws)
        pk.pa_q8_fork_seqs(*pool.all, par, chi, src, dst, block_size=size, workspace=ws)

    keep = [t.clone() for t in pool.all]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for t, k in zip(pool.all, keep):
        t.copy_(k)
    pk.pa_q8_device_status()
    rng = np.random.default_rng(3)
    for k in range(20):
        e, n, p, c = (int(rng.integers(rows)), int(rng.integers(0, width * size + 1)), int(rng.integers(rows)),
                      int(rng.integers(rows)))
        for t, v in ((ends, e), (new, n), (par, p), (chi, c)):
            t.fill_(v)
        ws.fill_(0xFF)
        g.replay()
        m.free([e])
        m.extend([e], [n])
        assert (as_u32(src), as_u32(dst)) == m.fork([p], [c])
        pool.check(m, f"replay {k}")


@gpu
def test_serving_run():
    """Pages for prompts, the writer, the prompt attention; a fork with its page copied; each branch goes
    its own way through the fused append and decode; rows end, the pool is closed up, and the decode over
    the moved pages gives the same bits."""
    import torch
    import int8_paged_kv_gb300 as pk
    from tests.test_prefill import check, plain
    H, Hk, D, B, rows, width, pages = 8, 2, 128, 16, 8, 12, 70
    pool = Pool(rows, width, pages, B)
    kc = torch.full((pages, Hk, B, D // 4 + 1), -1, dtype=torch.int32, device="cuda")
    vc = torch.full_like(kc, -1)
    scale = D ** -0.5
    gen = torch.Generator(device="cuda").manual_seed(2)

    def randn(*shape):
        return torch.randn(shape, device="cuda", generator=gen)

    def host(t):
        return t.cpu().numpy().view(np.uint32)

    lens = [37, 100, 64, 5]
    pk.pa_q8_extend_seqs(*pool.all, u32([0, 1, 2, 3]), u32(lens), block_size=B)
    seq = torch.cat([torch.full((n,), s, device="cuda") for s, n in enumerate(lens)])
    pos = torch.cat([torch.arange(n, device="cuda") for n in lens])
    slots = (pool.table[seq, pos // B] * B + pos % B).to(torch.int32)
    T = sum(lens)
    q, key, value = randn(T, H, D), randn(T, Hk * D), randn(T, Hk * D)
    pk.pa_q8_reshape_and_cache(key, value, kc, vc, slots, num_kv_heads=Hk, head_size=D, block_size=B)
    starts = u32(np.concatenate([[0], np.cumsum(lens + [0] * 4)]))
    out = pk.pa_q8_prefill(torch.empty_like(q), q, kc, vc, pool.table, pool.lens, starts, num_kv_heads=Hk,
                           block_size=B, scale=scale)
    want, top = plain(q.cpu().numpy(), host(kc), host(vc), host(pool.table), lens, np.cumsum([0] + lens), scale, D, B)
    check(out.cpu().numpy(), want, top, "float32", "prompts")

    src, dst = u32([0, 0, 0]), u32([0, 0, 0])
    pk.pa_q8_fork_seqs(*pool.all, u32([0, 1, 2]), u32([4, 5, 6]), src, dst, block_size=B)
    pk.pa_q8_copy_blocks(kc, vc, src, dst)
    assert [x == PAD for x in as_u32(dst)] == [False, False, True]       # 64 tokens fill their pages
    # one token more for every row; the branches get different ones
    now = pool.lens.cpu().numpy()
    live = [s for s in range(rows) if now[s]]
    pk.pa_q8_extend_seqs(*pool.all, u32(live), u32(now[live] + 1), block_size=B)
    kv, vv, q1 = randn(rows, 1, Hk, D), randn(rows, 1, Hk, D), randn(rows, 1, H, D)
    got = pk.pa_q8_decode_append(torch.empty_like(q1), q1, kv, vv, kc, vc, pool.table, pool.lens, num_kv_heads=Hk,
                                 block_size=B, scale=scale)
    lens1 = host(pool.lens)
    want, top = plain(q1[live, 0].cpu().numpy(), host(kc), host(vc), host(pool.table)[live], lens1[live],
                      np.arange(len(live) + 1), scale, D, B)
    check(got[live, 0].cpu().numpy(), want, top, "float32", "branches")
    # the branches' pages: whole ones shared with the parent, open ones their own
    table = host(pool.table)
    assert table[0, :2].tolist() == table[4, :2].tolist() and table[0, 2] != table[4, 2]
    # a chunk of prompt behind the shared prefix of a branch, in bf16
    pk.pa_q8_extend_seqs(*pool.all, u32([6]), u32([65 + 40]), block_size=B)
    pos = 65 + torch.arange(40, device="cuda")
    pk.pa_q8_reshape_and_cache(randn(40, Hk * D), randn(40, Hk * D), kc, vc,
                               (pool.table[6, pos // B] * B + pos % B).to(torch.int32), num_kv_heads=Hk, head_size=D,
                               block_size=B)
    qc = randn(40, H, D).bfloat16()
    out = pk.pa_q8_prefill(torch.empty_like(qc), qc, kc, vc, pool.table, pool.lens,
                           u32([0, 0, 0, 0, 0, 0, 0, 40, 40]), num_kv_heads=Hk, block_size=B, scale=scale)
    want, top = plain(qc.float().cpu().numpy(), host(kc), host(vc), host(pool.table)[6:7], [105], [0, 40], scale, D, B)
    check(out.float().cpu().numpy(), want, top, "bfloat16", "chunk")

    pk.pa_q8_free_seqs(*pool.all, u32([1, 3, 4]), block_size=B)
    q2 = randn(rows, H, D)
    before = pk.pa_q8_decode(torch.empty_like(q2), q2, kc, vc, pool.table, pool.lens, num_kv_heads=Hk, block_size=B,
                             scale=scale)
    n = pages // 2
    src, dst = torch.empty(n, dtype=torch.int32, device="cuda"), torch.empty(n, dtype=torch.int32, device="cuda")
    pk.pa_q8_compact_blocks(*pool.all, src, dst, block_size=B)
    pk.pa_q8_copy_blocks(kc, vc, src, dst)
    held = pages - int(pool.count)
    assert int(pool.table[[0, 2, 5, 6]].max()) >= 0 and int((dst != -1).sum()) > 0
    after = pk.pa_q8_decode(torch.empty_like(q2), q2, kc[:held].contiguous(), vc[:held].contiguous(), pool.table,
                            pool.lens, num_kv_heads=Hk, block_size=B, scale=scale)
    assert torch.equal(before, after) and pk.pa_q8_device_status() == 0


@gpu
def test_refusals_of_the_binding():
    import torch
    import int8_paged_kv_gb300 as pk
    pool = Pool(4, 4, 16, 4)
    one = u32([0])
    with pytest.raises(ValueError):
        pk.pa_q8_extend_seqs(*pool.all, one, u32([1, 2]), block_size=4)
    with pytest.raises(TypeError):
        pk.pa_q8_free_seqs(*pool.all, one.float(), block_size=4)
    with pytest.raises(TypeError):
        pk.pa_q8_free_seqs(*pool.all, one.cpu(), block_size=4)
    with pytest.raises(pk.PaQ8Error, match="unsupported"):
        pk.pa_q8_free_seqs(*pool.all, one, block_size=12)
    with pytest.raises(pk.PaQ8Error, match="invalid"):
        pk.pa_q8_compact_blocks(*pool.all, u32([0] * 7), u32([0] * 7), block_size=4)
    with pytest.raises(pk.PaQ8Error, match="workspace"):
        pk.pa_q8_fork_seqs(*pool.all, one, one, one.clone(), one.clone(), block_size=4,
                           workspace=torch.empty(4, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        pk.pa_q8_copy_blocks(torch.zeros((2, 1, 4, 17), dtype=torch.int32, device="cuda"),
                             torch.zeros((3, 1, 4, 17), dtype=torch.int32, device="cuda"), one, one)
    for call in (lambda: pk.pa_q8_extend_seqs(*pool.all, u32([]), u32([]), block_size=4),
                 lambda: pk.pa_q8_free_seqs(*pool.all, u32([]), block_size=4)):
        call()
    assert pool.count.item() == 16


def test_argument_errors(lib):
    """Status codes of the C entry points, none of which touches a device."""
    import ctypes
    from int8_paged_kv_gb300 import _binding
    L = _binding.lib()
    ok, odd = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10002)

    def copy(kc=ok, src=ok, n=4, Hk=2, D=128, B=16, nb=8):
        return L.pa_q8_copy_blocks(kc, ok, src, ok, n, Hk, D, B, nb, None)

    for kw, code in ((dict(n=-1), -1), (dict(Hk=0), -1), (dict(D=96), -2), (dict(B=6), -1), (dict(B=24), -2), (dict(nb=0), -1),
                     (dict(kc=None), -1), (dict(src=None), -1), (dict(kc=ctypes.c_void_p(0x10004)), -3), (dict(src=odd), -3),
                     (dict(nb=1 << 31), -2)):
        assert copy(**kw) == code, kw
    assert copy(n=0, kc=None) == 0

    def extend(bt=ok, seqs=ok, n=3, S=4, Nb=4, B=16, nb=8, ws=ok, bytes_=1 << 20):
        return L.pa_q8_extend_seqs(bt, ok, ok, ok, ok, seqs, ok, n, S, Nb, B, nb, ws, bytes_, None)

    for kw, code in ((dict(n=-1), -1), (dict(S=0), -1), (dict(Nb=0), -1), (dict(B=0), -1), (dict(B=12), -2), (dict(nb=0), -1),
                     (dict(bt=None), -1), (dict(seqs=None), -1), (dict(bt=odd), -3), (dict(seqs=odd), -3),
                     (dict(ws=None), -5), (dict(bytes_=8), -5), (dict(ws=ctypes.c_void_p(0x10004)), -3),
                     (dict(nb=1 << 31), -2), (dict(Nb=1 << 28, B=1024), -2)):
        assert extend(**kw) == code, kw
    assert extend(n=0, seqs=None) == 0
    assert L.pa_q8_fork_seqs(ok, ok, ok, ok, ok, ok, ok, None, ok, 1, 4, 4, 16, 8, ok, 1 << 20, None) == -1
    assert L.pa_q8_free_seqs(ok, ok, ok, ok, ok, None, 1, 4, 4, 16, 8, None) == -1
    assert L.pa_q8_compact_blocks(ok, ok, ok, ok, ok, ok, ok, 3, 4, 4, 16, 8, ok, 1 << 20, None) == -1
    assert L.pa_q8_compact_blocks(ok, ok, ok, ok, ok, None, ok, 4, 4, 4, 16, 8, ok, 1 << 20, None) == -1
    assert L.pa_q8_pool_init(None, ok, ok, 4, None) == -1
    assert L.pa_q8_pool_workspace_size(4, 8, 2) > 0 and L.pa_q8_pool_workspace_size(0, 8, 2) == 0
