"""Timed cases of the prompt attention and of the page operators.

Both work on the int8 paged cache: u32 words (as int32) of shape
[num_blocks, num_kv_heads, block_size, head_size / 4 + 1], head_size codes and
the f32 bits of the token's scale.  `run` computes a case in its plain form
(elementary torch operations in f32 and integers), or, with `own` set, by the
calls that a user makes of the package.
"""
import math
import random

import torch

own = False

PAD = -1                    # 0xFFFFFFFF as int32: no page
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
# head layouts: (query heads, kv heads, head size, page size)
LAYOUTS = {"tiny": (4, 2, 64, 16), "llama8b": (32, 8, 128, 16), "long": (32, 8, 128, 32),
           "large": (64, 8, 128, 16), "edge": (16, 1, 256, 32)}


def listed():
    return [
        # two short prompts of a small f32 model: latency
        {"name": "prefill tiny f32", "op": "prefill", "layout": "tiny", "type": "f32", "seqs": 2, "rows": 100,
         "prefix": 0, "lens": 3},
        # a batch of whole prompts of an 8B-like model in bf16
        {"name": "prefill llama8b bf16", "op": "prefill", "layout": "llama8b", "type": "bf16", "seqs": 8,
         "rows": 4096, "prefix": 0, "lens": 1},
        # the next chunk of two very long prompts, behind what the cache holds of them
        {"name": "prefill long chunk f16", "op": "prefill", "layout": "long", "type": "f16", "seqs": 2, "rows": 512,
         "prefix": 130000, "lens": 2},
        # many ragged prompts, one kv head of size 256, f32
        {"name": "prefill edge f32", "op": "prefill", "layout": "edge", "type": "f32", "seqs": 32, "rows": 4095,
         "prefix": 0, "lens": 5},
        # a few open pages copied before they are written (beam search, one step)
        {"name": "copy 5 pages", "op": "copy", "layout": "llama8b", "pages": 64, "pairs": 5},
        # a large share of a pool copied page by page
        {"name": "copy 8192 pages", "op": "copy", "layout": "large", "pages": 24576, "pairs": 8192},
        # one conversation branches in four
        {"name": "fork 4", "op": "fork", "layout": "llama8b", "seqs": 16, "forks": 4, "rows": 4096, "lens": 4},
        # a sampling batch: 128 continuations of 64 prompts
        {"name": "fork 128", "op": "fork", "layout": "large", "seqs": 256, "forks": 128, "rows": 8192, "lens": 6},
        # one sequence ends and the next one takes its row
        {"name": "turnover 1", "op": "turnover", "layout": "llama8b", "seqs": 64, "ends": 1, "rows": 4096, "lens": 7},
        # a batch of sequences ends, sharing pages with others; as many new ones come in
        {"name": "turnover 128", "op": "turnover", "layout": "large", "seqs": 256, "ends": 128, "rows": 8192, "lens": 8},
        # a small pool closed up
        {"name": "compact tiny", "op": "compact", "layout": "tiny", "seqs": 8, "rows": 100, "lens": 9},
        # the pool of a large batch closed up after a third of it ended
        {"name": "compact large", "op": "compact", "layout": "large", "seqs": 256, "rows": 8192, "lens": 10},
    ]


def _spread(rng, lo, hi):
    """A whole number from lo to hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "prefill", "copy", "fork", "turnover", "compact"])
    lens = rng.randrange(1 << 20)
    if op == "prefill":
        layout = rng.choice(sorted(LAYOUTS))
        heads = LAYOUTS[layout][0]
        rows = _spread(rng, 1, 4096)
        prefix = rng.choice([0, 0, _spread(rng, 1, 130000)])
        # rows x tokens x heads over all sequences: at most half of the largest listed case's
        room = (8 * 4096 * 4096 * 32) // 2 // (rows * (rows + prefix) * heads)
        while room < 1:
            rows = (rows + 1) // 2
            room = (8 * 4096 * 4096 * 32) // 2 // (rows * (rows + prefix) * heads)
        return {"op": op, "layout": layout, "type": rng.choice(sorted(TYPES)),
                "seqs": min(_spread(rng, 1, 64), room, max(1, 260000 // (rows + prefix))), "rows": rows,
                "prefix": prefix, "lens": lens}
    layout = rng.choice(["tiny", "llama8b", "large"])
    if op == "copy":
        pairs = _spread(rng, 1, 8000)
        return {"op": op, "layout": layout, "pages": 2 * pairs + rng.randrange(64), "pairs": pairs}
    seqs = _spread(rng, 4, 240)
    case = {"op": op, "layout": layout, "seqs": seqs, "rows": _spread(rng, 20, 8000), "lens": lens}
    if op == "fork":
        case["forks"] = rng.randint(1, max(1, seqs // 2))
    if op == "turnover":
        case["ends"] = rng.randint(1, max(1, seqs // 2))
    return case


def _lengths(case):
    """Per sequence: its rows of this call and its tokens in all."""
    r = random.Random(case["lens"])
    n, most, prefix = case["seqs"], case["rows"], case.get("prefix", 0)
    if case["op"] == "prefill":
        rows = [most] + [r.randint(max(1, most // 8), most) for _ in range(n - 1)]
        if case["layout"] == "edge" and prefix == 0:    # lengths around a page's border among them
            rows = [min(most, x) for x in ([most, 1, 31, 33] + [r.randint(1, most) for _ in range(n)])[:n]]
        return rows, [x + (r.randint(prefix // 2, prefix) if prefix else 0) for x in rows]
    rows = [min(most, max(1, int(round(r.lognormvariate(math.log(max(2, most / 4)), 1.0))))) for _ in range(n)]
    return rows, rows


def _pages_of(lens, size):
    return [-(-x // size) for x in lens]


def _cache(gen, pages, layout):
    """A K or V cache of quantised normal vectors."""
    _, kv, dim, size = LAYOUTS[layout]
    x = torch.randn((pages, kv, size, dim), device="cuda", generator=gen)
    amax = x.abs().amax(-1, keepdim=True)
    words = torch.empty((pages, kv, size, dim // 4 + 1), dtype=torch.int32, device="cuda")
    words[..., :-1] = (x * (127.0 / amax)).round_().to(torch.int8).view(torch.int32)
    words[..., -1] = (amax / 127.0).view(torch.int32)[..., 0]
    return words


def _words(gen, pages, layout):
    """A cache whose words only move: any bits."""
    _, kv, dim, size = LAYOUTS[layout]
    return torch.randint(-2**31, 2**31, (pages, kv, size, dim // 4 + 1), dtype=torch.int32, device="cuda", generator=gen)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _table(gen, lens, size, pool, width):
    """Pages of every sequence drawn from the pool, and the pages left over."""
    perm = torch.randperm(pool, device="cuda", generator=gen).to(torch.int32)
    need = _pages_of(lens, size)
    col = torch.arange(width, device="cuda")[None, :]
    start = torch.cumsum(_ints([0] + need[:-1]), 0)[:, None]
    used = col < _ints(need)[:, None]
    table = torch.where(used, perm[torch.where(used, start + col, 0)], PAD).to(torch.int32).contiguous()
    return table, perm[sum(need):].contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, layout = case["op"], case["layout"]
    heads, kv, dim, size = LAYOUTS[layout]
    if op == "copy":
        pages = case["pages"]
        perm = torch.randperm(pages, device="cuda", generator=gen).to(torch.int32)
        return {"case": case, "key": _words(gen, pages, layout), "value": _words(gen, pages, layout),
                "src": perm[:case["pairs"]].contiguous(), "dst": perm[case["pairs"]:2 * case["pairs"]].contiguous()}
    rows, lens = _lengths(case)
    need = _pages_of(lens, size)
    if op == "prefill":
        pool = sum(need) + 7
        table, _ = _table(gen, lens, size, pool, max(need))
        total = sum(rows)
        q = torch.randn((total, heads, dim), device="cuda", generator=gen).to(TYPES[case["type"]])
        starts = [0]
        for x in rows:
            starts.append(starts[-1] + x)
        return {"case": case, "q": q, "key": _cache(gen, pool, layout), "value": _cache(gen, pool, layout),
                "tables": table, "lens": _ints(lens), "starts": _ints(starts), "most_rows": max(rows),
                "scale": 1.0 / math.sqrt(dim)}
    # a pool and the tables of its sequences; every eighth sequence shares the whole pages of the one before it
    width = max(-(-case["rows"] // size), 1) + 1
    spare = {"fork": case.get("forks", 0), "turnover": 0, "compact": 0}[op]
    pool = sum(need) + max(8, sum(need) // 8) + spare
    table, free = _table(gen, lens + [0] * spare, size, pool, width)
    lens_t = _ints(lens + [0] * spare)
    seqs = len(lens)
    who = torch.arange(seqs + spare, device="cuda")
    shares = (who % 8 == 7) & (who < seqs) & (lens_t < torch.roll(lens_t, 1))
    whole = torch.where(shares, lens_t // size, 0)[:, None]
    col = torch.arange(width, device="cuda")[None, :]
    table = torch.where(col < whole, torch.roll(table, 1, 0), table).contiguous()
    in_use = col < ((lens_t + size - 1) // size)[:, None]
    refs = torch.zeros(pool + 1, dtype=torch.int32, device="cuda")
    refs.index_add_(0, torch.where(in_use, table, pool).reshape(-1).long(), torch.ones_like(table).reshape(-1))
    refs = refs[:pool]
    # free pages, in the order in which they were freed
    free = torch.randperm(pool, device="cuda", generator=gen).to(torch.int32)
    order = torch.argsort((refs[free.long()] > 0).to(torch.int32), stable=True)
    free = torch.where(refs[free[order].long()] > 0, PAD, free[order]).to(torch.int32)
    state = {"case": case, "sizes": (seqs + spare, width, pool)}
    if op == "compact":     # a third of the sequences has ended
        gone = torch.rand(seqs, device="cuda", generator=gen) < 1 / 3
        gone[0] = True
        lens_t = torch.where(gone, 0, lens_t).to(torch.int32)
        in_use = col < ((lens_t + size - 1) // size)[:, None]
        refs = torch.zeros(pool + 1, dtype=torch.int32, device="cuda")
        refs.index_add_(0, torch.where(in_use, table, pool).reshape(-1).long(), torch.ones_like(table).reshape(-1))
        refs = refs[:pool]
        free = torch.where(torch.arange(pool, device="cuda") < (refs == 0).sum(),
                           torch.argsort((refs > 0).to(torch.int32), stable=True), PAD).to(torch.int32)
        live = int((refs > 0).sum())
        state["moves"] = int((refs[live:] > 0).sum())
    # tables, lengths, counts and the free list in one buffer, put back before every pass
    count = (refs == 0).sum().to(torch.int32).reshape(1)
    state["saved"] = torch.cat([table.reshape(-1), lens_t, refs, free, count]).contiguous()
    state["pool"] = torch.empty_like(state["saved"])
    pick = random.Random(seed)
    if op == "fork":
        parents = [pick.randrange(min(seqs, 64)) for _ in range(spare)]
        state["parents"], state["children"] = _ints(parents), _ints(list(range(seqs, seqs + spare)))
    if op == "turnover":
        ends = pick.sample(range(seqs), case["ends"])
        state["ends"] = _ints(ends)
        state["new_lens"] = _ints([pick.randint(1, max(1, min(lens[i], 4 * size))) for i in ends])
    if op in ("fork", "compact"):
        state["key"], state["value"] = _words(gen, pool, layout), _words(gen, pool, layout)
    return state


def _views(state):
    """The pool's tensors, put back to what they were."""
    rows, width, pool = state["sizes"]
    flat = state["pool"].copy_(state["saved"])
    table = flat[:rows * width].view(rows, width)
    lens, refs, free, count = torch.split(flat[rows * width:], [rows, pool, pool, 1])
    return table, lens, refs, free, count


def _plain_prefill(state):
    case, q = state["case"], state["q"]
    heads, kv, dim, size = LAYOUTS[case["layout"]]
    table, lens, starts = state["tables"], state["lens"].long(), state["starts"].long()
    seqs, most = table.shape[0], state["most_rows"]

    def gather(cache):      # [seqs, kv, tokens, dim] in f32
        got = cache[table.clamp(min=0).long()].permute(0, 2, 1, 3, 4).reshape(seqs, kv, -1, dim // 4 + 1)
        codes = got[..., :-1].contiguous().view(torch.int8).float()
        return codes * got[..., -1:].contiguous().view(torch.float32)

    key, value = gather(state["key"]), gather(state["value"])
    count = (starts[1:] - starts[:-1])[:, None]
    at = torch.arange(most, device=q.device)[None, :]
    live = at < count
    row = torch.where(live, starts[:-1, None] + at, 0)
    group = heads // kv
    qf = q[row].float().view(seqs, most, kv, group, dim).permute(0, 2, 3, 1, 4).reshape(seqs, kv, group * most, dim)
    score = torch.matmul(qf, key.transpose(-1, -2)).mul_(state["scale"]).view(seqs, kv, group, most, -1)
    sees = lens[:, None] - (count - 1 - at)
    hidden = torch.arange(score.shape[-1], device=q.device)[None, None, :] >= sees[:, :, None]
    score.masked_fill_(hidden[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    weight = score.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = weight.sum(-1, keepdim=True)
    out = torch.matmul(weight.view(seqs, kv, group * most, -1), value).view(seqs, kv, group, most, dim)
    out = out / torch.where(total == 0, 1.0, total)
    out = out.permute(0, 3, 1, 2, 4).reshape(seqs, most, heads, dim)
    at_row = torch.where(live, row, q.shape[0]).reshape(-1)     # rows of no sequence go behind the last one
    packed = torch.empty((q.shape[0] + 1, heads, dim), dtype=q.dtype, device=q.device)
    packed[at_row] = out.reshape(-1, heads, dim).to(q.dtype)
    return packed[:-1]


def _plain_fork(state):
    table, lens, refs, free, count = _views(state)
    size = LAYOUTS[state["case"]["layout"]][3]
    parents, children = state["parents"].long(), state["children"].long()
    tokens = lens[parents]
    whole = (tokens // size)[:, None]
    open_page = (tokens % size > 0).to(torch.int32)
    rank = torch.cumsum(open_page, 0) - 1
    fresh = torch.where(open_page > 0, free[(count - 1 - rank).clamp(min=0).long()], PAD)
    rows = table[parents]
    col = torch.arange(table.shape[1], device=table.device)[None, :]
    src = torch.where(open_page > 0, rows.gather(1, whole.long())[:, 0], PAD)
    shared = col < whole
    add = torch.zeros(refs.shape[0] + 1, dtype=torch.int32, device=refs.device)
    add.index_add_(0, torch.where(shared, rows, refs.shape[0]).reshape(-1).long(), torch.ones_like(rows).reshape(-1))
    add.index_add_(0, torch.where(open_page > 0, fresh, refs.shape[0]).long(), open_page)
    refs += add[:-1]
    opened = (col == whole) & (open_page > 0)[:, None]
    table[children] = torch.where(shared, rows, torch.where(opened, fresh[:, None], table[children]))
    lens[children] = tokens
    # pages taken from the stack are left in it above its top
    count -= open_page.sum()
    moved, to = torch.where(open_page > 0, src, fresh), fresh
    first = fresh.amax()                    # forks without an open page repeat one that has: the same bytes again
    at = torch.argmax(fresh)
    moved, to = torch.where(open_page > 0, moved, src[at]).long(), torch.where(open_page > 0, to, first).long()
    state["key"][to], state["value"][to] = state["key"][moved], state["value"][moved]
    return table, lens, refs, count, src, fresh, state["key"], state["value"]


def _plain_turnover(state):
    table, lens, refs, free, count = _views(state)
    size = LAYOUTS[state["case"]["layout"]][3]
    pool = refs.shape[0]
    ends = state["ends"].long()
    rows = table[ends]
    col = torch.arange(table.shape[1], device=table.device)[None, :]
    held = col < ((lens[ends] + size - 1) // size)[:, None]
    was = refs > 0
    less = torch.zeros(pool + 1, dtype=torch.int32, device=refs.device)
    less.index_add_(0, torch.where(held, rows, pool).reshape(-1).long(), torch.ones_like(rows).reshape(-1))
    refs -= less[:-1]
    freed = was & (refs == 0)
    at = torch.where(freed, count + torch.cumsum(freed, 0) - 1, pool)
    more = torch.cat([free, free[:1]])
    more[at] = torch.arange(pool, dtype=torch.int32, device=free.device)
    free.copy_(more[:-1])
    count += freed.sum()
    need = (state["new_lens"] + size - 1) // size
    first = (torch.cumsum(need, 0) - need)[:, None]
    takes = col < need[:, None]
    page = free[(count - 1 - first - col).clamp(min=0).long()]
    table[ends] = torch.where(takes, page, table[ends])
    one = torch.zeros(pool + 1, dtype=torch.int32, device=refs.device)
    one.index_add_(0, torch.where(takes, page, pool).reshape(-1).long(), torch.ones_like(page).reshape(-1))
    refs += one[:-1]
    lens[ends] = state["new_lens"]
    count -= need.sum()
    # pages taken stay in the stack above its top, and in the table behind a row's length
    return table, lens, refs, free, count


def _plain_compact(state):
    table, lens, refs, free, count = _views(state)
    size = LAYOUTS[state["case"]["layout"]][3]
    pool = refs.shape[0]
    page = torch.arange(pool, dtype=torch.int32, device=refs.device)
    used = refs > 0
    live = used.sum()
    hole, mover = ~used & (page < live), used & (page >= live)
    src = torch.full((pool // 2 + 1,), PAD, dtype=torch.int32, device=refs.device)
    dst = src.clone()
    dst[torch.where(hole, torch.cumsum(hole, 0) - 1, pool // 2)] = page
    src[torch.where(mover, torch.cumsum(mover, 0) - 1, pool // 2)] = page
    src, dst = src[:-1], dst[:-1]
    moved, to = src[:state["moves"]].long(), dst[:state["moves"]].long()
    where = page.clone()
    where[moved] = to.to(torch.int32)
    refs[to], refs[moved] = refs[moved], 0
    col = torch.arange(table.shape[1], device=table.device)[None, :]
    held = col < ((lens + size - 1) // size)[:, None]
    table.copy_(torch.where(held, where[torch.where(held, table, 0).long()], table))
    free.copy_(torch.where(page < pool - live, pool - 1 - page, PAD))
    state["key"][to], state["value"][to] = state["key"][moved], state["value"][moved]
    return table, lens, refs, free, count, state["key"], state["value"]


def run(state):
    case = state["case"]
    op = case["op"]
    heads, kv, dim, size = LAYOUTS[case["layout"]]
    if not own:
        if op == "copy":
            src, dst = state["src"].long(), state["dst"].long()
            state["key"][dst], state["value"][dst] = state["key"][src], state["value"][src]
            return state["key"], state["value"]
        return {"prefill": _plain_prefill, "fork": _plain_fork, "turnover": _plain_turnover,
                "compact": _plain_compact}[op](state)
    import int8_paged_kv_gb300 as pk
    if op == "prefill":
        out = torch.empty_like(state["q"])
        return pk.pa_q8_prefill(out, state["q"], state["key"], state["value"], state["tables"], state["lens"],
                                state["starts"], num_kv_heads=kv, block_size=size, scale=state["scale"])
    if op == "copy":
        pk.pa_q8_copy_blocks(state["key"], state["value"], state["src"], state["dst"])
        return state["key"], state["value"]
    table, lens, refs, free, count = _views(state)
    if op == "fork":
        src, dst = torch.empty_like(state["parents"]), torch.empty_like(state["parents"])
        pk.pa_q8_fork_seqs(table, lens, refs, free, count, state["parents"], state["children"], src, dst,
                           block_size=size)
        pk.pa_q8_copy_blocks(state["key"], state["value"], src, dst)
        return table, lens, refs, count, src, dst, state["key"], state["value"]
    if op == "turnover":
        pk.pa_q8_free_seqs(table, lens, refs, free, count, state["ends"], block_size=size)
        pk.pa_q8_extend_seqs(table, lens, refs, free, count, state["ends"], state["new_lens"], block_size=size)
        return table, lens, refs, free, count
    src = torch.empty(refs.shape[0] // 2, dtype=torch.int32, device=refs.device)
    dst = torch.empty_like(src)
    pk.pa_q8_compact_blocks(table, lens, refs, free, count, src, dst, block_size=size)
    pk.pa_q8_copy_blocks(state["key"], state["value"], src, dst)
    return table, lens, refs, free, count, state["key"], state["value"]


def work(case):
    op = case["op"]
    heads, kv, dim, size = LAYOUTS[case["layout"]]
    page = 2 * kv * size * (dim + 4)                # a K and a V page, in bytes
    if op == "copy":
        return {"bytes": 2 * page * case["pairs"] + 8 * case["pairs"], "flops": 0}
    rows, lens = _lengths(case)
    need = _pages_of(lens, size)
    if op == "prefill":
        item = torch.empty((), dtype=TYPES[case["type"]]).element_size()
        pairs = sum(n * c - n * (n - 1) // 2 for n, c in zip(rows, lens))
        return {"bytes": 2 * sum(rows) * heads * dim * item + sum(lens) * 2 * kv * (dim + 4) + 4 * sum(need),
                "flops": 4 * pairs * heads * dim}
    mean = sum(need) / len(need)
    if op == "fork":        # the parents' rows read, the children's written, counts read and written, open pages copied
        return {"bytes": case["forks"] * (16 * mean + 2 * page), "flops": 0}
    if op == "turnover":    # the rows read, counts read and written
        return {"bytes": case["ends"] * 12 * mean + 4 * sum(need), "flops": 0}
    # counts and tables read and written; about a third of two thirds of the pages moved
    return {"bytes": 16 * sum(need) + 2 * page * (2 * sum(need) // 9), "flops": 0}


def exact(case, seed):
    """The prompt attention sequence by sequence and head by head in 64 bits; the other operators give whole numbers."""
    if case["op"] != "prefill":
        return None
    state = prepare(case, seed)
    heads, kv, dim, size = LAYOUTS[case["layout"]]
    rows, lens = _lengths(case)
    q, table = state["q"], state["tables"]
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    first = 0
    for s, (n, c) in enumerate(zip(rows, lens)):
        t = torch.arange(c, device=q.device)
        page, off = table[s, t // size].long(), t % size
        for g in range(kv):
            k, v = state["key"][page, g, off], state["value"][page, g, off]
            k, v = (x[:, :-1].contiguous().view(torch.int8).double() *
                    x[:, -1:].contiguous().view(torch.float32).double() for x in (k, v))
            per = heads // kv
            step = max(1, 200_000_000 // (c * per))
            for lo in range(0, n, step):
                hi = min(n, lo + step)
                rows_q = q[first + lo:first + hi, g * per:(g + 1) * per].double()
                z = torch.einsum("ihd,td->hit", rows_q, k) * state["scale"]
                seen = torch.arange(c, device=q.device)[None, :] <= c - n + torch.arange(lo, hi, device=q.device)[:, None]
                z = torch.where(seen, z, -math.inf)
                p = torch.softmax(z, -1)
                out[first + lo:first + hi, g * per:(g + 1) * per] = torch.einsum("hit,td->ihd", p, v)
        first += n
    return out
