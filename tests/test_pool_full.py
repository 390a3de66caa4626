"""extend in a pool that is full or nearly so: a request that needs no page is
served whatever happened to the ones before it.  The same plain model as in
test_pages.py, with that rule."""
import numpy as np
import pytest

from tests.test_pages import Model, Pool, _clean, both, lib  # noqa: F401  (fixtures)

gpu = pytest.mark.gpu


class FullModel(Model):
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
            if need and want > room:
                self.flags |= 16
                continue
            for k in range(need):
                b = self.stack.pop()
                self.table[s][self.held(s) + k] = b
                self.refs[b] = 1
            self.lens[s] = n


@gpu
def test_one_token_for_every_row_of_a_full_pool():
    """Rows whose last page has room grow; the others are flagged."""
    pool, m = Pool(12, 8, 23, 4), FullModel(12, 8, 23, 4)
    lens = [8, 7, 4, 6, 12, 9, 1, 8, 5, 8, 7, 4]
    both(pool, m, "extend", list(range(12)), lens)
    assert len(m.stack) == 0
    both(pool, m, "extend", list(range(12)), [n + 1 for n in lens])
    assert m.lens == [n + (n % 4 > 0) for n in lens]
    both(pool, m, "free", [4])                                           # three pages: for the first three that need one
    both(pool, m, "extend", list(range(12)), [n + 1 for n in m.lens[:4]] + [0] + [n + 1 for n in m.lens[5:]])


@gpu
@pytest.mark.parametrize("rows,width,pages,size", [(40, 30, 300, 16), (3000, 6, 4000, 8), (1500, 9, 1, 4)])
def test_small_steps_until_the_pool_is_full_and_on(rows, width, pages, size):
    rng = np.random.default_rng(pages)
    pool, m = Pool(rows, width, pages, size), FullModel(rows, width, pages, size)
    for step in range(12):
        n = int(rng.integers(1, rows + 1))
        seqs = rng.permutation(rows)[:n]
        both(pool, m, "extend", seqs.tolist(), [min(width * size, m.lens[s] + int(rng.integers(0, 2 * size))) for s in seqs])
        if step % 4 == 3:
            both(pool, m, "free", rng.integers(0, rows, max(1, n // 8)).tolist())
