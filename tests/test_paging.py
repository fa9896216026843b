"""PagePool's bookkeeping, on the CPU: random runs of every call against plain
lists of tokens, with the rows and page copies that the pool asks for carried
out on a list in the device's place."""
import random

import pytest
import torch

from store_h3kv_build_gb300.paging import PagePool, PoolFull


class Model:
    def __init__(self, pages, ps):
        self.pool, self.ps = PagePool(pages, ps), ps
        self.cells = [None] * (pages * ps)
        self.tokens = {}

    def copy(self, pairs):
        assert len({b for _, b in pairs}) == len(pairs) and not {a for a, _ in pairs} & {b for _, b in pairs}
        for a, b in pairs:
            self.cells[b * self.ps:(b + 1) * self.ps] = self.cells[a * self.ps:(a + 1) * self.ps]

    def check(self):
        p = self.pool
        refs = [0] * p.pages
        for s, want in self.tokens.items():
            assert p.length(s) == len(want)
            assert [self.cells[r] for r in p.rows(s).tolist()] == want
            assert len(p.pages_of(s)) == -(-len(want) // self.ps)
            for page in p.pages_of(s):
                refs[page] += 1
        assert refs == p._refs
        assert sorted(p._free) == [i for i, r in enumerate(refs) if r == 0] and p.free_pages == refs.count(0)


@pytest.mark.parametrize("seed", range(12))
def test_random_runs_against_lists(seed):
    rng = random.Random(seed)
    ps = rng.choice([16, 32, 64, 128])
    m = Model(rng.choice([6, 20, 60]), ps)
    p, full, stamp = m.pool, 0, 0
    for _ in range(300):
        call = rng.choice(["new", "extend", "extend", "extend", "fork", "free", "truncate", "keep", "compact"])
        seqs = p.sequences()
        s = rng.choice(seqs) if seqs else None
        if call == "new" or s is None:
            m.tokens[p.new()] = []
        elif call == "extend":
            n = rng.choice([0, 1, rng.randrange(1, 3 * ps)])
            before = (list(p._free), {k: list(v) for k, v in p._table.items()}, list(p._refs))
            try:
                rows, pairs = p.extend(s, n)
            except PoolFull:
                full += 1
                assert before == (list(p._free), {k: list(v) for k, v in p._table.items()}, list(p._refs))
                continue
            m.copy(pairs)
            assert rows.dtype == torch.int32 and len(set(rows.tolist())) == n
            for r in rows.tolist():
                m.cells[r] = stamp
                m.tokens[s].append(stamp)
                stamp += 1
        elif call == "fork":
            m.tokens[p.fork(s)] = list(m.tokens[s])
        elif call == "free":
            p.free(s)
            del m.tokens[s]
        elif call == "truncate":
            n = rng.randrange(0, len(m.tokens[s]) + 1)
            p.truncate(s, n)
            del m.tokens[s][n:]
        elif call == "keep":  # what paged_keep does with the last rows
            n = len(m.tokens[s])
            base = rng.randrange(max(0, n - 64), n + 1)
            try:
                m.copy(p.own(s, base))
            except PoolFull:
                full += 1
                continue
            rows = p.rows(s, base).tolist()
            kept = [j for j in range(n - base) if rng.random() < 0.4]
            values = [m.cells[rows[j]] for j in kept]
            for r, v in zip(rows, values):
                m.cells[r] = v
            p.truncate(s, base + len(kept))
            m.tokens[s] = m.tokens[s][:base] + values
        else:
            m.copy(p.compact())
            assert sorted(p._free) == list(range(p.pages - p.free_pages, p.pages))
        m.check()
    assert full or m.pool.pages == 60


def test_pages_are_handed_out_lowest_first():
    p = PagePool(8, 16)
    a, b = p.new(), p.new()
    p.extend(a, 40)
    p.extend(b, 16)
    assert p.pages_of(a) == (0, 1, 2) and p.pages_of(b) == (3,)
    p.truncate(a, 17)
    rows, pairs = p.extend(b, 1)
    assert p.pages_of(b) == (3, 2) and rows.tolist() == [32] and pairs == []


def test_a_shared_full_page_is_not_copied_and_a_part_full_one_is():
    p = PagePool(8, 16)
    a = p.new()
    p.extend(a, 32)
    f = p.fork(a)
    assert p.extend(f, 3)[1] == []          # the shared pages are full
    g = p.fork(f)
    assert p.extend(g, 1)[1] == [(2, 3)]    # the last one is not
    assert p.pages_of(f) == (0, 1, 2) and p.pages_of(g) == (0, 1, 3)
    assert p.extend(f, 1)[1] == []          # and is f's alone now


def test_tables_and_refusals():
    p = PagePool(4, 16)
    a, b = p.new(), p.new()
    p.extend(a, 33)
    assert p.table([a, b]).tolist() == [[0, 1, 2], [-1, -1, -1]] and p.lengths([b, a]).tolist() == [0, 33]
    assert p.table([b]).shape == (1, 1) and p.table([], 5).shape == (0, 5)
    assert p.rows(b).tolist() == []
    with pytest.raises(ValueError, match="max_pages"):
        p.table([a], 2)
    with pytest.raises(PoolFull):
        p.extend(b, 17)
    with pytest.raises(ValueError):
        p.extend(a, -1)
    with pytest.raises(ValueError):
        p.truncate(a, 34)
    with pytest.raises(ValueError):
        p.own(a, 34)
    with pytest.raises(ValueError):
        p.rows(a, 5, 34)
    with pytest.raises(ValueError, match="page_size"):
        PagePool(4, 48)
    with pytest.raises(ValueError, match="31 bits"):
        PagePool(1 << 24, 128)
    p.free(a)
    with pytest.raises(KeyError):
        p.length(a)
