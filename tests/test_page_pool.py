"""The page pool's books (no device needed): a model of the pool that keeps
every sequence's tokens by value, with the copies carried out on a list of
pages, must always read back the same tokens."""

import random

import pytest

from quantized_weight_skinny_amd.page_pool import OutOfPages, PagePool


class Shadow:
    """Pages as lists of values, and what each sequence should hold."""

    def __init__(self, pages, size):
        self.pool, self.data, self.want, self.size = PagePool(pages, size), [[None] * size for _ in range(pages)], {}, size
        self.stamp = 0

    def copies(self):
        pairs = self.pool.take_copies()
        src, dst = {s for s, _ in pairs}, [d for _, d in pairs]
        assert len(set(dst)) == len(dst) and not src & set(dst)
        before = [list(p) for p in self.data]
        for s, d in pairs:
            self.data[d] = before[s]

    def write(self, seq, n):
        slots = self.pool.extend(seq, n)
        self.copies()
        assert len(slots) == n
        for slot in slots:
            assert self.pool.references(slot // self.size) == 1      # nobody else sees the write
            self.stamp += 1
            self.data[slot // self.size][slot % self.size] = self.stamp
            self.want[seq].append(self.stamp)

    def check(self):
        used = set()
        for seq, want in self.want.items():
            assert self.pool.length(seq) == len(want)
            got = [self.data[s // self.size][s % self.size] for s in self.pool.slots(seq, 0, len(want))]
            assert got == want
            assert len(self.pool.table(seq)) == -(-len(want) // self.size)
            used |= set(self.pool.table(seq))
        assert self.pool.free_pages == self.pool.pages - len(used)
        for page in range(self.pool.pages):
            assert self.pool.references(page) == sum(page in self.pool.table(s) for s in self.want)


@pytest.mark.parametrize("size", [1, 4, 16])
@pytest.mark.parametrize("seed", range(5))
def test_random_histories(size, seed):
    rng, s = random.Random(seed), Shadow(40, size)
    for _ in range(400):
        op = rng.random()
        seqs = list(s.want)
        if op < 0.12 or not seqs:
            s.want[s.pool.new()] = []
        elif op < 0.55:
            seq = rng.choice(seqs)
            before = (s.pool.free_pages, s.pool.table(seq), s.pool.length(seq))
            try:
                s.write(seq, rng.randint(0, 3 * size))
            except OutOfPages:
                assert before == (s.pool.free_pages, s.pool.table(seq), s.pool.length(seq))
                assert s.pool.take_copies() == []
        elif op < 0.70:
            seq = rng.choice(seqs)
            s.want[s.pool.fork(seq)] = list(s.want[seq])
        elif op < 0.85:
            seq = rng.choice(seqs)
            n = rng.randint(0, len(s.want[seq]))
            s.pool.truncate(seq, n)
            del s.want[seq][n:]
        elif op < 0.93:
            seq = rng.choice(seqs)
            s.pool.free(seq)
            del s.want[seq]
        else:
            used = s.pool.compact()
            s.copies()
            assert all(p < used for q in s.want for p in s.pool.table(q))
        s.check()


def test_fork_copies_a_shared_last_page_once():
    p = PagePool(8, 4)
    a = p.new()
    p.extend(a, 6)
    b = p.fork(a)
    assert p.take_copies() == [] and p.free_pages == 6
    last = p.table(a)[1]
    p.extend(b, 1)                       # b writes into the shared half-full page
    assert p.take_copies() == [(last, p.table(b)[1])] and p.table(a)[1] == last
    p.extend(a, 1)                       # a is its only holder now
    assert p.take_copies() == []
    p.extend(b, 0)
    assert p.take_copies() == []


def test_pages_of_pending_copies_are_not_taken_again():
    """Several changes before the copies are made: no page is a source and a
    destination, or a destination twice, and nothing is written into a source."""
    p = PagePool(6, 4)
    a = p.new()
    p.extend(a, 2)
    x = p.table(a)[0]
    b = p.fork(a)
    p.extend(b, 1)                       # x -> y is pending
    y = p.table(b)[0]
    p.free(a)                            # x has no holder now, but must be read first
    p.free(b)                            # and y is still to be written
    c = p.new()
    p.extend(c, 2)
    d = p.fork(c)
    p.extend(d, 1)
    assert not {x, y} & {p.table(c)[0], p.table(d)[0]}
    pairs = p.take_copies()
    assert len({s for s, _ in pairs} | {t for _, t in pairs}) == 2 * len(pairs) == 4
    assert p.free_pages == 4


def test_a_copy_of_a_page_whose_own_copy_is_pending_reads_the_first():
    p = PagePool(8, 4)
    a = p.new()
    p.extend(a, 2)
    b = p.fork(a)
    p.extend(b, 1)                       # a's page -> b's is pending
    p.truncate(b, 2)
    c = p.fork(b)
    p.extend(c, 1)                       # b's page holds nothing yet: c's copy is of a's
    x, y, z = (p.table(s)[0] for s in (a, b, c))
    assert len({x, y, z}) == 3
    assert sorted(p.take_copies()) == sorted([(x, y), (x, z)])


def test_pages_that_compact_empties_are_not_taken_before_its_moves_are_made():
    p = PagePool(6, 4)
    a, b = p.new(), p.new()
    p.extend(a, 16)
    p.extend(b, 6)                       # pages 4 and 5
    p.truncate(a, 8)
    assert p.compact() == 4              # 4 and 5 move to 2 and 3
    assert p.table(b) == [2, 3]
    c = p.fork(b)
    with pytest.raises(OutOfPages):
        p.extend(c, 1)                   # its copy would be written into a page that a move reads
    p.take_copies()
    p.extend(c, 1)
    assert p.take_copies() == [(3, p.table(c)[1])] and p.free_pages == 1


def test_full_last_page_is_not_copied():
    p = PagePool(8, 4)
    a = p.new()
    p.extend(a, 4)
    b = p.fork(a)
    p.extend(b, 2)
    assert p.take_copies() == [] and p.table(a)[0] == p.table(b)[0]


def test_refusals():
    p = PagePool(2, 4)
    a = p.new()
    p.extend(a, 3)
    with pytest.raises(OutOfPages):
        p.extend(a, 6)
    assert p.length(a) == 3 and p.free_pages == 1
    with pytest.raises(ValueError):
        p.extend(a, -1)
    with pytest.raises(ValueError):
        p.truncate(a, 4)
    with pytest.raises(ValueError):
        p.slots(a, 2, 4)
    with pytest.raises(ValueError):
        PagePool(4, 0)
    b = p.fork(a)
    p.extend(b, 1)
    with pytest.raises(RuntimeError):
        p.compact()                      # a copy is still to be made
    p.free(a)
    with pytest.raises(KeyError):
        p.length(a)
