"""The page pool told what has been appended (track_writes): a copy or a move
that would miss tokens whose slots are out is refused, every other history
reads back the same tokens."""

import random

import pytest

from quantized_weight_skinny_amd.page_pool import NotWritten, OutOfPages, PagePool


def test_a_fork_of_tokens_that_are_not_appended_yet_is_not_extended():
    p = PagePool(8, 4, track_writes=True)
    a = p.new()
    p.extend(a, 2)
    b = p.fork(a)
    for seq in (a, b):                   # whoever writes first would get the copy
        before = (p.free_pages, p.table(seq), p.length(seq))
        with pytest.raises(NotWritten):
            p.extend(seq, 1)
        assert before == (p.free_pages, p.table(seq), p.length(seq)) and p.take_copies() == []
    p.written(a)                         # the fork shares the page
    p.extend(b, 1)
    assert p.take_copies() == [(p.table(a)[0], p.table(b)[0])]
    c = p.fork(b)                        # b's own token is not there yet
    with pytest.raises(NotWritten):
        p.extend(c, 1)
    p.truncate(c, 2)
    p.extend(c, 1)                       # without it the copy is whole


def test_slots_that_are_out_again_count_as_not_appended():
    p = PagePool(8, 4, track_writes=True)
    a = p.new()
    p.extend(a, 3)
    p.written(a)
    p.truncate(a, 1)
    p.extend(a, 2)
    b = p.fork(a)
    with pytest.raises(NotWritten):
        p.extend(b, 1)
    p.truncate(b, 1)
    p.extend(b, 1)


def test_compact_does_not_move_tokens_that_are_not_appended_yet():
    p = PagePool(8, 4, track_writes=True)
    a, b = p.new(), p.new()
    p.extend(a, 4)
    p.extend(b, 6)
    p.written(a)
    p.free(a)
    before = (p.free_pages, p.table(b))
    with pytest.raises(NotWritten):
        p.compact()
    assert before == (p.free_pages, p.table(b)) and p.take_copies() == []
    p.written(b)
    assert p.compact() == 2 and p.table(b) == [1, 0]
    p.take_copies()
    c = p.fork(b)
    p.extend(c, 1)                       # what was appended is known of the page's new place


def test_without_tracking_the_callers_word_is_taken():
    p = PagePool(8, 4)
    a = p.new()
    p.extend(a, 2)
    p.extend(p.fork(a), 1)
    p.written(a)


class Shadow:
    """Pages as lists of values, appends that wait in `out` (slot -> value), and
    what each sequence should hold once they are made."""

    def __init__(self, pages, size):
        self.pool, self.size = PagePool(pages, size, track_writes=True), size
        self.data, self.want, self.out, self.stamp = [[None] * size for _ in range(pages)], {}, {}, 0

    def slots(self, seq):
        return self.pool.slots(seq, 0, self.pool.length(seq))

    def drop_stale(self):
        live = {s for seq in self.want for s in self.slots(seq)}
        self.out = {s: v for s, v in self.out.items() if s in live}

    def extend(self, seq, n):
        at, size = self.pool.length(seq), self.size
        last = self.pool.table(seq)[at // size] if at % size else None
        shared = n > 0 and last is not None and self.pool.references(last) > 1
        missing = shared and any(last * size + o in self.out for o in range(at % size))
        before = (self.pool.free_pages, self.pool.table(seq), at)
        try:
            slots = self.pool.extend(seq, n)
        except NotWritten:
            assert missing and before == (self.pool.free_pages, self.pool.table(seq), at)
            return
        except OutOfPages:
            return
        assert not missing
        for s in slots:
            self.stamp += 1
            self.out[s] = self.stamp
            self.want[seq].append(self.stamp)

    def append(self):
        """Copies, then the appends, then the mark: a step of a serving loop."""
        before = [list(p) for p in self.data]
        for s, d in self.pool.take_copies():
            self.data[d] = list(before[s])
        for slot, v in self.out.items():
            self.data[slot // self.size][slot % self.size] = v
        self.out = {}
        for seq, want in self.want.items():
            self.pool.written(seq)
            assert [self.data[s // self.size][s % self.size] for s in self.slots(seq)] == want


@pytest.mark.parametrize("size", [1, 4, 16])
@pytest.mark.parametrize("seed", range(6))
def test_random_histories_with_appends_that_wait(size, seed):
    rng, s = random.Random(seed), Shadow(40, size)
    for _ in range(600):
        op, seqs = rng.random(), list(s.want)
        if op < 0.1 or not seqs:
            s.want[s.pool.new()] = []
        elif op < 0.45:
            s.extend(rng.choice(seqs), rng.randint(0, 2 * size))
        elif op < 0.60:
            seq = rng.choice(seqs)
            s.want[s.pool.fork(seq)] = list(s.want[seq])
        elif op < 0.72:
            seq = rng.choice(seqs)
            n = rng.randint(0, len(s.want[seq]))
            s.pool.truncate(seq, n)
            del s.want[seq][n:]
        elif op < 0.80:
            seq = rng.choice(seqs)
            s.pool.free(seq)
            del s.want[seq]
        elif op < 0.85:
            if s.out:
                with pytest.raises((NotWritten, RuntimeError)):
                    s.pool.compact()
            else:
                s.append()
                s.pool.compact()
        else:
            s.append()
        s.drop_stale()
    s.append()
