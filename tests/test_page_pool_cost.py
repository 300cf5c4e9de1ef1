"""What the page pool's books cost: every change takes time by the pages that it
touches, not by the copies that are pending. Bounds are twenty times and more
above what the operations take, and far below what a search of the pending
copies for each new one would (seconds)."""

import time

from quantized_weight_skinny_amd.page_pool import PagePool


def _seconds(f):
    t = time.perf_counter()
    f()
    return time.perf_counter() - t


def test_compacting_a_large_pool():
    n = 20000
    p = PagePool(2 * n, 16)
    low, high = p.new(), p.new()
    p.extend(low, 16 * n)
    p.extend(high, 16 * n)
    p.free(low)                              # every page in use moves
    assert _seconds(p.compact) < 0.8
    assert p.table(high) == list(range(n)) and len(p.take_copies()) == n
    assert p.free_pages == n


def test_many_copies_on_write():
    n = 12000
    p = PagePool(2 * n + 1, 16)
    seqs = []
    for _ in range(n):
        seqs.append(p.new())
        p.extend(seqs[-1], 1)
    forks = [p.fork(s) for s in seqs]

    def write():
        for f in forks:
            p.extend(f, 1)

    assert _seconds(write) < 0.8
    assert p.take_copies() == [(p.table(s)[0], p.table(f)[0]) for s, f in zip(seqs, forks)]
