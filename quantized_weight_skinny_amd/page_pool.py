"""The books of a 4-bit cache's pages: which are free, who holds which, and the
copies that keep shared pages apart.

A sequence is a list of page indices and a length. Forking it shares every page
(a reference count each); the first write into a shared page gives the writer a
copy of its own. Copies are collected as (source, destination) pairs and made
on the device by one ``kv4_copy_pages`` launch over all layers. Nothing here
touches the device by itself, so the books can be kept, and tested, without
one.

    pool = PagePool(pages, page_size, track_writes=True)
    s = pool.new()
    slots = pool.extend(s, tokens)        # where the next tokens go
    copies = pool.take_copies()           # [(src, dst)] to be made before the next append
    pool.written(s)                       # the tokens have been appended
    fork = pool.fork(s)
    pool.truncate(s, length)              # rejected drafts leave
    pool.free(fork)

Copies are made before the append that follows them, so they hold what was
appended until then. Tokens whose slots are out but which are not appended yet
would be missing from a copy of their page (a fork's, when it is extended) and
from the place that compact moves it to. Append them first. With track_writes
the pool is told by written() and raises NotWritten instead of losing them;
without, it takes the caller's word.
"""


class OutOfPages(RuntimeError):
    """The pool has too few free pages for the request; nothing was changed.
    (Pages of copies that take_copies has not given out yet are not free.)"""


class NotWritten(RuntimeError):
    """A page would be copied or moved that has tokens which were not appended
    yet (track_writes); nothing was changed."""


class PagePool:
    def __init__(self, pages, page_size, track_writes=False):
        if pages < 0 or page_size < 1:
            raise ValueError("pages must be >= 0 and page_size >= 1")
        self.pages, self.page_size, self.track_writes = pages, page_size, track_writes
        self._refs = [0] * pages
        self._filled = [0] * pages                    # leading tokens of a page that were appended (track_writes)
        self._free = list(range(pages - 1, -1, -1))   # taken from the end
        self._held = {}                               # sequence -> [page, ...]
        self._len = {}
        self._next = 0
        self._copies = {}                             # destination -> source, of copies still to be made
        self._copied = set()                          # their pages,
        self._late = []                               # and those of them that nobody holds any more

    # ------------------------------------------------------------- queries

    @property
    def free_pages(self):
        return len(self._free)

    def length(self, seq):
        return self._len[seq]

    def table(self, seq):
        """The sequence's page indices, in order."""
        return list(self._held[seq])

    def references(self, page):
        return self._refs[page]

    def slots(self, seq, start, stop):
        """Slots (page * page_size + offset) of tokens start .. stop - 1."""
        if not 0 <= start <= stop <= self._len[seq]:
            raise ValueError(f"tokens {start} .. {stop} of a sequence of {self._len[seq]}")
        held, size = self._held[seq], self.page_size
        return [held[t // size] * size + t % size for t in range(start, stop)]

    # ------------------------------------------------------------- changes

    def new(self):
        """An empty sequence."""
        seq, self._next = self._next, self._next + 1
        self._held[seq], self._len[seq] = [], 0
        return seq

    def extend(self, seq, tokens):
        """Room for `tokens` more tokens; returns their slots. A shared last page
        that they would be written into is replaced by a copy first (see
        take_copies): the tokens in it must have been appended, else NotWritten
        with track_writes. Raises OutOfPages, and changes nothing, if the pool
        cannot hold them. Slots hold until the sequence is cut below them, or
        the pool compacted."""
        if tokens < 0:
            raise ValueError("tokens must be >= 0")
        held, at, size = self._held[seq], self._len[seq], self.page_size
        part = at % size != 0
        own = tokens > 0 and part and self._refs[held[at // size]] > 1   # a copy on write
        need = -(-(at + tokens) // size) - len(held) + own
        if need > len(self._free):
            raise OutOfPages(f"{need} pages needed, {len(self._free)} free")
        if own:
            last = held[at // size]
            if self.track_writes and self._filled[last] < at % size:
                raise NotWritten(f"page {last} is shared and has tokens that were not appended yet")
            page = self._take()
            self._copy(last, page)
            self._filled[page] = min(self._filled[last], at % size)
            self._drop(last)
            held[at // size] = page
        elif self.track_writes and tokens > 0 and part:
            self._filled[held[at // size]] = min(self._filled[held[at // size]], at % size)  # these slots are out again
        while len(held) * size < at + tokens:
            held.append(self._take())
        self._len[seq] = at + tokens
        return self.slots(seq, at, at + tokens)

    def written(self, seq):
        """The sequence's tokens have been appended, all of them (for track_writes)."""
        held, size = self._held[seq], self.page_size
        for i in range(len(held) - 1, -1, -1):
            if self._filled[held[i]] == size:
                break                                 # and so are those before it
            self._filled[held[i]] = max(self._filled[held[i]], min(size, self._len[seq] - i * size))

    def fork(self, seq):
        """A sequence of the same tokens that shares all of seq's pages. Tokens
        that were not appended yet must be before either is extended."""
        other = self.new()
        self._held[other], self._len[other] = list(self._held[seq]), self._len[seq]
        for page in self._held[other]:
            self._refs[page] += 1
        return other

    def truncate(self, seq, length):
        """Keeps the first `length` tokens; pages that hold none of them are released."""
        if not 0 <= length <= self._len[seq]:
            raise ValueError(f"length {length} of a sequence of {self._len[seq]}")
        held = self._held[seq]
        keep = -(-length // self.page_size)
        for page in held[keep:]:
            self._drop(page)
        del held[keep:]
        self._len[seq] = length

    def free(self, seq):
        """Releases the sequence."""
        self.truncate(seq, 0)
        del self._held[seq], self._len[seq]

    def compact(self):
        """Moves the pages in use to the lowest indices (each into a hole below
        it), so that the pool's end is free once the copies have been taken.
        Adds the moves to the copies and returns the number of pages in use.
        Copies must have been taken before, too: a page may not be a source
        and a destination at once; and all tokens must have been appended, as their
        slots change (else NotWritten with track_writes)."""
        if self._copies:
            raise RuntimeError("take_copies() first: a move must not meet a copy that is still to be made")
        if self.track_writes:
            for seq, held in self._held.items():
                if any(self._filled[p] < min(self.page_size, self._len[seq] - i * self.page_size)
                       for i, p in enumerate(held)):
                    raise NotWritten(f"sequence {seq} has tokens that were not appended yet")
        used = self.pages - len(self._free)
        holes = sorted(p for p in self._free if p < used)
        high = [p for p in range(used, self.pages) if self._refs[p]]
        to = dict(zip(high, holes))
        for src, dst in to.items():
            self._copy(src, dst)
            self._refs[dst], self._refs[src] = self._refs[src], 0
            self._filled[dst] = self._filled[src]
        for held in self._held.values():
            held[:] = [to.get(p, p) for p in held]
        self._free = [p for p in range(self.pages - 1, used - 1, -1) if p not in to]
        self._late = list(to)            # free once they have been read
        return used

    def take_copies(self):
        """The (source, destination) pairs to be made before anything is written
        to the pool again; afterwards none are pending."""
        out = [(src, dst) for dst, src in self._copies.items()]
        self._copies.clear()
        self._copied.clear()
        self._free += self._late
        self._late = []
        return out

    # ------------------------------------------------------------- inside

    def _take(self):
        page = self._free.pop()
        self._refs[page], self._filled[page] = 1, 0
        return page

    def _copy(self, src, dst):
        # a page whose own copy is still to be made is read where that reads
        src = self._copies.get(src, src)
        self._copies[dst] = src
        self._copied.update((src, dst))

    def _drop(self, page):
        self._refs[page] -= 1
        if self._refs[page] == 0:
            # a page of a copy that is still to be made must not be taken before it is
            (self._late if page in self._copied else self._free).append(page)
